"""The decoder block around the W8A8 expert layer: torch plumbing of the block
operators of libmoe_w8a8 (include/moe_w8a8.h).

    q, s = act_quant(x, inv_smooth)                 per-token codes
    W8A8Linear(K, N).forward(x or codes=(q, s))     W8A8 matrix product
    W8A8FFN(H, F).forward(x or codes=(q, s))        W8A8 gated feed-forward block
    add_norm(y, residual, ...)                      norms around a block, gate,
                                                    residual add, codes

Every tensor is checked (type, shape, strides, device) before a pointer is
handed to the library. Calls run on torch's current stream of the operands'
device, whichever device is current. Outputs and workspaces come from torch's
allocator call by call, so calls on different streams, and graphs captured
from them, share nothing but the weights.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

import w8a8_int8_expert_amd as _m

_BF16, _F32, _I8, _E4M3 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
_OUT_TYPES, _ONLY_BF16 = (_BF16, _F32), (_BF16,)
_FORMATS = {"int8": 0, "fp8": 1}
_NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}
_MAX_PITCH = 1 << 26  # elements, the library's limit
# A call of one token is a few microseconds of GPU work: what the binding does
# per call is kept as small. The stream's handle, the current device and whether a
# graph is being captured come from the functions that torch.cuda wraps (a call with
# GPU operands finds torch.cuda initialised).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else \
    (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)


def _fail(msg):
    raise _m.MoEW8A8Error(msg)


def _device(device):
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _call(name, device, *args, captured=None):
    """One library call with `device` current, on torch's current stream of it;
    `captured` is called after it where the call was captured into a graph."""
    if device.type != "cuda":
        _fail("the operands must be on a GPU")
    i = device.index
    if _current_device() != i:
        with torch.cuda.device(i):
            return _call(name, device, *args, captured=captured)
    rc = getattr(_m._lib or _m.load_library(), name)(*args, _raw_stream(i))
    if rc != 0:
        _m._check(rc, name)
    if captured is not None and _capturing():
        captured()


def _rows(t, name, dtypes, T, width, device):
    """(address, row pitch) of a [T][width] tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        _fail("%s must be a torch tensor" % name)
    if t.dtype not in dtypes:
        _fail("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.shape != (T, width):
        _fail("%s must have shape %s, got %s" % (name, (T, width), tuple(t.shape)))
    if t.device != device:
        _fail("%s must be on %s, got %s" % (name, device, t.device))
    ld, step = t.stride()
    if step != 1 and width > 1:
        _fail("the rows of %s must be contiguous" % name)
    if T <= 1:
        ld = width
    elif ld < width:
        _fail("the rows of %s overlap (row stride %d for %d columns)" % (name, ld, width))
    elif ld > _MAX_PITCH:
        _fail("the rows of %s lie too far apart (row stride %d)" % (name, ld))
    return t.data_ptr(), ld


def _vector(t, name, n, device):
    """Address of a contiguous fp32 [n] tensor, None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != _F32 or t.numel() != n or \
            not t.is_contiguous() or t.device != device:
        _fail("%s must be a contiguous fp32 tensor of %d values on %s" % (name, n, device))
    return t.data_ptr()


def _empty_codes(T, K, fp8, device):
    if not 1 <= K <= 65536:
        _fail("unsupported width %d" % K)
    pitch = (K + 127) // 128 * 128
    return (torch.empty(T, pitch, dtype=_E4M3 if fp8 else _I8, device=device),
            torch.empty(T, dtype=_F32, device=device))


def act_quant(x, inv_smooth=None, fp8: bool = False):
    """Per-token codes of bf16 rows x [T][K], times inv_smooth (fp32 [K]):
    (codes [T][Kp], scales fp32 [T]), Kp = moe_w8a8_row_pitch(K), zeros past K."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _fail("x must be a [T][K] tensor")
    T, K = x.shape
    dev = x.device
    px, ld = _rows(x, "x", _ONLY_BF16, T, K, dev)
    inv = _vector(inv_smooth, "inv_smooth", K, dev)
    q, s = _empty_codes(T, K, fp8, dev)
    _call("moe_w8a8_act_quant", dev, K, int(bool(fp8)), px, ld, T, inv, q.data_ptr(), s.data_ptr())
    return q, s


class _Weights:
    """Packed codes and scales of one weight matrix, and the struct that names
    them.

    Its buffers have their places for good: a captured call follows what is loaded
    later. Of the two optional vectors (the tokens' inv_smooth and the bias) it
    keeps the places of those there were: one that a later load leaves out holds
    ones or zeros from then on, and one that the captured call went without can no
    longer be loaded."""

    def __init__(self, K, N, fp8, gated, device):
        size = _m.moe_w8a8_linear_codes_bytes(N, K, gated)
        if size == 0:
            _fail("unsupported weight shape [%d][%d]" % (N, K))
        self.K, self.N, self.fp8, self.gated, self.device = K, N, fp8, gated, device
        self.codes = torch.empty(size, dtype=_I8, device=device)
        self.scale = torch.empty(_m.moe_w8a8_linear_scales(N, gated), dtype=_F32,
                                 device=device)
        self.inv_smooth = torch.empty(K, dtype=_F32, device=device)
        self.bias = torch.empty(N, dtype=_F32, device=device)
        self.struct = _m.moe_w8a8_linear_weights(K, N, int(fp8), int(gated),
                                                 self.codes.data_ptr(), self.scale.data_ptr(),
                                                 None, None)
        self.ref = ctypes.byref(self.struct)
        self.without = set()  # what a captured call went without

    def captured(self, coded):
        """A call was captured (`coded`: of tokens that it codes itself)."""
        if self.struct.bias is None:
            self.without.add("bias")
        if coded and self.struct.inv_smooth is None:
            self.without.add("smoothing")

    def _check_vectors(self, smoothing, bias):
        for name, t in (("smoothing", smoothing), ("bias", bias)):
            if t is not None and name in self.without:
                _fail("a call of this operator without %s was captured into a graph, which would "
                      "go on without: load these weights into a new operator" % name)

    def vectors(self, inv_smooth, bias):
        """Copy the two optional vectors in; None turns one off."""
        for name, t, none in (("inv_smooth", inv_smooth, 1.0), ("bias", bias, 0.0)):
            own = getattr(self, name)
            if t is None:
                own.fill_(none)
            else:
                own.copy_(t.detach().reshape(own.shape))
            setattr(self.struct, name, None if t is None else own.data_ptr())

    # The checks stand apart, so that a call that has several things to load
    # refuses before it has changed any of them.
    def check_source(self, w, smooth, bias):
        self._check_vectors(smooth, bias)
        _vector(bias, "bias", self.N, self.device)
        return (*_rows(w, "weight", (_BF16, _F32), self.N, self.K, self.device),
                _vector(smooth, "smooth", self.K, self.device))

    def quantise(self, w, smooth, bias=None):
        p, ld, ps = self.check_source(w, smooth, bias)
        _call("moe_w8a8_linear_quantise", self.device, self.ref, p, 1 if w.dtype == _F32 else 0,
              ld, ps)
        self.vectors(None if smooth is None else 1.0 / smooth, bias)

    def check_codes(self, q, s, inv_smooth, bias):
        self._check_vectors(inv_smooth, bias)
        _vector(bias, "bias", self.N, self.device)
        _vector(inv_smooth, "inv_smooth", self.K, self.device)
        types = (_E4M3, _I8) if self.fp8 else (_I8,)  # int8: e4m3 bytes, as the layer takes them
        p, ld = _rows(q, "codes", types, self.N, self.K, self.device)
        ps = _vector(s, "scales", self.N, self.device)
        if ps is None:
            _fail("codes come with their scales")
        return p, ld, ps

    def load(self, q, s, inv_smooth=None, bias=None):
        p, ld, ps = self.check_codes(q, s, inv_smooth, bias)
        _call("moe_w8a8_linear_pack", self.device, self.ref, p, ld, ps)
        self.vectors(inv_smooth, bias)


class _Product:
    """What the two products share: their operands, their workspace's size (a
    function of the number of tokens, asked for once each) and their result."""

    def _workspace(self, T):
        n = self._sizes.get(T)
        if n is None:
            if len(self._sizes) >= 4096:
                self._sizes.clear()
            n = self._sizes[T] = self._size(T)
        return n, torch.empty(n, dtype=torch.uint8, device=self.device) if n else None

    def _captured(self):
        for w in self._all:
            w.captured(True)

    def _captured_codes(self):
        for w in self._all:
            w.captured(False)

    def _operands(self, x, codes, K, N, add, gate, out, out_dtype):
        dev = self.device
        if (x is None) == (codes is None):
            _fail("give either x or codes")
        first = x if codes is None else codes[0]
        if not isinstance(first, torch.Tensor) or first.dim() != 2:
            _fail("tokens must be a [T][K] tensor")
        T = first.shape[0]
        act = _m.moe_w8a8_act()
        if codes is None:
            act.x, act.ld_x = _rows(x, "x", _ONLY_BF16, T, K, dev)
        else:
            pitch = (K + 127) // 128 * 128
            act.q, ld = _rows(first, "codes", (_E4M3,) if self.fp8 else (_I8,), T, pitch, dev)
            if ld != pitch:
                _fail("codes must be contiguous")
            act.s = _vector(codes[1], "code scales", T, dev)
            if act.s is None and T > 0:
                _fail("codes come with their scales")
        res = _m.moe_w8a8_result()
        if out is None:
            if out_dtype is not None and out_dtype not in _OUT_TYPES:
                _fail("out_dtype must be bfloat16 or float32, got %s" % out_dtype)
            out = torch.empty(T, N, dtype=out_dtype or _BF16, device=dev)
            res.out, res.ld_out = out.data_ptr(), N
        else:
            res.out, res.ld_out = _rows(out, "out", _OUT_TYPES, T, N, dev)
            if out_dtype is not None and out.dtype != out_dtype:
                _fail("out must be %s, got %s" % (out_dtype, out.dtype))
        res.out_type = 1 if out.dtype == _F32 else 0
        if gate is not None:
            res.gate = _vector(gate, "gate", T, dev)
        if add is not None:
            res.add, res.ld_add = _rows(add, "add", _ONLY_BF16, T, N, dev)
        return T, act, res, out


class W8A8Linear(_Product):
    """y = x . W^T in W8A8: INT8 (or, with fp8=True, e4m3) codes with a scale
    per token and per output channel. Fill it with quantise() or
    load_quantized(), then call forward(). Captured calls follow later loads; a
    load that brings smoothing or a bias which a captured call went without is
    refused."""

    def __init__(self, in_features: int, out_features: int, device="cuda", fp8: bool = False):
        _m.load_library()
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.fp8, self.device = bool(fp8), _device(device)
        self._w = _Weights(self.in_features, self.out_features, self.fp8, False, self.device)
        self._all = (self._w,)
        self._sizes = {}

    def _size(self, T):
        return _m.moe_w8a8_linear_workspace_size(self.out_features, self.in_features, T)

    def quantise(self, weight, smooth=None, bias=None):
        """weight: fp32 or bf16 [N][K]. smooth: SmoothQuant scales s fp32 [K]
        (the weight's columns are multiplied by s, the tokens by 1/s)."""
        self._w.quantise(weight, smooth, bias)

    def load_quantized(self, q, s, inv_smooth=None, bias=None):
        """Codes [N][K] (int8; with fp8 float8_e4m3fn, or its bytes as int8)
        quantised elsewhere and their scales fp32 [N]; inv_smooth fp32 [K]
        multiplies the tokens."""
        self._w.load(q, s, inv_smooth, bias)

    def forward(self, x=None, codes=None, add=None, gate=None, out=None,
                out_dtype: Optional["torch.dtype"] = None):  # noqa: F821
        """out = gate[:, None] * (x . W^T + bias) + add, rounded once to bf16
        (or fp32). x: bf16 [T][K], or codes=(q, s) as act_quant and add_norm
        give them in the weights' format. gate fp32 [T]; add bf16 [T][N] (may be out itself)."""
        T, act, res, out = self._operands(x, codes, self.in_features, self.out_features, add,
                                          gate, out, out_dtype)
        n, ws = self._workspace(T)
        _call("moe_w8a8_linear", self.device, self._w.ref, ctypes.byref(act), T,
              ctypes.byref(res), ws.data_ptr() if n else None, n,
              captured=self._captured if codes is None else self._captured_codes)
        return out

    __call__ = forward


class W8A8FFN(_Product):
    """Gated feed-forward block in W8A8: down(silu(gate(x)) * up(x)), the hidden
    rows requantised per token. Loads and captured calls as W8A8Linear."""

    def __init__(self, hidden: int, ffn: int, device="cuda", fp8: bool = False,
                 out_features: Optional[int] = None):
        _m.load_library()
        self.hidden, self.ffn = int(hidden), int(ffn)
        self.out_features = self.hidden if out_features is None else int(out_features)
        self.fp8, self.device = bool(fp8), _device(device)
        self._gu = _Weights(self.hidden, 2 * self.ffn, self.fp8, True, self.device)
        self._dn = _Weights(self.ffn, self.out_features, self.fp8, False, self.device)
        self._all = (self._gu, self._dn)
        self._sizes = {}

    def _size(self, T):
        return _m.moe_w8a8_ffn_workspace_size(self.hidden, self.ffn, self.out_features, T)

    def quantise(self, w_gate_up, w_down, smooth=None, bias=None):
        """w_gate_up: fp32 or bf16 [2F][H], gate rows then up rows; w_down
        [N][F]; smooth fp32 [H]; bias fp32 [N] of the down projection."""
        self._dn.check_source(w_down, None, bias)
        self._gu.quantise(w_gate_up, smooth)
        self._dn.quantise(w_down, None, bias)

    def load_quantized(self, q_gate_up, s_gate_up, q_down, s_down, inv_smooth=None, bias=None):
        """Codes [2F][H] (gate rows, then up rows) and [N][F] quantised
        elsewhere, their scales fp32 [2F] and [N]."""
        self._dn.check_codes(q_down, s_down, None, bias)
        self._gu.load(q_gate_up, s_gate_up, inv_smooth)
        self._dn.load(q_down, s_down, None, bias)

    def forward(self, x=None, codes=None, add=None, gate=None, out=None,
                out_dtype: Optional["torch.dtype"] = None):  # noqa: F821
        """out = gate[:, None] * ffn(x) + add; operands as W8A8Linear.forward.
        As a shared expert: ffn.forward(x, add=moe.forward(x, ...), gate=g)."""
        T, act, res, out = self._operands(x, codes, self.hidden, self.out_features, add, gate,
                                          out, out_dtype)
        n, ws = self._workspace(T)
        _call("moe_w8a8_ffn", self.device, self._gu.ref, self._dn.ref, ctypes.byref(act), T,
              ctypes.byref(res), ws.data_ptr() if n else None, n,
              captured=self._captured if codes is None else self._captured_codes)
        return out

    __call__ = forward


class AddNorm(NamedTuple):
    residual: Optional["torch.Tensor"]  # noqa: F821
    normed: Optional["torch.Tensor"]  # noqa: F821
    codes: Optional["torch.Tensor"]  # noqa: F821
    scales: Optional["torch.Tensor"]  # noqa: F821


def add_norm(y, residual=None, norm="rms", weight=None, bias=None, eps: float = 1e-6,
             post_norm=None, post_weight=None, post_bias=None, gate=None, gate_group=None,
             residual_scale: float = 1.0, block_scale: float = 1.0, residual_out=True,
             normed=True, codes: Optional[str] = None, inv_smooth=None) -> AddNorm:
    """Norms before and after a block, in one pass over its rows:

        r = residual_scale * residual + block_scale * gate * post(y)
        n = norm(r)

    y: bf16 [T][H]; residual: bf16 or fp32 [T][H], or None.
    norm, post_norm: "rms", "layer" or "none"; weights and biases fp32 [H].
    post_norm defaults to `norm`'s kind where post_weight is given, else none.
    gate: fp32 [T] or [T][1] (per token), or bf16 [G][H]: row t takes gate row
    t // gate_group, where gate_group defaults to ceil(T / G) (one row: a gate
    per channel; T rows: a gate of its own; a row per sequence otherwise).
    residual_out, normed: True (a new tensor), False, or the tensor to write
    (residual_out may be residual, normed may be y).
    codes: None, "int8" or "fp8": codes of n * inv_smooth for the next product.
    Returns AddNorm(residual, normed, codes, scales), None where not asked."""
    if not isinstance(y, torch.Tensor) or y.dim() != 2:
        _fail("y must be a [T][H] tensor")
    T, H = y.shape
    dev = y.device
    if post_norm is None and (post_weight is not None or post_bias is not None):
        post_norm = norm
    if norm not in _NORMS or post_norm not in _NORMS:
        _fail("norm must be 'rms', 'layer' or 'none'")
    if codes is not None and codes not in _FORMATS:
        _fail("codes must be 'int8' or 'fp8'")
    p_y, ld_y = _rows(y, "y", _ONLY_BF16, T, H, dev)
    p_res = p_out = p_norm = p_token = p_rows = q = s = None
    ld_res = ld_out = ld_norm = ld_gate = group = 0
    rtype = _BF16
    if residual is not None:
        p_res, ld_res = _rows(residual, "residual", _OUT_TYPES, T, H, dev)
        rtype = residual.dtype
    elif isinstance(residual_out, torch.Tensor):
        rtype = residual_out.dtype
    if residual_out is True:
        residual_out = torch.empty(T, H, dtype=rtype, device=dev)
        p_out, ld_out = residual_out.data_ptr(), H
    elif residual_out is False or residual_out is None:
        residual_out = None
    else:
        p_out, ld_out = _rows(residual_out, "residual_out",
                              _OUT_TYPES if residual is None else (rtype,), T, H, dev)
    if normed is True:
        normed = torch.empty(T, H, dtype=_BF16, device=dev)
        p_norm, ld_norm = normed.data_ptr(), H
    elif normed is False or normed is None:
        normed = None
    else:
        p_norm, ld_norm = _rows(normed, "normed", _ONLY_BF16, T, H, dev)
    if gate is not None and T > 0:
        if isinstance(gate, torch.Tensor) and gate.dtype == _F32:
            if gate.shape not in ((T,), (T, 1)):
                _fail("an fp32 gate must be [T] or [T][1]")
            p_token = _vector(gate, "gate", T, dev)
        else:
            if not isinstance(gate, torch.Tensor) or gate.dim() != 2 or gate.shape[0] < 1:
                _fail("gate must be fp32 [T] or bf16 [G][H]")
            G = gate.shape[0]
            p_rows, ld_gate = _rows(gate, "gate", _ONLY_BF16, G, H, dev)
            group = -(-T // G) if gate_group is None else int(gate_group)
            if group < 1 or -(-T // group) > G:
                _fail("gate has %d rows, too few for %d tokens in groups of %d" % (G, T, group))
            group = min(group, T)  # (a number past 64 bits would wrap to another)
    if codes is not None:
        q, s = _empty_codes(T, H, codes == "fp8", dev)
    a = _m.moe_w8a8_add_norm_args(
        H, _NORMS[norm], _NORMS[post_norm], 1 if rtype == _F32 else 0, _FORMATS.get(codes, 0),
        eps, residual_scale, block_scale, p_y, ld_y, p_res, ld_res, p_out, ld_out,
        None if post_weight is None else _vector(post_weight, "post_weight", H, dev),
        None if post_bias is None else _vector(post_bias, "post_bias", H, dev),
        None if weight is None else _vector(weight, "weight", H, dev),
        None if bias is None else _vector(bias, "bias", H, dev), p_token, p_rows, ld_gate, group,
        p_norm, ld_norm,
        None if codes is None or inv_smooth is None else _vector(inv_smooth, "inv_smooth", H, dev),
        None if q is None else q.data_ptr(), None if s is None else s.data_ptr())
    _call("moe_w8a8_add_norm", dev, ctypes.byref(a), T)
    return AddNorm(residual_out, normed, q, s)
