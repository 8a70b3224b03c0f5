"""Attention between a decoder block's projections, over a paged cache in the W8A8
layer's quantisation, and log probabilities from the LM head's logits: torch plumbing
of libmoe_w8a8 (include/moe_w8a8.h).

    cache = KVCache(num_pages, page_size, kv_heads, head_dim, "fp8")
    batch = SequenceBatch(cu_tokens, lengths, pages, max_tokens, max_length)
    q = qk_norm_rope(qkv(codes=...), cache, batch, heads, inv_freq=...)
    y = proj(paged_attention(q, cache, batch))
    r = token_logprobs(lm_head(codes=..., out_dtype=torch.float32), tokens, top=20)

Every tensor is checked (type, shape, strides, device) before a pointer is handed to
the library. Calls run on torch's current stream of the operands' device, whichever
device is current. Outputs and workspaces come from torch's allocator call by call, so
calls on different streams, and graphs captured from them, share nothing but the cache
and the batch's arrays.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

import w8a8_int8_expert_amd as _m

from .block import _BF16, _E4M3, _F32, _I8, _ONLY_BF16, _OUT_TYPES, _call, _device, _fail, _rows, \
    _vector

_I32, _I64, _F64 = torch.int32, torch.int64, torch.float64
_CACHE_TYPES = {_I8: 0, _E4M3: 1, _BF16: 2}
_CACHE_FORMATS = {"int8": _I8, "fp8": _E4M3, "bf16": _BF16}


class KVCache:
    """Keys and values of many sequences in pages: k, v [pages][kv heads][page size]
    [head dim], bf16, or int8 / float8_e4m3fn codes with k_scale, v_scale fp32 [pages]
    [kv heads][page size]. Which page holds what is the caller's (SequenceBatch)."""

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
                 format: str = "bf16", device="cuda"):
        if format not in _CACHE_FORMATS:
            _fail("format must be 'bf16', 'int8' or 'fp8'")
        device = _device(device)
        shape = (int(num_pages), int(kv_heads), int(page_size), int(head_dim))
        if min(shape) < 1:
            _fail("unsupported cache %s" % (shape,))
        # (empty places are zeros; float8 tensors are cleared as bytes)
        dtype = _CACHE_FORMATS[format]
        k, v = (torch.zeros(shape, dtype=_I8 if dtype == _E4M3 else dtype, device=device)
                .view(dtype) for _ in range(2))
        ks = vs = None
        if format != "bf16":
            ks, vs = (torch.zeros(shape[:3], dtype=_F32, device=device) for _ in range(2))
        self._set(k, v, ks, vs)

    @classmethod
    def of(cls, k, v, k_scale=None, v_scale=None) -> "KVCache":
        """A cache over tensors that exist (kept, not copied). Pages must be contiguous;
        from page to page there may be more (the layers of a larger buffer)."""
        self = cls.__new__(cls)
        self._set(k, v, k_scale, v_scale)
        return self

    @staticmethod
    def _pages(t, name, dtype, shape, device, step):
        if not isinstance(t, torch.Tensor):
            _fail("%s must be a torch tensor" % name)
        if t.dtype != dtype:
            _fail("%s must be %s, got %s" % (name, dtype, t.dtype))
        if tuple(t.shape) != shape:
            _fail("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
        if t.device != device:
            _fail("%s must be on %s, got %s" % (name, device, t.device))
        each = t[0].numel()
        if not t[0].is_contiguous():
            _fail("the pages of %s must be contiguous" % name)
        stride = t.stride(0) if shape[0] > 1 else -(-each // step) * step
        if stride < each or stride % step:
            _fail("the pages of %s lie %d elements apart: at least %d and a multiple of %d are "
                  "wanted" % (name, stride, each, step))
        return t.data_ptr(), stride

    def _set(self, k, v, k_scale, v_scale):
        _m.load_library()
        if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.dtype not in _CACHE_TYPES:
            _fail("k must be a bf16, int8 or float8_e4m3fn tensor [pages][kv heads][page size]"
                  "[head dim]")
        shape = tuple(k.shape)
        if min(shape) < 1 or shape[0] >= 1 << 31:
            _fail("unsupported cache %s" % (shape,))
        P, H, S, D = shape
        if D not in (64, 128, 256) or S not in (16, 32, 64, 128, 256) or H > 1024:
            _fail("unsupported cache: head dim %d (64, 128, 256), page size %d (16 to 256, a power "
                  "of two), %d kv heads (up to 1024)" % (D, S, H))
        self.device = k.device
        pk, stride = self._pages(k, "k", k.dtype, shape, self.device, 16)
        pv, stride_v = self._pages(v, "v", k.dtype, shape, self.device, 16)
        if stride != stride_v:
            _fail("the pages of k and v lie differently far apart")
        ps = pt = None
        scale_stride = 0
        if k.dtype == _BF16:
            if k_scale is not None or v_scale is not None:
                _fail("a bf16 cache has no scales")
        else:
            ps, scale_stride = self._pages(k_scale, "k_scale", _F32, shape[:3], self.device, 4)
            pt, other = self._pages(v_scale, "v_scale", _F32, shape[:3], self.device, 4)
            if scale_stride != other:
                _fail("the pages of k_scale and v_scale lie differently far apart")
        for p in (pk, pv, ps, pt):
            if p is not None and p % 16:
                _fail("the cache's tensors must be aligned to 16 bytes")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = P, H, S, D
        self.struct = _m.moe_w8a8_kv_cache(P, S, H, D, _CACHE_TYPES[k.dtype], pk, pv, stride, ps,
                                           pt, scale_stride)
        self.ref = ctypes.byref(self.struct)


class SequenceBatch:
    """The sequences of a step. Sequence b's new tokens are rows cu_tokens[b] ..
    cu_tokens[b + 1] - 1 of the step's tensors and the last ones of its lengths[b] keys;
    place p of it lies in cache page pages[b][p // page_size].

    cu_tokens int32 [B + 1], lengths int32 [B], pages int32 [B][width] (entries that are
    not used may hold anything, -1 say). max_tokens: the most new tokens of a sequence, a
    bound. max_length: about the longest length (it sizes launches only). The tensors are
    kept and read when the kernels run: a captured call follows what is written there."""

    def __init__(self, cu_tokens, lengths, pages, max_tokens: int, max_length: int):
        _m.load_library()
        for t, name, dim in ((lengths, "lengths", 1), (cu_tokens, "cu_tokens", 1),
                             (pages, "pages", 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != _I32 or t.dim() != dim:
                _fail("%s must be an int32 tensor of %d dimension%s" % (name, dim, "s"[:dim - 1]))
            if t.device != lengths.device:
                _fail("%s must be on %s, got %s" % (name, lengths.device, t.device))
            if dim == 1 and not t.is_contiguous():
                _fail("%s must be contiguous" % name)
        B, width = pages.shape
        if lengths.shape[0] != B or cu_tokens.shape[0] != B + 1:
            _fail("a batch of %d sequences has %d lengths and %d ends of tokens" % (
                B, lengths.shape[0], cu_tokens.shape[0] - 1))
        ld = pages.stride(0) if B > 1 else width
        if width > 1 and pages.stride(1) != 1:
            _fail("the rows of pages must be contiguous")
        if ld < width or ld > 1 << 26:
            _fail("the rows of pages overlap or lie too far apart (row stride %d)" % ld)
        if B > 1 << 20:
            _fail("at most 2^20 sequences, got %d" % B)
        top = (1 << 31) - 1
        if not 0 <= int(max_tokens) <= top or not 0 <= int(max_length) <= top:
            _fail("max_tokens and max_length must be in [0, 2^31)")
        self.device, self.num_seqs = lengths.device, B
        self.max_tokens, self.max_length = int(max_tokens), int(max_length)
        self.cu_tokens, self.lengths, self.pages = cu_tokens, lengths, pages
        self.struct = _m.moe_w8a8_batch(B, self.max_tokens, self.max_length, width,
                                        cu_tokens.data_ptr(), lengths.data_ptr(),
                                        pages.data_ptr() if width else None, ld)
        self.ref = ctypes.byref(self.struct)
        self._sizes = {}

    def _workspace(self, cache, heads, T):
        """Bytes of attention's workspace for T rows over this kind of cache, asked for
        once each."""
        s = cache.struct
        key = (s.page_size, s.kv_heads, s.head_dim, s.format, heads, T)
        n = self._sizes.get(key)
        if n is None:
            if len(self._sizes) >= 4096:
                self._sizes.clear()
            n = self._sizes[key] = _m.moe_w8a8_paged_attention_workspace_size(s, self.struct,
                                                                              heads, T)
        return n


def _step(cache, batch, rows, name):
    if not isinstance(cache, KVCache) or not isinstance(batch, SequenceBatch):
        _fail("give a KVCache and a SequenceBatch")
    dev = cache.device
    if batch.device != dev:
        _fail("the batch must be on %s, got %s" % (dev, batch.device))
    if not isinstance(rows, torch.Tensor) or rows.dim() != 2:
        _fail("%s must be a [T][width] tensor" % name)
    return dev, rows.shape[0]


def qk_norm_rope(qkv, cache: KVCache, batch: SequenceBatch, heads: int, norm: bool = False,
                 q_weight=None, k_weight=None, eps: float = 1e-6, inv_freq=None,
                 interleaved: bool = False, positions=None, out=None):
    """Queries and keys normed for each head and rotated by position; keys and values go
    into the cache at their tokens' places; returns the queries, bf16 [T][heads * D].

    qkv: bf16 [T][(heads + 2 kv heads) * D], query heads, key heads, value heads (what
    W8A8Linear gives). norm: RMS norm over each head (eps), times q_weight, k_weight (fp32
    [D]). inv_freq: fp64 [R / 2], the angle of one position for each rotated pair; the first
    R elements of a head are rotated in pairs (i, i + R / 2), interleaved (2 i, 2 i + 1);
    None: no rotation. positions: int64 [T], or None: each token's place in its sequence.
    out: bf16 [T][heads * D], may be qkv[:, :heads * D]. Rows behind the batch's last
    sequence are not written."""
    dev, T = _step(cache, batch, qkv, "qkv")
    D = cache.head_dim
    heads = int(heads)
    if not 1 <= heads <= 65536 // D:
        _fail("heads must be in [1, %d], got %d" % (65536 // D, heads))
    p, ld = _rows(qkv, "qkv", _ONLY_BF16, T, (heads + 2 * cache.kv_heads) * D, dev)
    if not norm and (q_weight is not None or k_weight is not None):
        _fail("weights come with norm=True")
    R = 0
    p_freq = p_pos = None
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != _F64 or \
                inv_freq.dim() != 1 or not inv_freq.is_contiguous() or inv_freq.device != dev:
            _fail("inv_freq must be a contiguous fp64 vector on %s" % dev)
        R = 2 * inv_freq.shape[0]
        if R < 16 or R > D or R % 16:
            _fail("inv_freq has %d values: a multiple of 8 up to %d is wanted" % (R // 2, D // 2))
        p_freq = inv_freq.data_ptr()
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype != _I64 or \
                positions.shape != (T,) or not positions.is_contiguous() or \
                positions.device != dev:
            _fail("positions must be a contiguous int64 tensor of %d values on %s" % (T, dev))
        p_pos = positions.data_ptr()
    if out is None:
        out = torch.empty(T, heads * D, dtype=_BF16, device=dev)
        p_q, ld_q = out.data_ptr(), heads * D
    else:
        p_q, ld_q = _rows(out, "out", _ONLY_BF16, T, heads * D, dev)
        if T == 1 and p_q == p:
            ld_q = ld
    a = _m.moe_w8a8_qk_norm_rope_args(
        heads, int(bool(norm)), R, int(bool(interleaved)), eps, p, ld, p_q, ld_q,
        None if q_weight is None else _vector(q_weight, "q_weight", D, dev),
        None if k_weight is None else _vector(k_weight, "k_weight", D, dev), p_freq, p_pos)
    _call("moe_w8a8_qk_norm_rope", dev, ctypes.byref(a), cache.ref, batch.ref, T)
    return out


def paged_attention(q, cache: KVCache, batch: SequenceBatch, scale: Optional[float] = None,
                    causal: bool = True, window: int = 0, out=None):
    """Attention of the batch's new tokens over the cache: bf16 [T][heads * D] from q of
    that shape (heads: a multiple of the cache's kv heads; query head j reads kv head
    j // (heads // kv heads)). A token at place p of its sequence sees the keys c < length
    with c <= p (causal) and c > p - window (window > 0); one that sees none gets zeros.
    scale: of the scores, 1 / sqrt(D) by default. Rows behind the batch's last sequence are
    not written."""
    dev, T = _step(cache, batch, q, "q")
    D, width = cache.head_dim, q.shape[1]
    heads = width // D
    if width != heads * D or heads < 1 or heads % cache.kv_heads or width > 65536:
        _fail("q has %d columns: a multiple of %d heads of %d up to 65536 is wanted" % (
            width, cache.kv_heads, D))
    window = int(window)
    if not 0 <= window < 1 << 31:
        _fail("window must be in [0, 2^31), got %d" % window)
    p, ld = _rows(q, "q", _ONLY_BF16, T, width, dev)
    if out is None:
        out = torch.empty(T, width, dtype=_BF16, device=dev)
        p_o, ld_o = out.data_ptr(), width
    else:
        p_o, ld_o = _rows(out, "out", _ONLY_BF16, T, width, dev)
    n = batch._workspace(cache, heads, T)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    a = _m.moe_w8a8_attention_args(heads, int(bool(causal)), window,
                                   D ** -0.5 if scale is None else scale, p, ld, p_o, ld_o)
    _call("moe_w8a8_paged_attention", dev, ctypes.byref(a), cache.ref, batch.ref, T,
          ws.data_ptr() if n else None, n)
    return out


class TokenLogprobs(NamedTuple):
    logprobs: Optional["torch.Tensor"]  # noqa: F821
    entropy: Optional["torch.Tensor"]  # noqa: F821
    top_tokens: Optional["torch.Tensor"]  # noqa: F821
    top_logprobs: Optional["torch.Tensor"]  # noqa: F821


_logprob_sizes = {}


def token_logprobs(logits, tokens=None, top: int = 0, entropy: bool = True) -> TokenLogprobs:
    """Of each row of logits (bf16 or fp32 [T][V]): the log probability of tokens[t]
    (int64 [T]; NaN for one outside the vocabulary), the entropy (nats), and the `top` (up
    to 64) likeliest tokens, in falling order, of equal logits the lower token first, with
    their log probabilities. Returns TokenLogprobs(logprobs fp32 [T], entropy fp32 [T],
    top_tokens int64 [T][top], top_logprobs fp32 [T][top]), None where not asked."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        _fail("logits must be a [T][V] tensor")
    T, V = logits.shape
    dev = logits.device
    if not 1 <= V <= 1 << 20:
        _fail("unsupported vocabulary of %d" % V)
    top = int(top)
    if not 0 <= top <= min(V, 64):
        _fail("top must be in [0, %d], got %d" % (min(V, 64), top))
    p, ld = _rows(logits, "logits", _OUT_TYPES, T, V, dev)
    if tokens is None and not entropy and top == 0:
        _fail("nothing is asked for")
    lp = p_tokens = ent = tt = tl = None
    if tokens is not None:
        if not isinstance(tokens, torch.Tensor) or tokens.dtype != _I64 or \
                tokens.shape != (T,) or not tokens.is_contiguous() or tokens.device != dev:
            _fail("tokens must be a contiguous int64 tensor of %d values on %s" % (T, dev))
        p_tokens = tokens.data_ptr()
        lp = torch.empty(T, dtype=_F32, device=dev)
    if entropy:
        ent = torch.empty(T, dtype=_F32, device=dev)
    if top:
        tt = torch.empty(T, top, dtype=_I64, device=dev)
        tl = torch.empty(T, top, dtype=_F32, device=dev)
    key = (V, top, T)
    n = _logprob_sizes.get(key)
    if n is None:
        if len(_logprob_sizes) >= 4096:
            _logprob_sizes.clear()
        n = _logprob_sizes[key] = _m.moe_w8a8_token_logprobs_workspace_size(V, top, T)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    a = _m.moe_w8a8_logprobs_args(
        V, 1 if logits.dtype == _F32 else 0, top, p, ld, p_tokens,
        None if lp is None else lp.data_ptr(), None if ent is None else ent.data_ptr(),
        None if tt is None else tt.data_ptr(), None if tl is None else tl.data_ptr())
    _call("moe_w8a8_token_logprobs", dev, ctypes.byref(a), T, ws.data_ptr() if n else None, n)
    return TokenLogprobs(lp, ent, tt, tl)
