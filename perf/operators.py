"""The decoder-block operators around the W8A8 expert layer: what is measured.

Three operators, each with INT8 and FP8 (OCP e4m3) codes:
  linear  the W8A8 matrix product with a scale per token and per output channel
          (projections of a decoder block, LM head), from bf16 tokens or from
          codes that are already there;
  ffn     the gated feed-forward block in W8A8 (a dense layer's FFN, or the
          shared expert whose gated result is added to the routed experts');
  norm    the norms before and after a block with its gate, residual scale and
          residual add, and the codes that the next product takes.

Where a float decides a code, the decision is defined in fp32 (the layer's own
rule): v = fl(x * inv_smooth), code = rint(fl(v * fl(qmax / max|v|))). Plain and
exact forms both follow that definition; everything else is rounded once.
"""
import math

import torch

own = False

DEV = "cuda"
LARGEST = 16384 * 8192 * 4096      # multiply-adds of the largest listed product
QMAX = {"int8": 127.0, "fp8": 448.0}


def _pad(k):
    return -(-k // 128) * 128


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token through an attention output projection: latency
        dict(name="linear 1 token", op="linear", T=1, K=4096, N=4096, fmt="int8", src="bf16",
             smooth=True, bias=False, out="bf16", add=False),
        # a decode batch against an LM head of odd vocabulary, fp32 logits
        dict(name="linear lm head", op="linear", T=32, K=4096, N=32003, fmt="int8", src="bf16",
             smooth=False, bias=False, out="fp32", add=False),
        # a chunk of a prefill through a fused QKV projection, FP8 codes
        dict(name="linear chunk fp8", op="linear", T=256, K=4096, N=6144, fmt="fp8", src="bf16",
             smooth=True, bias=False, out="bf16", add=False),
        # ragged batch, odd widths, codes made by an earlier operator, bias
        dict(name="linear odd codes", op="linear", T=1021, K=4000, N=4999, fmt="int8", src="codes",
             smooth=False, bias=True, out="bf16", add=False),
        # a whole prefill of 32 x 512 tokens: the largest product
        dict(name="linear prefill", op="linear", T=16384, K=4096, N=8192, fmt="int8", src="bf16",
             smooth=True, bias=False, out="bf16", add=False),
        # shared expert of one token beside the routed ones: gated and added
        dict(name="ffn 1 token", op="ffn", T=1, H=4096, F=2048, fmt="int8", smooth=True, add=True),
        # decode batch through a dense FFN, FP8
        dict(name="ffn decode fp8", op="ffn", T=32, H=8192, F=2048, fmt="fp8", smooth=False,
             add=False),
        # prefill through the shared expert, gated and added
        dict(name="ffn prefill", op="ffn", T=8192, H=4096, F=4096, fmt="int8", smooth=True,
             add=True),
        # one token: residual add, RMS norm, FP8 codes for the next projection
        dict(name="norm 1 token", op="norm", T=1, H=4096, kind="rms", post=False, gate="none",
             res="bf16", normed=False, codes="fp8", smooth=True),
        # prefill: residual add and RMS norm to bf16
        dict(name="norm prefill", op="norm", T=16384, H=4096, kind="rms", post=False, gate="none",
             res="bf16", normed=True, codes="none", smooth=False),
        # norms on both sides of the block, gate per channel, fp32 residual
        # stream, FP8 codes
        dict(name="norm sandwich", op="norm", T=8192, H=8192, kind="rms", post=True,
             gate="channel", res="fp32", normed=True, codes="fp8", smooth=True),
        # odd width, layer norm, gate per token, INT8 codes
        dict(name="norm odd layer", op="norm", T=1999, H=2047, kind="layer", post=True,
             gate="token", res="bf16", normed=True, codes="int8", smooth=False),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def _size(rng, lo, hi):
    """Log-uniform; half of the sizes are round ones, the rest as they fall."""
    v = _log(rng, lo, hi)
    step = rng.choice([1, 1, 16, 128])
    return max(lo, min(hi, v // step * step)) if v >= 4 * step else v


def draw(rng):
    op = rng.choice(["linear", "linear", "ffn", "ffn", "norm", "norm"])
    T = _size(rng, 1, 16384)
    fmt = rng.choice(["int8", "fp8"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "linear":
        K, N = _size(rng, 64, 8192), _size(rng, 64, 32768)
        if T * K * N > LARGEST:
            T = max(1, LARGEST // (K * N))
        out = rng.choice(["bf16", "bf16", "fp32"]) if fmt == "int8" else "bf16"
        return dict(op=op, T=T, K=K, N=N, fmt=fmt, src=rng.choice(["bf16", "bf16", "codes"]),
                    smooth=flag(), bias=flag(), out=out, add=out == "bf16" and flag())
    if op == "ffn":
        H, F = _size(rng, 128, 8192), _size(rng, 128, 8192)
        if 3 * T * H * F > LARGEST:
            T = max(1, LARGEST // (3 * H * F))
        return dict(op=op, T=T, H=H, F=F, fmt=fmt, smooth=flag(), add=flag())
    H = _size(rng, 64, 16384)
    T = min(T, max(1, 16384 * 4096 // H))
    return dict(op=op, T=T, H=H, kind=rng.choice(["rms", "rms", "layer"]), post=flag(),
                gate=rng.choice(["none", "token", "channel", "rows"]),
                res=rng.choice(["bf16", "fp32"]), normed=True,
                codes=rng.choice(["none", "int8", "fp8"]), smooth=flag())


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _tokens(g, T, H):
    """Tokens as they enter a product: N(0, 1) times a log-normal size per
    token, 1 % of the channels 20 times larger."""
    x = torch.randn(T, H, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    big = torch.rand(H, generator=g, device=DEV) < 0.01
    return torch.where(big, 20 * x, x).bfloat16(), big


def _inv_smooth(g, H, big):
    """1 / s of SmoothQuant: outlier channels shrink, the rest vary a little."""
    s = torch.exp(0.2 * torch.randn(H, generator=g, device=DEV))
    return 1.0 / torch.where(big, 6 * s, s)


def _weight(g, N, K, fmt):
    """Codes [N][K] and scales [N] of N(0, 1/K) weights quantised per row."""
    w = torch.randn(N, K, generator=g, device=DEV)
    a = w.abs().amax(1, keepdim=True)
    c = w * (QMAX[fmt] / a)
    c = c.round().to(torch.int8) if fmt == "int8" else c.clamp(-448, 448).to(torch.float8_e4m3fn)
    return c, (a[:, 0] / QMAX[fmt] / math.sqrt(K)).contiguous()


def _inputs(case, seed):
    g, c = _gen(seed), dict(case)
    s = {"case": c}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        s["w"], s["sw"] = _weight(g, N, K, c["fmt"])
        x, big = _tokens(g, T, K)
        s["inv"] = _inv_smooth(g, K, big) if c["smooth"] and c["src"] == "bf16" else None
        s["bias"] = torch.randn(N, generator=g, device=DEV) * 0.1 if c["bias"] else None
        if c["src"] == "codes":  # rows padded with zeros, as the operators that make codes give them
            q, s["sx"] = _codes(x.float(), c["fmt"])
            s["q"] = torch.nn.functional.pad(q, (0, _pad(K) - K)).to(
                torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn)
        else:
            s["x"] = x
        s["gate"] = s["add"] = None
        if c["add"]:
            s["gate"] = torch.rand(T, generator=g, device=DEV)
            s["add"] = torch.randn(T, N, generator=g, device=DEV).bfloat16()
    elif c["op"] == "ffn":
        T, H, F = c["T"], c["H"], c["F"]
        s["wgu"], s["sgu"] = _weight(g, 2 * F, H, c["fmt"])
        s["wd"], s["sd"] = _weight(g, H, F, c["fmt"])
        s["x"], big = _tokens(g, T, H)
        s["inv"] = _inv_smooth(g, H, big) if c["smooth"] else None
        s["gate"] = s["add"] = None
        if c["add"]:
            s["gate"] = torch.sigmoid(torch.randn(T, generator=g, device=DEV))
            s["add"] = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    else:
        T, H = c["T"], c["H"]
        s["y"], big = _tokens(g, T, H)
        s["res"] = (2 * torch.randn(T, H, generator=g, device=DEV)).to(
            torch.float32 if c["res"] == "fp32" else torch.bfloat16)
        s["w"] = 1 + 0.2 * torch.randn(H, generator=g, device=DEV)
        s["b"] = 0.1 * torch.randn(H, generator=g, device=DEV) if c["kind"] == "layer" else None
        s["pw"] = 1 + 0.2 * torch.randn(H, generator=g, device=DEV) if c["post"] else None
        s["inv"] = _inv_smooth(g, H, big) if c["smooth"] and c["codes"] != "none" else None
        s["gate"] = None
        if c["gate"] == "token":
            s["gate"] = torch.sigmoid(torch.randn(T, 1, generator=g, device=DEV))
        elif c["gate"] == "channel":
            s["gate"] = (0.5 + 0.2 * torch.randn(1, H, generator=g, device=DEV)).bfloat16()
        elif c["gate"] == "rows":
            s["gate"] = (0.5 + 0.2 * torch.randn(T, H, generator=g, device=DEV)).bfloat16()
        s["rs"], s["bs"] = 0.875, 1.25
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(s)
    return s


# --------------------------------------------------------- the framework's own
def _prepare_own(s):
    """The handles that a user's program keeps: weights laid out once."""
    import w8a8_int8_expert_amd as m
    c = s["case"]
    fp8 = c.get("fmt") == "fp8"
    if c["op"] == "linear":
        s["layer"] = m.W8A8Linear(c["K"], c["N"], fp8=fp8)
        s["layer"].load_quantized(s["w"], s["sw"], inv_smooth=s["inv"], bias=s["bias"])
        s["out_dtype"] = torch.float32 if c["out"] == "fp32" else torch.bfloat16
    elif c["op"] == "ffn":
        s["layer"] = m.W8A8FFN(c["H"], c["F"], fp8=fp8)
        s["layer"].load_quantized(s["wgu"], s["sgu"], s["wd"], s["sd"], inv_smooth=s["inv"])


def _run_own(s):
    c = s["case"]
    if c["op"] == "linear":
        if c["src"] == "codes":
            return s["layer"].forward(codes=(s["q"], s["sx"]), add=s["add"], gate=s["gate"],
                                      out_dtype=s["out_dtype"])
        return s["layer"].forward(s["x"], add=s["add"], gate=s["gate"], out_dtype=s["out_dtype"])
    if c["op"] == "ffn":
        return s["layer"].forward(s["x"], add=s["add"], gate=s["gate"])
    import w8a8_int8_expert_amd as m
    r = m.add_norm(s["y"], s["res"], norm=c["kind"], weight=s["w"], bias=s["b"], eps=1e-6,
                   post_weight=s["pw"], gate=s["gate"], residual_scale=s["rs"],
                   block_scale=s["bs"], normed=c["normed"],
                   codes=None if c["codes"] == "none" else c["codes"], inv_smooth=s["inv"])
    out = {"residual": r.residual}
    if c["normed"]:
        out["normed"] = r.normed
    if c["codes"] != "none":
        q = r.codes[:, :c["H"]]
        # INT8 codes as the numbers they stand for; e4m3 codes are numbers already
        out["codes"] = q.bfloat16() if c["codes"] == "int8" else q
        out["scales"] = r.scales
    return out


# ---------------------------------------------------------------- plain forms
def _codes(v, fmt):
    """Per-row codes (as fp32 numbers) and scales of fp32 rows."""
    a = v.abs().amax(1, keepdim=True)
    top = torch.full_like(a, QMAX[fmt])  # a tensor: a quotient with a number is not a division here
    rr = torch.where(a > 0, top / a, torch.zeros_like(a))
    p = (v * rr).clamp(-QMAX[fmt], QMAX[fmt])
    q = p.round() if fmt == "int8" else p.to(torch.float8_e4m3fn).float()
    return q, (a / top)[:, 0]


def _end(y, gate, add, dtype):
    if gate is not None:
        y = y * gate[:, None]
    if add is not None:
        y = y + add.float()
    return y.to(dtype)


def _norm(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
    v = v * w
    return v if b is None else v + b


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        if c["src"] == "codes":
            q, sx = s["q"][:, :c["K"]].float(), s["sx"]
        else:
            v = s["x"].float()
            q, sx = _codes(v if s["inv"] is None else v * s["inv"], c["fmt"])
        y = q @ s["w"].float().t() * sx[:, None] * s["sw"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return _end(y, s["gate"], s["add"], torch.float32 if c["out"] == "fp32" else torch.bfloat16)
    if c["op"] == "ffn":
        v = s["x"].float()
        q, sx = _codes(v if s["inv"] is None else v * s["inv"], c["fmt"])
        gu = q @ s["wgu"].float().t() * sx[:, None] * s["sgu"]
        gt, u = gu[:, :c["F"]], gu[:, c["F"]:]
        q, sh = _codes(gt * torch.sigmoid(gt) * u, c["fmt"])
        y = q @ s["wd"].float().t() * sh[:, None] * s["sd"]
        return _end(y, s["gate"], s["add"], torch.bfloat16)
    b = s["y"].float()
    if c["post"]:
        b = _norm(b, c["kind"], s["pw"], None)
    if s["gate"] is not None:
        b = b * s["gate"].float()
    r = s["rs"] * s["res"].float() + s["bs"] * b
    n = _norm(r, c["kind"], s["w"], s["b"])
    out = {"residual": r.to(s["res"].dtype)}
    if c["normed"]:
        out["normed"] = n.bfloat16()
    if c["codes"] != "none":
        q, out["scales"] = _codes(n if s["inv"] is None else n * s["inv"], c["codes"])
        out["codes"] = q.to(torch.bfloat16 if c["codes"] == "int8" else torch.float8_e4m3fn)
    return out


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _fp32_decision(v, top):
    """Codes of rows whose values are fp32 numbers, decided in fp32 as the
    definition says: the largest magnitude, its reciprocal step, one product."""
    v = v.to(torch.float32)
    big = torch.max(v, dim=1).values.maximum(-torch.min(v, dim=1).values)
    step = torch.div(torch.full_like(big, top), big)
    step[big == 0] = 0
    lvl = torch.mul(v, step.unsqueeze(1))
    lvl = torch.minimum(torch.maximum(lvl, torch.tensor(-top, device=v.device)),
                        torch.tensor(top, device=v.device))
    lvl = torch.round(lvl) if top == 127 else lvl.to(torch.float8_e4m3fn)
    return lvl.to(torch.float64), big.to(torch.float64) / top


def _product(q, w, out):
    """out[t][n] = sum_k q[t][k] w[n][k] in 64 bits, some output channels at a time."""
    for n in range(0, w.shape[0], 4096):
        part = w[n:n + 4096].to(torch.float32).to(torch.float64)
        out[:, n:n + 4096] = torch.matmul(q, part.t())
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    c, D = case, torch.float64
    new = lambda t, n: torch.empty(t, n, dtype=D, device=DEV)  # noqa: E731

    def finish(y):
        if s["gate"] is not None:
            y *= s["gate"].to(D).unsqueeze(1)
        if s["add"] is not None:
            y += s["add"].to(D)
        return y

    def quantised():
        x = s["x"].to(torch.float32)
        return _fp32_decision(x if s["inv"] is None else torch.mul(x, s["inv"]), QMAX[c["fmt"]])

    if c["op"] == "linear":
        if c["src"] == "codes":
            q, sx = s["q"].to(torch.float32).to(D)[:, :c["K"]], s["sx"].to(D)
        else:
            q, sx = quantised()
        y = _product(q, s["w"], new(c["T"], c["N"]))
        y *= sx.unsqueeze(1)
        y *= s["sw"].to(D)
        if s["bias"] is not None:
            y += s["bias"].to(D)
        return finish(y)
    if c["op"] == "ffn":
        q, sx = quantised()
        gu = _product(q, s["wgu"], new(c["T"], 2 * c["F"]))
        gu *= sx.unsqueeze(1)
        gu *= s["sgu"].to(D)
        gate, up = gu.chunk(2, dim=1)
        h = gate / (1 + torch.exp(-gate)) * up
        q, sh = _fp32_decision(h, QMAX[c["fmt"]])
        y = _product(q, s["wd"], new(c["T"], c["H"]))
        y *= sh.unsqueeze(1)
        y *= s["sd"].to(D)
        return finish(y)

    def norm(v, w, bias):
        v = v.to(D)
        if c["kind"] == "layer":
            var, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
            v = (v - mean) / torch.sqrt(var + 1e-6)
        else:
            v = v / torch.sqrt(torch.mean(v * v, dim=1, keepdim=True) + 1e-6)
        v = v * w.to(D)
        return v if bias is None else v + bias.to(D)

    branch = s["y"].to(D)
    if c["post"]:
        branch = norm(branch, s["pw"], None)
    if s["gate"] is not None:
        branch = branch * s["gate"].to(D)
    r = s["res"].to(D) * s["rs"] + branch * s["bs"]
    n = norm(r, s["w"], s["b"])
    out = {"residual": r}
    if c["normed"]:
        out["normed"] = n
    if c["codes"] != "none":
        v = n.to(torch.float32)
        out["codes"], out["scales"] = _fp32_decision(
            v if s["inv"] is None else torch.mul(v, s["inv"]), QMAX[c["codes"]])
    return out


# --------------------------------------------------------------------- work
def work(case):
    c, T = case, case["T"]
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        x = T * K * (1 if c["src"] == "codes" else 2) + (4 * T if c["src"] == "codes" else 0)
        by = x + N * K + 4 * N * (2 if c["bias"] else 1) + T * N * (4 if c["out"] == "fp32" else 2)
        by += (4 * K if c["smooth"] and c["src"] == "bf16" else 0)
        by += (2 * T * N + 4 * T if c["add"] else 0)
        return {"bytes": by, "flops": 2 * T * N * K}
    if c["op"] == "ffn":
        H, F = c["H"], c["F"]
        by = 2 * T * H + 3 * H * F + 4 * (2 * F + H) + 2 * T * H
        by += (4 * H if c["smooth"] else 0) + (2 * T * H + 4 * T if c["add"] else 0)
        return {"bytes": by, "flops": 6 * T * H * F}
    H = c["H"]
    per = 2 + 2 * (4 if c["res"] == "fp32" else 2) + (2 if c["normed"] else 0)
    per += (1 if c["codes"] != "none" else 0) + (2 if c["gate"] == "rows" else 0)
    return {"bytes": per * T * H + 4 * H * 2 + (4 * T if c["codes"] != "none" else 0),
            "flops": (20 if c["post"] else 12) * T * H}
