"""Plain 64-bit reference of the operators between the projections (qk_norm_rope,
paged_attention) and of token_logprobs, with bounds that count the kernels' fp32
roundings. u = 2^-24 is half an fp32 step, relative; a bf16 rounding is half a step,
2^-8."""
from __future__ import annotations

import math

import torch

import block_ref as R

U, HALF = 2.0 ** -24, 2.0 ** -8
BF, F32, F64, E4, I8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, torch.int8
TYPES = {"bf16": BF, "int8": I8, "fp8": E4}


class Step:
    """A batch on the host: new tokens and lengths of its sequences, their pages."""

    def __init__(self, lens, page, seed=0, spare=2, T=None, cut=None):
        self.lens, self.page = lens, page
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(0, l) // page) for _, l in lens]
        width = max(need + [1]) + 1
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.cu = [0]
        for n, _ in lens:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1] if T is None else T
        self.most = max([n for n, _ in lens] + [0])
        self.longest = max([l for _, l in lens] + [0])

    def batch(self, m, most=None, longest=None):
        t = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        return m.SequenceBatch(t(self.cu), t([l for _, l in self.lens]), self.table.cuda(),
                               self.most if most is None else most,
                               self.longest if longest is None else longest)


def cached(shape, fmt, seed):
    """Cache contents on the host: (elements, scales or None)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if fmt == "bf16":
        return x.to(BF), None
    q, s = R.row_codes(x.reshape(-1, shape[-1]), fmt == "fp8")
    return q.reshape(shape).to(TYPES[fmt]), s.reshape(shape[:-1])


def dense(x, s, step, b, h):
    """Keys (or values) of one sequence and kv head in 64 bits, [length][D], and which of
    them lie in pages that exist."""
    L = step.lens[b][1]
    p = torch.arange(L)
    page = step.table[b][p // step.page].long()
    ok = (page >= 0) & (page < x.shape[0])
    y = x.float().double()[page.clamp(0, x.shape[0] - 1), h, p % step.page]
    if s is not None:
        y = y * s.double()[page.clamp(0, x.shape[0] - 1), h, p % step.page][:, None]
    return y, ok


def seen(n, L, causal, window, ok):
    """[n][L]: which keys each of the last n places of L sees."""
    place = torch.arange(L - n, L)[:, None]
    key = torch.arange(L)[None]
    m = ok[None].expand(n, L).clone()
    if causal:
        m &= key <= place
    if window:
        m &= key > place - window
    return m


def attention(q, k, ks, v, vs, step, heads, scale, causal=True, window=0):
    """(out, bound) fp64 [T][heads * D] of bf16 q [T][heads * D]; rows behind the last
    sequence are NaN. The bound: a score's fp32 sum of D exact products (D u of their
    absolute sum) and three products and a difference by which it may be off (with the
    base-2 exponent's ulp), a probability then rounded to bf16 once and to fp32 by its
    value's scale, sums over the keys in fp32, and the result's rounding."""
    T, Hkv, D = q.shape[0], k.shape[1], k.shape[3]
    G = heads // Hkv
    out = torch.full((T, heads * D), math.nan, dtype=F64)
    err = torch.zeros(T, heads * D, dtype=F64)
    for b, (n, L) in enumerate(step.lens):
        for h in range(Hkv if n else 0):
            kk, ok = dense(k, ks, step, b, h)
            vv, _ = dense(v, vs, step, b, h)
            m = seen(n, L, causal, window, ok)
            kz = torch.where(ok[:, None] & m.any(0)[:, None], kk, torch.zeros((), dtype=F64))
            rows = slice(step.cu[b], step.cu[b] + n)
            for j in range(h * G, (h + 1) * G):
                cols = slice(j * D, (j + 1) * D)
                qq = q[rows, cols].double()
                z = (qq @ kz.t()) * scale
                dz = (D + 4) * U * (qq.abs() @ kz.abs().t()) * abs(scale) + 4 * U * z.abs()
                z = torch.where(m, z, torch.full((), -math.inf, dtype=F64))
                top = z.amax(1, keepdim=True) if L else torch.zeros(n, 1, dtype=F64)
                none = ~m.any(1)
                top = torch.where(none[:, None], torch.zeros((), dtype=F64), top)
                p = torch.exp(z - top)
                # relative error of a probability: of its score and of the row's largest
                dmax = torch.where(m, dz, torch.zeros((), dtype=F64)).amax(1, keepdim=True) \
                    if L else torch.zeros(n, 1, dtype=F64)
                rel = torch.where(m, dz + dmax + 4 * U * (z - top).abs(),
                                  torch.zeros((), dtype=F64)) + 8 * U
                l = p.sum(1, keepdim=True)
                lrel = ((p * rel).sum(1, keepdim=True) / l.clamp_min(1e-300)) + (L + 16) * U
                # a masked place has no part, whatever it holds
                vz = torch.where(torch.isfinite(vv), vv, torch.zeros((), dtype=F64))
                w = p / l.clamp_min(1e-300)
                o = w @ vz
                e = (w * (rel + HALF + 2 * U)) @ vz.abs()
                e = (e + (w @ vz.abs()) * (lrel + (L + 16) * U)) * (1 + HALF)
                for c in torch.nonzero(~torch.isfinite(vv).all(1)).flatten().tolist():
                    o = o + torch.where(m[:, c:c + 1], torch.where(
                        torch.isfinite(vv[c]), torch.zeros((), dtype=F64), vv[c]),
                        torch.zeros((), dtype=F64))
                o = torch.where(none[:, None], torch.zeros((), dtype=F64), o)
                out[rows, cols] = o
                err[rows, cols] = e + HALF * (o.abs().nan_to_num(0, 0, 0) + e) + 1e-30
    return out, err


def rope(x, w, eps, norm, place, freq, pairs):
    """(y, bound) fp64 of head rows x bf16 [n][heads][D]: the square sum's D/8 + 8 fp32
    adds, mean, root, quotient and two products; an angle's fraction of a turn rounded to
    fp32 (pi u), sine and cosine of it (4 u), two products and a sum; and of far positions
    this form's own rounding of the angle to fp64, 2^-53 of it."""
    D = x.shape[2]
    y = x.double()
    err = torch.zeros_like(y)
    if norm:
        r = 1 / torch.sqrt((y * y).mean(2, keepdim=True) + eps)
        y = y * r
        if w is not None:
            y = y * w.double()
        err = (D / 16 + 12) * U * y.abs()
    if freq is not None:
        H = freq.shape[0]
        a = place.double()[:, None, None] * freq.double()
        c, s = torch.cos(a), torch.sin(a)
        i0 = torch.arange(H) * 2 if pairs else torch.arange(H)
        i1 = i0 + 1 if pairs else i0 + H
        p, q, dp, dq = y[..., i0].clone(), y[..., i1].clone(), err[..., i0], err[..., i1]
        y, err = y.clone(), err.clone()
        e = dp + dq + (12 * U + 2.0 ** -53 * a.abs()) * (p.abs() + q.abs())
        y[..., i0], y[..., i1] = p * c - q * s, q * c + p * s
        err[..., i0] = e
        err[..., i1] = e
    return y, err


def logprobs(x, tokens, top, steps):
    """(logprobs, entropy, top tokens, top logprobs) and bounds, 64 bits, rows x [T][V].
    `steps`: fp32 adds that a value goes through. A difference to the row's largest is
    rounded once (u of it), an exponential is within 2 ulp of it, a sum takes `steps`
    roundings, the logarithm two ulp."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    s = e.sum(1)
    de = torch.where(e > 0, d, torch.zeros((), dtype=F64)).abs()
    far = (e * de).sum(1) / s                       # mean distance, weighted
    rel = (steps + 8) * U + 2 * U * far
    z = torch.log(s)
    dz = rel + 4 * U * z.abs()
    lp = torch.full((x.shape[0],), math.nan, dtype=F64)
    if tokens is not None:
        ok = (tokens >= 0) & (tokens < x.shape[1])
        lp[ok] = (x[torch.arange(x.shape[0])[ok], tokens[ok]] - m[ok, 0]) - z[ok]
    ent = z + far
    far2 = (e * de * de).sum(1) / s
    dent = dz + (2 * rel + (steps + 8) * U) * far + 4 * U * far2 + 4 * U * ent.abs()
    order = torch.sort(x, dim=1, descending=True, stable=True)
    tt = order.indices[:, :top]
    tl = order.values[:, :top] - m - z[:, None]
    slack = lambda v: 4 * U * (v.abs() + z.abs().reshape(-1, *[1] * (v.dim() - 1)))  # noqa: E731
    return lp, dz + slack(lp), ent, dent, tt, tl, dz[:, None] + slack(tl)
