"""Plain 64-bit reference of the block operators, and the error bounds of the
kernels' fp32 arithmetic. u = 2^-24 is half an fp32 step, relative."""
from __future__ import annotations

import torch

U = 2.0 ** -24
QMAX = {False: 127.0, True: 448.0}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def pitch(K):
    return -(-K // 128) * 128


def row_codes(v, fp8):
    """The code rule on fp32 rows v (CPU), decided in fp32 as it is defined:
    (codes as fp32 numbers, scales fp32)."""
    v = v.to(torch.float32)
    finite = torch.isfinite(v).all(1)
    a = torch.where(finite, v.abs().amax(1), torch.ones(()))
    lift = torch.where(a < 2.0 ** -64, torch.tensor(2.0 ** 64), torch.tensor(1.0))
    al = a * lift
    top = torch.full_like(al, QMAX[fp8])
    rr = torch.where(a > 0, top / al, torch.zeros_like(al))
    p = (v * lift[:, None]) * rr[:, None]
    if fp8:
        q = p.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    else:
        q = p.round().clamp(-127.0, 127.0)
    s = al / top * torch.where(lift > 1, torch.tensor(2.0 ** -64), torch.tensor(1.0))
    q = torch.where(finite[:, None], q, torch.zeros(()))
    s = torch.where(finite, s, torch.tensor(float("nan")))
    return q, s


def smoothed(x, inv):
    """fl32(x * inv_smooth) of bf16 tokens."""
    v = x.float()
    return v if inv is None else v * inv.float()


def fp8_sum_bound(q, w):
    """Largest error of the FP8 matrix instructions' sums of q . w^T: the
    products of each 8 consecutive k are kept to 13 bits below the group's
    largest, and the K/8 group sums are added in fp32."""
    K = pitch(q.shape[1])
    pad = lambda t: torch.nn.functional.pad(t.abs(), (0, K - t.shape[1]))  # noqa: E731
    qa, wa = pad(q.double()), pad(w.double())
    g = lambda t: t.reshape(t.shape[0], K // 8, 8).amax(2)  # noqa: E731
    return 7 * 2.0 ** -13 * (g(qa) @ g(wa).t()) + (K // 8) * U * (qa @ wa.t())


def product(q, s, w, sw, fp8, bias=None):
    """(y, bound) in 64 bits of s * sw * (q . w^T) + bias: the bound counts the
    conversion of the sum, two products and the bias add (u each), and the FP8
    sums' own error."""
    q, w = q.double(), w.double()
    scale = s.double()[:, None] * sw.double()[None, :]
    y = (q @ w.t()) * scale
    err = 3 * U * y.abs()
    if fp8:
        err = err + fp8_sum_bound(q, w) * scale.abs() * (1 + 4 * U)
    if bias is not None:
        y = y + bias.double()
        err = err + U * y.abs()
    return y, err


def finish(y, err, dtype, gate=None, add=None):
    """Gate, add and the rounding to dtype: (exact value, bound)."""
    if gate is not None:
        g = gate.double()[:, None]
        y, err = y * g, err * g.abs()
        err = err + U * y.abs()
    if add is not None:
        y = y + add.double()
        err = err + U * y.abs()
    err = err * (1 + 8 * U) + half_step(dtype) * (y.abs() + err)
    return y, err + 1e-44


def check(got, want, bound, what):
    """Element by element: |got - want| <= bound; not finite where want is not."""
    got, want = got.double().cpu(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN elsewhere" % what
    over = ((got - want).abs() - bound)[fine]
    if over.numel() and over.max() > 0:
        i = int(torch.argmax(torch.where(fine, (got - want).abs() - bound,
                                         torch.full((), -1.0, dtype=torch.double))))
        r, c = divmod(i, want.shape[1])
        raise AssertionError("%s: [%d][%d] got %r want %r bound %r (%d of %d over)" % (
            what, r, c, float(got[r, c]), float(want[r, c]), float(bound[r, c]),
            int((over > 0).sum()), over.numel()))


def hidden(g, u, gerr, uerr):
    """h = silu(g) u and its error bound: |silu'| <= 1.1, |silu(g)| <= |g|, the
    exponential's argument rounding (|g| u, times |h|) and its own error, the
    reciprocal's and the products' (16 u in all: the hardware exponential and
    reciprocal are within 1 ulp = 2u each, amplified by at most 1 through
    1/(1+e); the products and sums u each)."""
    sg = g / (1 + torch.exp(-g))
    h = sg * u
    err = 1.1 * gerr * u.abs() + sg.abs() * uerr + 1.1 * gerr * uerr
    return h, err + (16 + 2 * g.abs()) * U * h.abs()


def requantised(h, herr, fp8):
    """Codes and scales of h in 64 bits, and per element by how much the
    kernel's code may differ (0 where h is further than its error from a
    rounding midpoint), and the scales' relative error."""
    qmax = QMAX[fp8]
    a = h.abs().amax(1)
    rel = torch.where(a > 0, herr.amax(1) / a.clamp_min(1e-300), torch.zeros_like(a)) + 4 * U
    v = torch.where(a[:, None] > 0, h * (qmax / a.clamp_min(1e-300))[:, None],
                    torch.zeros_like(h))
    dv = herr * (qmax / a.clamp_min(1e-300))[:, None] + v.abs() * rel[:, None]
    if not fp8:
        q = v.round().clamp(-127, 127)
        lo, hi = (v - dv).round().clamp(-127, 127), (v + dv).round().clamp(-127, 127)
    else:
        enc = lambda t: t.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
        # the fp32 value that is coded: one more rounding of v
        dv = dv + v.abs() * 2 * U
        q, lo, hi = enc(v), enc(v - dv), enc(v + dv)
    return q, a / qmax, torch.maximum((hi - q).abs(), (q - lo).abs()), rel
