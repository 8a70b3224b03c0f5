"""The block operators (act_quant, W8A8Linear, W8A8FFN, add_norm) on the GPU
against plain 64-bit forms: codes exactly, everything else within bounds that
count the kernels' roundings (tests/block_ref.py)."""
import sys

import pytest
import torch

import block_ref as R
from moe_testlib import unpack_tiled

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_int8_expert_amd as m
    m.load_library()
    return m


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def seed_of(*a):
    s = 0
    for v in a:
        s = (s * 1000003 + int(v)) % (1 << 31)
    return s


def tokens(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g))
    x[:, :: max(1, K // 3)] *= 20
    return x.to(BF)


def weight(N, K, fp8, seed):
    g = torch.Generator().manual_seed(seed + 77)
    w = torch.randn(N, K, generator=g)
    q, s = R.row_codes(w, fp8)
    return (q.to(E4) if fp8 else q.to(torch.int8)), s / K ** 0.5


def vec(n, seed, lo=0.5, hi=1.5):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed + 5)) * (hi - lo) + lo


def cu(t):
    return None if t is None else t.cuda()


# --------------------------------------------------------------- act_quant
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 7), (5, 64), (2, 127), (4, 128), (9, 129), (17, 513),
                                 (6, 1024), (4, 2047), (3, 4096), (2, 8193), (3, 16384),
                                 (1, 20001), (2, 33000), (1, 65536)])
def test_act_quant(lib, T, K, fp8):
    say("[act_quant]", T, K, fp8)
    x = tokens(T, K, seed_of(T, K))
    inv = vec(K, K) if K % 2 else None
    q, s = lib.act_quant(x.cuda(), cu(inv), fp8=fp8)
    torch.cuda.synchronize()
    want, ws = R.row_codes(R.smoothed(x, inv), fp8)
    assert q.shape == (T, R.pitch(K)) and q.dtype == (E4 if fp8 else torch.int8)
    got = q.cpu().float()
    assert torch.equal(got[:, :K], want) and torch.equal(s.cpu(), ws)
    assert not got[:, K:].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_act_quant_rows_out_of_the_ordinary(lib, fp8):
    """Zero rows, rows below 2^-64 and of subnormals, the largest bf16, and rows
    holding NaN or an infinity (codes 0, scale NaN, neighbours untouched)."""
    K = 300
    x = tokens(10, K, 3).float()
    x[1] = 0
    x[2] *= 2.0 ** -100
    x[3] = 0
    x[3, 5] = 2.0 ** -133
    x[3, 6] = -(2.0 ** -132)
    x[4, 7] = 3.3895e38
    x[5, 299] = float("nan")
    x[6, 0] = float("inf")
    x[7, 100] = float("-inf")
    x[7, 101] = float("nan")
    x = x.to(BF)
    q, s = lib.act_quant(x.cuda(), fp8=fp8)
    want, ws = R.row_codes(x.float(), fp8)
    assert torch.equal(q.cpu().float()[:, :K], want)
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(ws))
    assert torch.equal(torch.nan_to_num(s.cpu()), torch.nan_to_num(ws))
    assert torch.isnan(ws[5:8]).all() and not torch.isnan(ws[8:]).any()


@pytest.mark.parametrize("off,extra", [(0, 8), (1, 3), (3, 0), (7, 9)])
def test_act_quant_strided_rows(lib, off, extra):
    T, K = 6, 777
    big = tokens(T, K + off + extra, 11).cuda()
    x = big[:, off:off + K]
    q, s = lib.act_quant(x)
    want, ws = R.row_codes(x.cpu().float(), False)
    assert torch.equal(q.cpu().float()[:, :K], want) and torch.equal(s.cpu(), ws)


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,K", [(2, 1), (32, 128), (34, 200), (130, 300)])
def test_weights_packed(lib, N, K, fp8, gated):
    """Quantised and loaded weights hold the same codes, in the layout the
    header defines: fragment tiles, zeros in the padding, gated rows in
    alternating runs of 32."""
    from w8a8_int8_expert_amd.block import _Weights
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(N * K))
    w[N // 2] = 0
    smooth = vec(K, N)
    for src in (w, w.to(BF)):
        a = _Weights(K, N, fp8, gated, torch.device("cuda", 0))
        a.quantise(src.cuda(), smooth.cuda())
        q, s = R.row_codes(src.float() * smooth, fp8)
        b = _Weights(K, N, fp8, gated, torch.device("cuda", 0))
        b.load((q.to(E4) if fp8 else q.to(torch.int8)).cuda(), s.cuda())
        torch.cuda.synchronize()
        assert torch.equal(a.scale, b.scale)
        if fp8:  # a negative value that rounds to zero keeps its sign when quantised
            assert torch.equal(a.codes.view(E4).float(), b.codes.view(E4).float())
        else:
            assert torch.equal(a.codes, b.codes)
        Np, Kp = b.scale.numel(), R.pitch(K)
        rows = unpack_tiled(b.codes.cpu().numpy(), 1, Np, Kp)[0]
        rows = torch.from_numpy(rows.copy())
        vals = rows.view(E4).float() if fp8 else rows.float()
        F = N // 2
        for p in range(Np):
            n = p if not gated else (p // 32 % 2) * F + p // 64 * 32 + p % 32
            real = p < N if not gated else p // 64 * 32 + p % 32 < F
            if real:
                assert torch.equal(vals[p, :K], q[n]) and not rows[p, K:].any()
                assert b.scale[p].item() == s[n].item()
            else:
                assert not rows[p].any() and b.scale[p].item() == 0


# ------------------------------------------------------------------- linear
LINEAR = [
    # T, K, N
    (1, 1, 1), (1, 64, 16), (1, 4096, 100), (2, 129, 17), (3, 1000, 33), (4, 12288, 40), (1, 16384, 33), (1, 48000, 33), (3, 5400, 35), (40, 5000, 64), (50, 2100, 4200),
    (64, 4100, 1000), (2, 64, 1 << 20), (70, 9000, 30),
    (4, 300, 257), (5, 127, 15), (15, 512, 48), (16, 2048, 31), (17, 128, 16), (31, 640, 130),
    (33, 4097, 64), (48, 256, 333), (63, 1024, 5), (64, 1100, 96), (65, 128, 128), (65, 1, 1),
    (100, 2000, 300), (128, 512, 129), (129, 384, 255), (200, 4096, 500), (256, 1024, 1024),
    (300, 130, 2000), (511, 640, 1000), (1000, 256, 1100), (1537, 320, 2100), (3333, 192, 4000),
    (4100, 128, 4200),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(lib, T, K, N, fp8):
    say("[linear]", T, K, N, fp8)
    seed = seed_of(T, K, N, fp8)
    x, (w, sw) = tokens(T, K, seed), weight(N, K, fp8, seed)
    inv = vec(K, seed) if seed % 2 else None
    bias = vec(N, seed, -1, 1) if seed % 3 else None
    lin = lib.W8A8Linear(K, N, fp8=fp8)
    lin.load_quantized(w.cuda(), sw.cuda(), inv_smooth=cu(inv), bias=cu(bias))
    y = lin(x.cuda())
    f = lin(x.cuda(), out_dtype=F32)
    codes = lib.act_quant(x.cuda(), cu(inv), fp8=fp8)
    yc = lin(codes=codes, out_dtype=F32)
    torch.cuda.synchronize()
    q, s = R.row_codes(R.smoothed(x, inv), fp8)
    want, err = R.product(q, s, w.float(), sw, fp8, bias)
    R.check(y, *R.finish(want, err, BF), "bf16")
    R.check(f, *R.finish(want, err, F32), "fp32")
    if not fp8:
        assert torch.equal(f, yc)  # the codes and the sums are the same, exactly
    R.check(yc, *R.finish(want, err, F32), "from codes")


@pytest.mark.parametrize("T,K,N", [(1, 256, 70), (4, 100, 33), (20, 300, 130), (64, 128, 48),
                                   (70, 256, 100), (70, 2500, 100), (300, 512, 257), (4100, 128, 4200)])
def test_linear_gate_add_strides(lib, T, K, N):
    """Row gate, add (also in place), strided x, add and out at odd offsets;
    what lies beside and behind the output's rows stays as it was."""
    say("[linear strides]", T, K, N)
    seed = seed_of(T, K, N)
    xb = tokens(T, K + 11, seed).cuda()
    x = xb[:, 5:5 + K]
    w, sw = weight(N, K, False, seed)
    lin = lib.W8A8Linear(K, N)
    lin.load_quantized(w.cuda(), sw.cuda())
    gate = vec(T, seed, -1, 1)
    add = tokens(T, N + 3, seed + 1)
    q, s = R.row_codes(x.cpu().float(), False)
    y, err = R.product(q, s, w.float(), sw, False)
    for dtype in (BF, F32):
        buf = torch.full((T + 2, N + 9), 7.0, dtype=dtype, device="cuda")
        out = buf[1:T + 1, 3:3 + N]
        lin(x, add=add.cuda()[:, 2:2 + N], gate=gate.cuda(), out=out)
        torch.cuda.synchronize()
        R.check(out, *R.finish(y, err, dtype, gate, add[:, 2:2 + N]), str(dtype))
        rest = buf.clone()
        rest[1:T + 1, 3:3 + N] = 7.0
        assert bool((rest == 7.0).all())
    both = add.cuda()
    out = both[:, 1:1 + N]
    lin(x, add=out, gate=gate.cuda(), out=out)
    R.check(out, *R.finish(y, err, BF, gate, add[:, 1:1 + N]), "in place")
    assert torch.equal(both[:, 0].cpu(), add[:, 0]) and torch.equal(both[:, N + 1:].cpu(),
                                                                   add[:, N + 1:])


@pytest.mark.parametrize("T", [3, 40, 200])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_rows_not_finite(lib, T, fp8):
    """A token with a NaN or an infinity gives a NaN row and touches no other."""
    K, N = 200, 90
    x = tokens(T, K, T)
    w, sw = weight(N, K, fp8, T)
    lin = lib.W8A8Linear(K, N, fp8=fp8)
    lin.load_quantized(w.cuda(), sw.cuda())
    bad = x.clone()
    bad[1, 7] = float("nan")
    bad[T - 1, 0] = float("inf")
    a, b = lin(x.cuda()), lin(bad.cuda())
    rows = torch.ones(T, dtype=torch.bool)
    rows[1] = rows[T - 1] = False
    assert torch.equal(a[rows.cuda()], b[rows.cuda()])
    assert bool(torch.isnan(b[1]).all()) and bool(torch.isnan(b[T - 1]).all())


@pytest.mark.parametrize("T", [1, 30, 64, 65, 400])
def test_linear_extreme_codes(lib, T):
    """All codes +-127 at the widest K: the INT32 sums reach 127^2 * 65536 and
    are exact."""
    K, N = 65536, 20
    g = torch.Generator().manual_seed(T)
    sign = torch.randint(0, 2, (N, K), generator=g) * 2 - 1
    sign[0] = 1
    q = torch.full((T, K), 127, dtype=torch.int8)
    q[T // 2, ::2] = -127
    lin = lib.W8A8Linear(K, N)
    lin.load_quantized((127 * sign).to(torch.int8).cuda(), torch.ones(N).cuda())
    y = lin(codes=(q.cuda(), torch.ones(T).cuda()), out_dtype=F32)
    want = (q.double() @ (127 * sign).double().t())
    assert torch.equal(y.cpu(), want.float())


def test_linear_offsets_past_32_bits(lib):
    """Input and output rows whose element offsets pass 2^31 (and byte offsets
    2^32)."""
    T, K, N = 34000, 128, 66000
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 20 GB")
    w, sw = weight(N, K, False, 9)
    lin = lib.W8A8Linear(K, N)
    lin.load_quantized(w.cuda(), sw.cuda())
    buf = torch.empty(T, 65536, dtype=BF, device="cuda")
    x = buf[:, 65536 - K:]
    x.copy_(tokens(T, K, 10).cuda())
    y = lin(x)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 16383, 16384, 32767, 32768, T - 2, T - 1])
    q, s = R.row_codes(x[pick.cuda()].cpu().float(), False)
    R.check(y[pick.cuda()], *R.finish(*R.product(q, s, w.float(), sw, False), BF), "far rows")


# ---------------------------------------------------------------------- ffn
FFN = [(1, 64, 32), (1, 1, 1), (1, 4096, 512), (2, 300, 77), (4, 130, 33), (4, 8192, 100),
       (5, 128, 64), (16, 256, 100), (17, 512, 31), (33, 200, 130), (64, 1000, 96), (65, 128, 64),
       (100, 300, 257), (256, 512, 500), (700, 256, 1000), (2100, 128, 2100),
       (40, 5000, 70), (70, 2500, 100), (66, 2500, 1000), (2, 64, 33000), (3, 100, 1300)]


def ffn_weights(H, F, N, fp8, seed, small=False):
    g = torch.Generator().manual_seed(seed + 3)
    if small:  # FP8 codes that are whole numbers up to 16: no sum loses a bit
        qg = torch.randint(-8, 9, (2 * F, H), generator=g).float() * 2
        qg = torch.where(qg.abs() > 8, qg, qg / 2)
        sg = (0.3 + torch.rand(2 * F, generator=g)) / (8 * H ** 0.5)
        qd, sd = R.row_codes(torch.randn(N, F, generator=g), fp8)
        return qg, sg, qd, sd / F ** 0.5
    (qg, sg), (qd, sd) = weight(2 * F, H, fp8, seed), weight(N, F, fp8, seed + 1)
    return qg.float(), sg, qd.float(), sd


def ffn_reference(q, s, qg, sg, qd, sd, fp8, exact_up=False):
    F = qd.shape[1]
    gu, e = R.product(q, s, qg, sg, fp8 and not exact_up)
    h, herr = R.hidden(gu[:, :F], gu[:, F:], e[:, :F], e[:, F:])
    qh, sh, flip, rel = R.requantised(h, herr, fp8)
    y, err = R.product(qh, sh, qd, sd, fp8)
    scale = sh[:, None] * sd.double()[None, :]
    return y, err + (flip @ qd.double().abs().t()) * scale + y.abs() * rel[:, None]


@pytest.mark.parametrize("T,H,F", FFN)
def test_ffn_int8(lib, T, H, F):
    """Within the roundings, and what the codes of h may differ by where h is
    within its own error of a rounding midpoint."""
    say("[ffn int8]", T, H, F)
    seed = seed_of(T, H, F)
    N = H if seed % 2 else H + 3
    x, inv = tokens(T, H, seed), vec(H, seed)
    qg, sg, qd, sd = ffn_weights(H, F, N, False, seed)
    ffn = lib.W8A8FFN(H, F, out_features=N)
    bias = vec(N, seed, -1, 1)
    ffn.load_quantized(qg.to(torch.int8).cuda(), sg.cuda(), qd.to(torch.int8).cuda(), sd.cuda(),
                       inv_smooth=inv.cuda(), bias=bias.cuda())
    gate, add = vec(T, seed, -1, 1), tokens(T, N, seed + 9)
    out = ffn(x.cuda(), add=add.cuda(), gate=gate.cuda())
    f = ffn(codes=lib.act_quant(x.cuda(), inv.cuda()), out_dtype=F32)
    q, s = R.row_codes(R.smoothed(x, inv), False)
    y, err = ffn_reference(q, s, qg, sg, qd, sd, False)
    y = y + bias.double()
    err = err + R.U * y.abs()
    R.check(out, *R.finish(y, err, BF, gate, add), "gated and added")
    R.check(f, *R.finish(y, err, F32), "fp32 from codes")


@pytest.mark.parametrize("T,H,F", FFN)
def test_ffn_fp8(lib, T, H, F):
    """Gate and up codes are small whole numbers, so that their sums are exact
    and h carries fp32 roundings only; the down product has the FP8 sums' bound."""
    say("[ffn fp8]", T, H, F)
    seed = seed_of(T, H, F)
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-16, 17, (T, H), generator=g).float()
    x[:, H // 2] = 448  # the row maximum: the codes are the values themselves
    x = x.to(BF)
    qg, sg, qd, sd = ffn_weights(H, F, H, True, seed, small=True)
    qg[:, H // 2] = 0
    ffn = lib.W8A8FFN(H, F, fp8=True)
    ffn.load_quantized(qg.to(E4).cuda(), sg.cuda(), qd.to(E4).cuda(), sd.cuda())
    out = ffn(x.cuda())
    q, s = R.row_codes(x.float(), True)
    assert torch.equal(q, x.float()) and bool((s == 1).all())
    y, err = ffn_reference(q, s, qg, sg, qd, sd, True, exact_up=True)
    R.check(out, *R.finish(y, err, BF), "fp8")


@pytest.mark.parametrize("T", [2, 40, 300])
def test_ffn_rows_not_finite(lib, T):
    H, F = 256, 200
    qg, sg, qd, sd = ffn_weights(H, F, H, False, T)
    ffn = lib.W8A8FFN(H, F)
    ffn.load_quantized(qg.to(torch.int8).cuda(), sg.cuda(), qd.to(torch.int8).cuda(), sd.cuda())
    x = tokens(T, H, T)
    bad = x.clone()
    bad[T - 1, 3] = float("inf")
    a, b = ffn(x.cuda()), ffn(bad.cuda())
    assert torch.equal(a[:T - 1], b[:T - 1]) and bool(torch.isnan(b[T - 1]).all())


# ----------------------------------------------------------------- add_norm
def norm64(v, e, kind, w, b, eps):
    """(norm, bound): v with absolute error e. The mean and mean square are sums
    of H terms by threads, lanes and wavefronts (a chain of at most 64 + 6 + 16
    additions of relative error u each, 90 u); a value's own error moves the
    result by e / sigma and the statistics by at most rms(e) / sigma."""
    if kind == "none":
        return v, e
    H = v.shape[1]
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        em = e.mean(1, keepdim=True) + 92 * R.U * v.abs().mean(1, keepdim=True)
        v = v - mean
        e = e + em + R.U * v.abs()
    ms = v.square().mean(1, keepdim=True) + eps
    sig = ms.sqrt()
    ems = 2 * (e * v.abs()).mean(1, keepdim=True) + e.square().mean(1, keepdim=True)
    rel = 0.5 * (ems / ms + 94 * R.U) + 3 * R.U
    n = v / sig
    e = (e / sig + n.abs() * (rel + R.U)) * (1 + 1e-3)
    if w is not None:
        n, e = n * w.double(), e * w.double().abs()
        e = e + R.U * n.abs()
    if b is not None:
        n = n + b.double()
        e = e + R.U * n.abs()
    return n, e


def add_norm64(y, res, c):
    b, e = norm64(y.double(), torch.zeros_like(y, dtype=torch.double), c["post"], c.get("pw"),
                  c.get("pb"), c["eps"])
    g = c.get("gate")
    if g is not None:
        g = g.double()
        if g.dim() == 1:
            g = g[:, None]
        elif g.shape[0] != y.shape[0]:
            g = g.repeat_interleave(c["group"], 0)[: y.shape[0]]
        b, e = b * g, e * g.abs()
    b, e = b * c["bs"], e * abs(c["bs"])
    e = e + 3 * R.U * b.abs()
    r = b if res is None else b + c["rs"] * res.double()
    e = e + R.U * r.abs()
    n, en = norm64(r, e, c["norm"], c.get("w"), c.get("b"), c["eps"])
    return r, e, n, en


NORM = [(1, 1), (1, 4096), (2, 127), (3, 8), (5, 513), (4, 1000), (7, 2047), (3, 2048), (2, 4099),
        (2, 8192), (3, 12000), (1, 16384), (2, 20001), (1, 40000), (1, 65536)]


@pytest.mark.parametrize("kind,post", [("rms", "none"), ("layer", "rms"), ("rms", "layer"),
                                       ("none", "rms")])
@pytest.mark.parametrize("T,H", NORM)
def test_add_norm(lib, T, H, kind, post):
    say("[add_norm]", T, H, kind, post)
    seed = seed_of(T, H, len(kind), len(post))
    rd = F32 if seed % 2 else BF
    y = tokens(T, H, seed)
    res = None if seed % 5 == 0 else (tokens(T, H, seed + 1).float() * 0.3).to(rd)
    c = dict(norm=kind, post=post, eps=1e-5, bs=1.25, rs=0.75)
    if kind != "none":
        c["w"] = vec(H, seed)
        c["b"] = vec(H, seed + 1, -1, 1) if seed % 3 else None
    if post != "none":
        c["pw"] = vec(H, seed + 2)
        c["pb"] = vec(H, seed + 3, -1, 1) if seed % 7 % 2 else None
    if seed % 4 == 1:
        c["gate"] = vec(T, seed, -1, 1)
    elif seed % 4 == 2:
        c["gate"], c["group"] = tokens(1, H, seed + 4), T
    elif seed % 4 == 3:
        c["gate"], c["group"] = tokens(-(-T // 2), H, seed + 4), 2
    inv = vec(H, seed + 6) if seed % 2 else None
    outs = {}
    for fmt in ("int8", "fp8"):
        o = lib.add_norm(y.cuda(), cu(res), norm=kind, weight=cu(c.get("w")), bias=cu(c.get("b")),
                         eps=1e-5, post_norm=post, post_weight=cu(c.get("pw")),
                         post_bias=cu(c.get("pb")), gate=cu(c.get("gate")),
                         gate_group=c.get("group"), residual_scale=0.75, block_scale=1.25,
                         codes=fmt, inv_smooth=cu(inv))
        outs[fmt] = o
        r, e, n, en = add_norm64(y, res, c)
        dt = BF if res is None else rd
        assert o.residual.dtype == dt
        R.check(o.residual, r, e * (1 + 4 * R.U) + R.half_step(dt) * (r.abs() + e) + 1e-44, "r")
        R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, "n")
        # codes: those of n, within what its error can move them by
        v = n if inv is None else n * inv.double()
        ev = en if inv is None else en * inv.double() + R.U * v.abs()
        fp8 = fmt == "fp8"
        q, s, flip, rel = R.requantised(v, ev, fp8)
        got = o.codes.cpu().float().double()
        assert not got[:, H:].any()
        assert bool(((got[:, :H] - q).abs() <= flip + 1e-9).all()), fmt
        assert bool(((o.scales.cpu().double() - s).abs() <= s * rel + 1e-44).all())
    assert torch.equal(outs["int8"].normed, outs["fp8"].normed)


def test_rounding_to_bf16(lib):
    """Every bf16 value passes add_norm without a norm unchanged, and fp32
    residuals round to nearest, ties to even, subnormals and overflow included."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.uint16)
    allv = torch.from_numpy(bits.numpy().copy().view("int16")).view(BF).reshape(256, 256)
    o = lib.add_norm(allv.cuda(), None, norm="none")
    for got in (o.residual.cpu(), o.normed.cpu()):
        nan = torch.isnan(allv)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got.view(torch.int16)[~nan], allv.view(torch.int16)[~nan])
    g = torch.Generator().manual_seed(3)
    raw = torch.randint(-(1 << 31), 1 << 31, (64, 1000), generator=g).to(torch.int32)
    raw[:, ::3] = (raw[:, ::3] & -65536) | 0x8000                 # exact ties
    f = raw.view(F32)
    zero = torch.zeros(64, 1000, dtype=BF)
    o = lib.add_norm(zero.cuda(), f.cuda(), norm="none")
    keep = ~torch.isnan(f)
    assert torch.equal(o.normed.cpu()[keep], f.to(BF)[keep])
    assert torch.equal(o.residual.cpu()[keep], f[keep])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_of_the_largest_values(lib, kind):
    """Rows whose squares pass the fp32 range still normalise; rows beside them
    are what they are without them."""
    T, H = 5, 900
    y = tokens(T, H, 4).float()
    y[1] *= 2.0 ** 100
    y[3] = y[3].sign() * 2.0 ** 126
    y = y.to(BF)
    w = vec(H, 1)
    o = lib.add_norm(y.cuda(), None, norm=kind, weight=w.cuda(), codes="int8")
    c = dict(norm=kind, post="none", eps=1e-6, bs=1.0, rs=1.0, w=w)
    _, _, n, en = add_norm64(y, None, c)
    R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, kind)
    assert bool(torch.isfinite(o.scales).all())


def test_many_rows(lib):
    """More rows than 2^16, each right: the first, the last and some between."""
    T, H = 200003, 72
    y = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(BF)
    w = vec(H, 2)
    o = lib.add_norm(y.cuda(), y.cuda(), weight=w.cuda(), codes="int8")
    pick = torch.tensor([0, 1, 65535, 65536, 131071, T - 2, T - 1])
    c = dict(norm="rms", post="none", eps=1e-6, bs=1.0, rs=1.0, w=w)
    _, _, n, en = add_norm64(y[pick], y[pick], c)
    R.check(o.normed[pick.cuda()], n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, "n")
    q, s = lib.act_quant(y.cuda())
    want, ws = R.row_codes(y.float(), False)
    assert torch.equal(q.cpu().float()[:, :H], want) and torch.equal(s.cpu(), ws)


def test_add_norm_in_place_and_parts(lib):
    """residual_out over residual and normed over y; outputs not asked for are
    not made; strided rows leave their neighbours alone."""
    T, H = 9, 700
    y, res = tokens(T, H, 1).cuda(), tokens(T, H, 2).cuda()
    w = vec(H, 3).cuda()
    ref = lib.add_norm(y, res, weight=w, codes="int8")
    y2, r2 = y.clone(), res.clone()
    o = lib.add_norm(y2, r2, weight=w, residual_out=r2, normed=y2)
    assert o.residual is r2 and o.normed is y2 and o.codes is None and o.scales is None
    assert torch.equal(r2, ref.residual) and torch.equal(y2, ref.normed)
    o = lib.add_norm(y, res, weight=w, residual_out=False, normed=False, codes="int8")
    assert o.residual is None and o.normed is None
    assert torch.equal(o.codes, ref.codes) and torch.equal(o.scales, ref.scales)
    o = lib.add_norm(y, res, normed=False)
    assert torch.equal(o.residual, ref.residual)
    buf = torch.full((T, H + 13), 5.0, dtype=BF, device="cuda")
    yb = torch.full((T, H + 1), 5.0, dtype=BF, device="cuda")
    yb[:, 1:] = y
    lib.add_norm(yb[:, 1:], res, weight=w, residual_out=False, normed=buf[:, 7:7 + H])
    assert torch.equal(buf[:, 7:7 + H], ref.normed)
    assert bool((buf[:, :7] == 5).all()) and bool((buf[:, 7 + H:] == 5).all())


def test_add_norm_rows_not_finite(lib):
    T, H = 6, 300
    y, res = tokens(T, H, 1), tokens(T, H, 2)
    bad = y.clone()
    bad[2, 9] = float("nan")
    bad[4, 299] = float("inf")
    w = vec(H, 3).cuda()
    for kind in ("rms", "layer"):
        a = lib.add_norm(y.cuda(), res.cuda(), norm=kind, weight=w, codes="int8")
        b = lib.add_norm(bad.cuda(), res.cuda(), norm=kind, weight=w, codes="int8")
        keep = torch.tensor([0, 1, 3, 5]).cuda()
        assert torch.equal(a.normed[keep], b.normed[keep])
        assert torch.equal(a.codes[keep], b.codes[keep])
        assert torch.equal(a.scales[keep], b.scales[keep])
        gone = torch.tensor([2, 4]).cuda()
        assert bool(torch.isnan(b.scales[gone]).all()) and not b.codes[gone].any()


# ---------------------------------------------------- as they are used together
def block(lib, seed, H, F, V, fp8):
    """A decoder block's parts: QKV-like projection, FFN, head."""
    q, p = lib.W8A8Linear(H, H + 64, fp8=fp8), lib.W8A8Linear(H + 64, H, fp8=fp8)
    f, head = lib.W8A8FFN(H, F, fp8=fp8), lib.W8A8Linear(H, V, fp8=fp8)
    g = torch.Generator().manual_seed(seed)
    mk = lambda n, k: (torch.randn(n, k, generator=g) / k ** 0.5).cuda()  # noqa: E731
    sm = vec(H, seed).cuda()
    q.quantise(mk(H + 64, H), smooth=sm)
    p.quantise(mk(H, H + 64))
    f.quantise(mk(2 * F, H), mk(H, F), smooth=sm)
    head.quantise(mk(V, H))
    w = [vec(H, seed + i).cuda() for i in range(3)]
    inv = 1.0 / sm
    fmt = "fp8" if fp8 else "int8"

    def run(x, gate):
        a = lib.add_norm(x, None, weight=w[0], codes=fmt, inv_smooth=inv, normed=False)
        y = p(q(codes=(a.codes, a.scales)))
        b = lib.add_norm(y, a.residual, weight=w[1], codes=fmt, inv_smooth=inv)
        y = f(codes=(b.codes, b.scales), add=b.normed, gate=gate)
        c = lib.add_norm(y, b.residual, weight=w[2], post_weight=w[0], codes=fmt, normed=False)
        return c.residual, head(codes=(c.codes, c.scales), out_dtype=F32)
    return run


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 7, 130])
def test_block_runs_in_graphs_and_streams(lib, T, fp8):
    """The operators in a row: eager, on two other streams at once, and in two
    captured graphs replayed with new inputs and eager work in between, all
    with the same results."""
    H, F, V = 320, 200, 333
    run = block(lib, 5, H, F, V, fp8)
    xs = [tokens(T, H, i).cuda() for i in range(4)]
    gates = [vec(T, i).cuda() for i in range(4)]
    eager = [run(x, g) for x, g in zip(xs, gates)]
    torch.cuda.synchronize()
    again = [run(x, g) for x, g in zip(xs, gates)]
    for a, b in zip(eager, again):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None] * 4
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got[i] = run(xs[i], gates[i])
    torch.cuda.synchronize()
    for a, b in zip(eager, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    graphs = []
    for _ in range(2):
        x, g = xs[0].clone(), gates[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(x, g)
        graphs.append((graph, x, g, out))
    for i in range(4):
        for k, (graph, x, g, out) in enumerate(graphs):
            x.copy_(xs[(i + k) % 4])
            g.copy_(gates[(i + k) % 4])
            graph.replay()
        run(xs[0], gates[0])
        torch.cuda.synchronize()
        for k, (graph, x, g, out) in enumerate(graphs):
            assert all(torch.equal(u, v) for u, v in zip(eager[(i + k) % 4], out)), (i, k)


def test_reloaded_weights_in_a_captured_call(lib):
    """A captured call follows what is loaded into its operator later: codes,
    scales, smoothing and bias keep their places."""
    T, K, N = 3, 200, 60
    x = tokens(T, K, 1).cuda()
    lin = lib.W8A8Linear(K, N)
    sets = [weight(N, K, False, s) + (vec(K, s), vec(N, s)) for s in (1, 2)]
    load = lambda s: lin.load_quantized(s[0].cuda(), s[1].cuda(), inv_smooth=s[2].cuda(),  # noqa: E731
                                        bias=s[3].cuda())
    want = []
    for s in sets:
        load(s)
        want.append(lin(x).clone())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = lin(x)
    for k in (0, 1, 0):
        load(sets[k])
        torch.cuda.empty_cache()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])


def test_shared_expert_beside_the_layer(lib):
    """The FFN added onto the routed experts' output equals the two computed
    apart; its own part equals the layer with that one expert, up to what the
    two paths' roundings allow (codes of h within one step on few entries)."""
    H, F, T = 256, 128, 24
    g = torch.Generator().manual_seed(1)
    wg, wu = torch.randn(1, F, H, generator=g) / 16, torch.randn(1, F, H, generator=g) / 16
    wd = torch.randn(1, H, F, generator=g) / 12
    moe = lib.MoEW8A8(H, F, 1, 1)
    x = tokens(T, H, 2).cuda()
    moe.calibrate(x, wg.cuda(), wu.cuda(), wd.cuda(), 0.5)
    ids = torch.zeros(T, 1, dtype=torch.int32).cuda()
    ones = torch.ones(T, 1).cuda()
    routed = moe.forward(x, topk_ids=ids, topk_w=ones)
    ffn = lib.W8A8FFN(H, F)
    ffn.quantise(torch.cat([wg[0], wu[0]]).cuda(), wd[0].cuda(), smooth=moe.smooth)
    alone = ffn(x, out_dtype=F32)
    rms = float(alone.double().square().mean().sqrt())
    diff = (alone.double() - routed.double()).abs()
    assert float((diff - R.half_step(BF) * alone.double().abs()).max()) <= 2e-2 * rms
    gate = vec(T, 4).cuda()
    both = ffn(x, add=routed, gate=gate)
    want = gate.double()[:, None] * alone.double() + routed.double()
    bound = (R.half_step(BF) + 4 * R.U) * (want.abs() + 2 * alone.double().abs())
    assert bool(((both.double() - want).abs() <= bound).all())


def test_empty_batches(lib):
    lin, ffn = lib.W8A8Linear(70, 30), lib.W8A8FFN(64, 32)
    lin.quantise(torch.randn(30, 70).cuda())
    ffn.quantise(torch.randn(64, 64).cuda(), torch.randn(64, 32).cuda())
    x = torch.empty(0, 70, dtype=BF, device="cuda")
    assert lin(x).shape == (0, 30)
    q, s = lib.act_quant(x)
    assert q.shape == (0, 128) and s.shape == (0,)
    assert lin(codes=(q, s)).shape == (0, 30)
    assert ffn(torch.empty(0, 64, dtype=BF, device="cuda")).shape == (0, 64)
    o = lib.add_norm(x, x, codes="fp8")
    assert o.normed.shape == (0, 70) and o.codes.shape == (0, 128)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [72, 900, 5000])
def test_norm_of_the_smallest_values(lib, kind, H):
    """Without an eps (or with one as small) a row whose squares fall below the
    fp32 range normalises as any other; a row of zeros has no norm (0 / 0)."""
    y = tokens(9, H, 5).float()
    for t, p in ((1, -40), (2, -50), (3, -64), (4, -75), (5, -100), (6, -120)):
        y[t] *= 2.0 ** p
    y[7] = 0
    y[7, 3] = 2.0 ** -133
    y[8] = 0
    y = y.to(BF)
    for eps in (0.0, 2.0 ** -120):
        o = lib.add_norm(y.cuda(), None, norm=kind, eps=eps, codes="int8")
        c = dict(norm=kind, post="none", eps=eps, bs=1.0, rs=1.0)
        _, _, n, en = add_norm64(y[:8], None, c)
        R.check(o.normed[:8], n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, kind)
        assert bool(torch.isfinite(o.scales[:8]).all())
        last = o.normed[8]
        assert bool(torch.isnan(last).all()) if eps == 0.0 else not bool(last.any())


def test_refused_weights_change_nothing(lib):
    """A load that is refused for its last operand leaves what was loaded."""
    H, F, N, T = 72, 40, 30, 3
    x = tokens(T, H, 1).cuda()
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    lin = lib.W8A8Linear(H, N)
    lin.quantise(r(N, H), vec(H, 1).cuda(), vec(N, 2).cuda())
    ffn = lib.W8A8FFN(H, F, out_features=N)
    ffn.quantise(r(2 * F, H), r(N, F), vec(H, 1).cuda(), vec(N, 2).cuda())
    want = lin(x), ffn(x)
    i8 = lambda *s: torch.ones(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    for call in (lambda: lin.quantise(r(N, H) * 2, bias=one(N + 1)),
                 lambda: lin.quantise(r(N, H) * 2, smooth=one(H + 1)),
                 lambda: lin.load_quantized(i8(N, H), one(N), bias=one(N + 1)),
                 lambda: lin.load_quantized(i8(N, H), one(N), inv_smooth=one(H).double()),
                 lambda: lin.load_quantized(i8(N, H), None),
                 lambda: ffn.quantise(r(2 * F, H) * 2, r(N, F + 1)),
                 lambda: ffn.quantise(r(2 * F, H) * 2, r(N, F), bias=one(N + 1)),
                 lambda: ffn.load_quantized(i8(2 * F, H), one(2 * F), i8(N, F), one(N + 1)),
                 lambda: ffn.load_quantized(i8(2 * F, H), one(2 * F), i8(N, F), None),
                 lambda: ffn.load_quantized(i8(2 * F, H), one(2 * F), i8(N, F), one(N),
                                            bias=one(N + 1))):
        with pytest.raises(lib.MoEW8A8Error):
            call()
        assert torch.equal(lin(x), want[0]) and torch.equal(ffn(x), want[1])


@pytest.mark.parametrize("H", list(range(1, 17)) + [509, 510, 2043, 2045])
def test_row_ends(lib, H):
    """Every remainder of eight, rows narrower than eight included: the values
    are those of the same rows inside a wider matrix, NaN beside them is not
    read, and what lies beside the outputs is left as it was."""
    T, wide = 5, H + 9
    pad = torch.full((T, wide), float("nan"))
    for rd in (BF, F32):
        y, res = pad.to(BF).cuda(), pad.to(rd).cuda()
        y[:, 4:4 + H] = tokens(T, H, H).cuda()
        res[:, 4:4 + H] = tokens(T, H, H + 1).to(rd).cuda()
        w, b = vec(H, H).cuda(), vec(H, H + 1, -1, 1).cuda()
        out, nrm = torch.full_like(res, 7), torch.full_like(y, 7)
        o = lib.add_norm(y[:, 4:4 + H], res[:, 4:4 + H], weight=w, bias=b, codes="int8",
                         inv_smooth=w, residual_out=out[:, 4:4 + H], normed=nrm[:, 4:4 + H])
        c = dict(norm="rms", post="none", eps=1e-6, bs=1.0, rs=1.0, w=w.cpu(), b=b.cpu())
        r, e, n, en = add_norm64(y[:, 4:4 + H].cpu(), res[:, 4:4 + H].cpu(), c)
        R.check(o.residual, r, e * (1 + 4 * R.U) + R.half_step(rd) * (r.abs() + e) + 1e-44, "r")
        R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, "n")
        for t in (out, nrm):
            assert bool((t[:, :4] == 7).all()) and bool((t[:, 4 + H:] == 7).all())
        assert bool(torch.isfinite(o.scales).all()) and not bool(o.codes[:, H:].any())
    q, s = lib.act_quant(y[:, 4:4 + H], w)
    want, ws = R.row_codes(R.smoothed(y[:, 4:4 + H].cpu(), w.cpu()), False)
    assert torch.equal(q.cpu().float()[:, :H], want) and torch.equal(s.cpu(), ws)


@pytest.mark.parametrize("N", list(range(1, 17)) + [131])
@pytest.mark.parametrize("T", [3, 70])
def test_output_row_ends(lib, T, N):
    """The same of a product's outputs and of what is added to them, in the
    streaming and in the tiled kernel: with INT8 the fp32 result of exact sums,
    then one rounding each."""
    K = 130
    qw = torch.randint(-127, 128, (N, K), generator=torch.Generator().manual_seed(N)).to(torch.int8)
    sw, x = vec(N, N) / 100, tokens(T, K, N)
    lin = lib.W8A8Linear(K, N)
    lin.load_quantized(qw.cuda(), sw.cuda())
    q, s = R.row_codes(x.float(), False)
    y = (q.double() @ qw.double().t()) * s.double()[:, None] * sw.double()
    add = torch.full((T, N + 9), float("nan")).to(BF)
    add[:, 4:4 + N] = tokens(T, N, N + 1)
    a = add[:, 4:4 + N].double()
    for dt in (F32, BF):
        out = torch.full((T, N + 9), 7.0, dtype=dt).cuda()
        lin(x.cuda(), add=add.cuda()[:, 4:4 + N], out=out[:, 4:4 + N])
        v = y + a
        # sum to fp32, two products, one sum: four roundings
        bound = 4 * R.U * (y.abs() + a.abs()) * (1 + 1e-3)
        R.check(out[:, 4:4 + N], v, bound + R.half_step(dt) * (v.abs() + bound) + 1e-44, "out")
        assert bool((out[:, :4] == 7).all()) and bool((out[:, 4 + N:] == 7).all())


# Each tile shape of the tiled product, with ragged last tiles both ways: 256 x 256,
# 256 x 192, 128 x 256, 128 x 192, 128 x 128, 64 x 128 (one and two blocks a unit).
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K,N", [(2990, 200, 4090), (1999, 130, 6130), (990, 300, 8187),
                                   (1021, 200, 6001), (500, 400, 6099), (250, 300, 6143),
                                   (251, 1, 11007), (130, 130, 32003)])
def test_linear_tiles(lib, T, K, N, fp8):
    test_linear(lib, T, K, N, fp8)


@pytest.mark.parametrize("T,H,F", [(500, 200, 3007), (990, 130, 4091), (120, 300, 8200)])
def test_ffn_tiles(lib, T, H, F):
    test_ffn_int8(lib, T, H, F)
    test_ffn_fp8(lib, T, H, F)
