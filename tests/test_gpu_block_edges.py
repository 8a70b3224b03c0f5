"""The block operators on the GPU where a shape, a value or a call is out of the
ordinary: FP8 sums that no truncation may touch, every streaming kernel, norms at
the ends of the fp32 range at every width, reloads under a captured call."""
import pytest
import torch

import block_ref as R
from test_gpu_block_ops import (BF, E4, F32, add_norm64, cu, lib, say,  # noqa: F401
                                seed_of, test_linear, tokens, vec, weight)

pytestmark = pytest.mark.gpu
linear_case = test_linear
del test_linear  # (its own cases run where it stands)


# ----------------------------------------------------------------- FP8 sums
def wide_codes(rows, K, seed, most=16):
    """Whole numbers up to 8 in size, 448 in a few columns (the same for every
    matrix of this K): the products reach 448^2 = 200704 beside single units, so
    that sums which keep 13 bits below a group's largest product lose some, while
    every partial sum stays below 2^24 and is exact in fp32 in any order."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-8, 9, (rows, K), generator=g).float()
    big = torch.arange(0, K, max(8, -(-K // most)))
    q[:, big] = 448.0 * (torch.randint(0, 2, (rows, big.numel()), generator=g) * 2 - 1).float()
    assert big.numel() * 448 ** 2 + 64 * K < 1 << 24
    return q


# Streaming and tiled kernels: one token to several tiles, K in one piece and split.
WIDE = [(1, 4096, 100), (3, 300, 40), (16, 2048, 33), (32, 1000, 8200), (33, 512, 70),
        (64, 4096, 130), (65, 128, 64), (70, 2500, 100), (100, 8192, 300), (200, 1024, 2000),
        (256, 4096, 700), (300, 640, 5000), (1000, 512, 4100), (1400, 256, 6144), (3000, 384, 4090)]


@pytest.mark.parametrize("T,K,N", WIDE)
def test_fp8_sums_kept_in_fp32(lib, T, K, N):
    """FP8 products with an fp32 result, and bf16 ones of up to 32 tokens, add
    whole products: sums that are exact in fp32 come out exactly."""
    say("[fp8 sums]", T, K, N)
    q, w = wide_codes(T, K, seed_of(T, K)), wide_codes(N, K, seed_of(N, K) + 1)
    ops = lib.W8A8Linear(K, N, fp8=True)
    ops.load_quantized(w.to(E4).cuda(), torch.ones(N).cuda())
    codes = torch.nn.functional.pad(q, (0, R.pitch(K) - K)).to(E4).cuda()
    want = q.double() @ w.double().t()
    assert float(want.abs().max()) < 1 << 24
    y = ops(codes=(codes, torch.ones(T).cuda()), out_dtype=F32)
    assert torch.equal(y.cpu().double(), want)
    y = ops(codes=(codes, torch.ones(T).cuda()))
    if T <= 32:
        assert torch.equal(y.cpu(), want.to(BF))
    else:
        R.check(y, want, R.fp8_sum_bound(q, w) + R.half_step(BF) * want.abs() * (1 + 1e-3), "bf16")


@pytest.mark.parametrize("T,K,N", [(1, 4096, 4096), (1, 8192, 100), (4, 4096, 300), (2, 8192, 48),
                                   (1, 4100, 8000), (1, 4096, 16500), (3, 1000, 20000),
                                   (4, 300, 70), (4, 8192, 70), (5, 4096, 9000), (16, 4096, 300),
                                   (32, 4096, 9000), (40, 4096, 5000), (64, 4200, 500),
                                   (70, 2000, 300), (300, 512, 1000)])
def test_fp8_sums_from_tokens_and_from_codes(lib, T, K, N):
    """The order of a sum depends on the sizes only: a product of tokens and one of
    their codes give the same bits, FP8 included, and so do feed-forward blocks."""
    say("[same sums]", T, K, N)
    x, (w, sw) = tokens(T, K, seed_of(T, K)).cuda(), weight(N, K, True, seed_of(T, K, N))
    lin = lib.W8A8Linear(K, N, fp8=True)
    lin.load_quantized(w.cuda(), sw.cuda())
    codes = lib.act_quant(x, fp8=True)
    assert torch.equal(lin(x, out_dtype=F32), lin(codes=codes, out_dtype=F32))
    assert torch.equal(lin(x), lin(codes=codes))
    F = N // 2
    ffn = lib.W8A8FFN(K, F, out_features=33, fp8=True)
    wd, sd = weight(33, F, True, N)
    ffn.load_quantized(w[:2 * F].cuda(), sw[:2 * F].cuda(), wd.cuda(), sd.cuda())
    assert torch.equal(ffn(x, out_dtype=F32), ffn(codes=codes, out_dtype=F32))


@pytest.mark.parametrize("T,H,F", [(3, 256, 100), (24, 512, 2100), (64, 300, 130), (65, 128, 64),
                                   (70, 2500, 300), (100, 1024, 1000), (300, 300, 257),
                                   (700, 256, 1000), (2100, 128, 2100)])
def test_ffn_fp8_hidden_codes(lib, T, H, F):
    """The gate and up sums of an FP8 feed-forward block are exact where fp32
    holds them, at every T, so that its hidden codes are the exact ones but for
    what fp32 roundings may move; an fp32 result adds whole products as well."""
    say("[ffn fp8 hidden]", T, H, F)
    seed = seed_of(T, H, F)
    x, qg = wide_codes(T, H, seed), wide_codes(2 * F, H, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    sg = (0.5 + torch.rand(2 * F, generator=g)) / 400000
    wd, sd = weight(H, F, True, seed)
    ffn = lib.W8A8FFN(H, F, fp8=True)
    ffn.load_quantized(qg.to(E4).cuda(), sg.cuda(), wd.cuda(), sd.cuda())
    out = ffn(x.to(BF).cuda(), out_dtype=F32)
    q, s = R.row_codes(x, True)
    assert torch.equal(q, x) and bool((s == 1).all())
    gu, e = R.product(q, s, qg, sg, False)
    h, herr = R.hidden(gu[:, :F], gu[:, F:], e[:, :F], e[:, F:])
    qh, sh, flip, rel = R.requantised(h, herr, True)
    qd = wd.float()
    y, err = R.product(qh, sh, qd, sd, False)
    scale = sh[:, None] * sd.double()[None, :]
    # F additions, each within one fp32 step of a partial sum
    err = err + 2 * R.U * R.pitch(F) * (qh.abs() @ qd.double().abs().t()) * scale
    err = err + (flip @ qd.double().abs().t()) * scale + y.abs() * rel[:, None]
    R.check(out, *R.finish(y, err, F32), "ffn")


# ------------------------------------------------------- every streaming kernel
# By rows (up to 16, 32, 64), wavefronts of one panel (16, 8), panels a block (1, 2,
# 4) and source; each shape runs from tokens (coded by the kernel, or in tiles)
# and from row-major codes.
STREAM = [(1, 4096, 300), (1, 1000, 300), (1, 4096, 6000), (3, 1000, 9000), (2, 4096, 17000),
          (3, 300, 20000),                                               # rows coded by the kernel
          (4, 5000, 300), (4, 5000, 6000), (4, 5000, 9000),              # too wide for that
          (9, 4096, 3000), (9, 4096, 6000), (16, 4200, 9000), (12, 600, 17000),
          (20, 4096, 3000), (20, 4096, 6000), (32, 4200, 9000), (25, 2000, 9000), (32, 600, 17000),
          (33, 4096, 3000), (40, 4096, 6000), (64, 1000, 8190)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K,N", STREAM)
def test_streaming_kernels(lib, T, K, N, fp8):
    linear_case(lib, T, K, N, fp8)


@pytest.mark.parametrize("T,K,N", STREAM)
def test_streaming_kernels_fp8_sums(lib, T, K, N):
    test_fp8_sums_kept_in_fp32(lib, T, K, N)
    q, w = wide_codes(T, K, 5), wide_codes(N, K, 6)
    lin = lib.W8A8Linear(K, N, fp8=True)
    lin.load_quantized(w.to(E4).cuda(), torch.ones(N).cuda())
    y = lin(q.to(BF).cuda(), out_dtype=F32)  # (a row's largest is 448: its codes are itself)
    assert torch.equal(y.cpu().double(), q.double() @ w.double().t())


def ffn64(x, inv, qg, sg, qd, sd, fp8, loose_down):
    """(y, bound) of a feed-forward block in 64 bits. FP8 sums add whole products:
    K additions, each within one fp32 step of a partial sum; loose_down: those of the
    down product by the FP8 instructions instead."""
    F = qd.shape[1]
    q, s = R.row_codes(R.smoothed(x, inv), fp8)

    def product(q, s, w, sw, loose):
        y, err = R.product(q, s, w, sw, fp8 and loose)
        if fp8 and not loose:
            sums = q.double().abs() @ w.double().abs().t()
            err = err + 2 * R.U * R.pitch(w.shape[1]) * sums * (
                s.double()[:, None] * sw.double()[None, :])
        return y, err
    gu, e = product(q, s, qg, sg, False)
    h, herr = R.hidden(gu[:, :F], gu[:, F:], e[:, :F], e[:, F:])
    qh, sh, flip, rel = R.requantised(h, herr, fp8)
    y, err = product(qh, sh, qd, sd, loose_down)
    moved = (flip @ qd.double().abs().t()) * (sh[:, None] * sd.double()[None, :])
    return y, err + moved + y.abs() * rel[:, None]


# Hidden rows coded by the down product's kernel: 8 and 16 wavefronts, one, two and
# four panels; by a launch of their own, in streaming and tiled products.
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,F,N", [(1, 300, 700, 200), (1, 200, 5000, 100), (2, 128, 4000, 5000),
                                     (1, 64, 8000, 17000), (3, 100, 300, 16400), (4, 64, 90, 6000),
                                     (1, 300, 9000, 200), (7, 300, 2300, 90), (20, 256, 2300, 4200),
                                     (32, 300, 130, 9000), (40, 300, 257, 130), (70, 300, 257, 66),
                                     (300, 200, 300, 257), (700, 256, 500, 130)])
def test_ffn_streaming_kernels_and_ordinary_codes(lib, T, H, F, N, fp8):
    say("[ffn]", T, H, F, N, fp8)
    seed = seed_of(T, H, F, N)
    x, inv = tokens(T, H, seed), vec(H, seed)
    (qg, sg), (qd, sd) = weight(2 * F, H, fp8, seed), weight(N, F, fp8, seed + 1)
    ffn = lib.W8A8FFN(H, F, out_features=N, fp8=fp8)
    bias, gate, add = vec(N, seed, -1, 1), vec(T, seed, -1, 1), tokens(T, N, seed + 9)
    ffn.load_quantized(qg.cuda(), sg.cuda(), qd.cuda(), sd.cuda(), inv_smooth=inv.cuda(),
                       bias=bias.cuda())
    f = ffn(x.cuda(), out_dtype=F32)
    out = ffn(x.cuda(), add=add.cuda(), gate=gate.cuda())
    for got, loose, dt, kw in ((f, False, F32, {}), (out, T > 32, BF, dict(gate=gate, add=add))):
        y, err = ffn64(x, inv, qg.float(), sg, qd.float(), sd, fp8, loose)
        y = y + bias.double()
        err = err + R.U * y.abs()
        R.check(got, *R.finish(y, err, dt, **kw), str(dt))


# ------------------------------------------------------------------- norms
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [7, 900, 4096, 5000, 8191, 20001, 40000, 65536])
def test_norm_of_the_largest_values_at_every_width(lib, kind, H):
    """Rows of values near the largest bf16, of one sign or both, and of powers of
    two up to 2^127, normalise as any other: neither their squares nor their
    differences from the mean leave the range."""
    T = 7
    g = torch.Generator().manual_seed(H)
    sign = (torch.randint(0, 2, (T, H), generator=g) * 2 - 1).float()
    y = 3.38e38 * (1 - 0.2 * torch.rand(T, H, generator=g)) * sign
    y[1] = 2.0 ** 127 * sign[1]
    y[2] = 2.0 ** 110 * torch.randn(H, generator=g)
    y[3] = 3.38e38 * torch.where(torch.arange(H) % 10 == 0, -1.0, 1.0)  # far from its mean
    y[4] = tokens(1, H, H)[0].float()
    y[5] = y[5].abs() * torch.where(torch.arange(H) == H // 2, -1.0, 1.0)
    y[6] = 2.0 ** 64 * torch.randn(H, generator=g)
    y = y.to(BF)
    w = vec(H, 1)
    o = lib.add_norm(y.cuda(), None, norm=kind, weight=w.cuda(), codes="int8")
    c = dict(norm=kind, post="none", eps=1e-6, bs=1.0, rs=1.0, w=w)
    _, _, n, en = add_norm64(y, None, c)
    R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, kind)
    assert bool(torch.isfinite(o.scales).all()) and bool((o.scales > 0).all())
    # an fp32 residual up to the last fp32 value, and the post norm
    res = torch.full((T, H), torch.finfo(F32).max) * sign
    o = lib.add_norm(torch.zeros_like(y).cuda(), res.cuda(), norm=kind, weight=w.cuda())
    _, _, n, en = add_norm64(torch.zeros_like(y), res, c)
    R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, kind + " fp32")
    o = lib.add_norm(y.cuda(), None, norm="none", post_norm=kind, post_weight=w.cuda())
    c = dict(norm="none", post=kind, eps=1e-6, bs=1.0, rs=1.0, pw=w)
    _, _, n, en = add_norm64(y, None, c)
    R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, kind + " post")


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_with_the_largest_eps(lib, kind):
    """eps beside which a row is small, up to the last fp32 value."""
    T, H = 3, 700
    y = tokens(T, H, 1).float()
    y[1] *= 2.0 ** 60
    y[2] *= 2.0 ** 100
    y = y.to(BF)
    w = torch.full((H,), 2.0 ** 60)
    for eps in (1.0, 1e30, 2.0 ** 127, torch.finfo(F32).max):
        o = lib.add_norm(y.cuda(), None, norm=kind, weight=w.cuda(), eps=eps)
        c = dict(norm=kind, post="none", eps=eps, bs=1.0, rs=1.0, w=w)
        _, _, n, en = add_norm64(y, None, c)
        # (below the bf16 range a rounding is half of 2^-133)
        R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 2.0 ** -134, str(eps))


@pytest.mark.parametrize("H", [1, 5, 700, 2047, 4099, 20001])
def test_layer_norm_of_constant_rows(lib, H):
    """A row of one value has a layer norm of zero whatever the value. The mean's
    rounding (92 u of it, by the chains of its sum) is taken off with the mean of
    what it leaves: 92 u of 92 u |c| remain, and the rounding of that difference."""
    cs = torch.tensor([0.0, 1.0, -3.3, 1000.7, 30001.0, -123456.7, 1e-3, 7e6])
    res = cs[:, None].expand(8, H).contiguous()
    b, eps = vec(H, 3), 1e-6
    zero = torch.zeros(8, H, dtype=BF)
    for r in (res, res.to(BF)):
        o = lib.add_norm(zero.cuda(), r.cuda(), norm="layer", bias=b.cuda(), eps=eps)
        left = (93 * 92 * R.U ** 2 * cs.double().abs() / eps ** 0.5)[:, None]
        want = b.double()[None, :].expand(8, H)
        R.check(o.normed, want, left + (R.half_step(BF) + R.U) * (want + left), "constant")


# ---------------------------------------------------------------- captured calls
@pytest.mark.parametrize("T", [3, 20, 50, 90])
@pytest.mark.parametrize("fp8", [False, True])
def test_captured_calls_follow_reloads_with_and_without_vectors(lib, T, fp8):
    """A captured product or feed-forward block gives what an eager call of the
    weights loaded now gives, whichever of smoothing and bias they have; what a
    captured call went without can no longer be loaded, and the refusal changes
    nothing."""
    K, F, N = 300, 70, 60
    say("[reloads]", T, fp8)
    x = tokens(T, K, 1).cuda()

    def build():
        return lib.W8A8Linear(K, N, fp8=fp8), lib.W8A8FFN(K, F, out_features=N, fp8=fp8)

    def load(ops, s):
        w, inv, bias = s
        ops[0].load_quantized(w[0], w[1], inv_smooth=inv, bias=bias)
        ops[1].load_quantized(*w[2:], inv_smooth=inv, bias=bias)
    sets, want = [], []
    for i, (smooth, bias) in enumerate([(1, 1), (0, 0), (1, 0), (0, 1)]):
        w = [cu(t) for j, shape in enumerate([(N, K), (2 * F, K), (N, F)])
             for t in weight(*shape, fp8, 10 * i + j)]
        sets.append((w, cu(vec(K, i)) if smooth else None, cu(vec(N, i)) if bias else None))
        ops = build()
        load(ops, sets[-1])
        want.append([op(x) for op in ops])
    for first, s in enumerate(sets):
        ops = build()
        load(ops, s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [op(x) for op in ops]
        last = first
        for k in (0, 1, 2, 3, 1, 0):
            fits = all(now is None or then is not None for now, then in zip(sets[k][1:], s[1:]))
            if fits:
                load(ops, sets[k])
                last = k
            else:
                for i, op in enumerate(ops):
                    w = sets[k][0]
                    with pytest.raises(lib.MoEW8A8Error, match="captured"):
                        op.load_quantized(*(w[2:] if i else w[:2]), inv_smooth=sets[k][1],
                                          bias=sets[k][2])
            graph.replay()
            torch.cuda.synchronize()
            for op, got, right in zip(ops, out, want[last]):
                assert torch.equal(got, right) and torch.equal(op(x), right)


def test_smoothing_loaded_after_a_capture_from_codes(lib):
    """A captured call that was given codes does not use the smoothing: it may
    come later."""
    K, N = 200, 40
    lin = lib.W8A8Linear(K, N)
    w, s = weight(N, K, False, 1)
    lin.load_quantized(w.cuda(), s.cuda())
    codes = lib.act_quant(tokens(5, K, 2).cuda())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lin(codes=codes)
    w2, s2 = weight(N, K, False, 3)
    lin.load_quantized(w2.cuda(), s2.cuda(), inv_smooth=vec(K, 1).cuda())
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lin(codes=codes))
    with pytest.raises(lib.MoEW8A8Error, match="captured"):
        lin.load_quantized(w.cuda(), s.cuda(), bias=vec(N, 1).cuda())


# ------------------------------------------------- kernels that the rest passes by
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K", [(2049, 4096), (2050, 2051), (2049, 8192), (2100, 4103), (2, 33001),
                                 (1, 65533)])
def test_act_quant_many_rows(lib, T, K, fp8):
    """More than 2048 rows of 2049 to 8192 columns take two chunks a thread."""
    x, inv = tokens(T, K, seed_of(T, K)), vec(K, K)
    q, s = lib.act_quant(x.cuda(), inv.cuda(), fp8=fp8)
    want, ws = R.row_codes(R.smoothed(x, inv), fp8)
    got = q.cpu().float()
    assert torch.equal(got[:, :K], want) and torch.equal(s.cpu(), ws) and not got[:, K:].any()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", [(3, 2051), (5, 4095), (2, 32769), (1, 40001), (1, 65535)])
def test_add_norm_odd_wide_rows(lib, T, H, kind):
    y, res = tokens(T, H, H), tokens(T, H, H + 1)
    w, b = vec(H, 1), vec(H, 2, -1, 1)
    o = lib.add_norm(y.cuda(), res.cuda(), norm=kind, weight=w.cuda(), bias=b.cuda(), eps=1e-5)
    c = dict(norm=kind, post="none", eps=1e-5, bs=1.0, rs=1.0, w=w, b=b)
    r, e, n, en = add_norm64(y, res, c)
    R.check(o.residual, r, e * (1 + 4 * R.U) + R.half_step(BF) * (r.abs() + e) + 1e-44, "r")
    R.check(o.normed, n, en + R.half_step(BF) * (n.abs() + en) + 1e-44, "n")


@pytest.mark.parametrize("fp8", [False, True])
def test_small_tiles_two_a_unit(lib, fp8):
    """64 x 128 tiles, more than one a compute unit."""
    linear_case(lib, 393, 200, 8873, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_ffn_hidden_rows_of_middle_width(lib, fp8):
    test_ffn_streaming_kernels_and_ordinary_codes(lib, 20, 256, 1000, 90, fp8)
