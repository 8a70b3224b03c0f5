"""The block operators on the GPU where a shape, a value or a call is out of the
ordinary: FP8 sums that no truncation may touch, every streaming kernel, norms at
the ends of the fp32 range at every width, reloads under a captured call."""
import pytest
import torch

import block_ref as R
from test_gpu_block_ops import (BF, E4, F32, add_norm64, cu, lib, say, seed_of, tokens,  # noqa: F401
                                vec, weight)

pytestmark = pytest.mark.gpu


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
