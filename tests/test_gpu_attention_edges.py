"""Calls of qk_norm_rope and paged_attention at the edges of what their documentation
allows, on the GPU against the plain 64-bit forms of tests/attention_ref.py."""
import math

import pytest
import torch

import attention_ref as A
import block_ref as R

pytestmark = pytest.mark.gpu
BF, F32, F64 = A.BF, A.F32, A.F64


@pytest.fixture(scope="module", autouse=True)
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_int8_expert_amd as mod
    mod.load_library()
    return mod


def cu(t):
    return None if t is None else t.cuda()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def contents(step, Hkv, D, fmt, seed):
    """Cache contents on the host: k, scales, v, scales."""
    shape = (step.num_pages, Hkv, step.page, D)
    return A.cached(shape, fmt, seed) + A.cached(shape, fmt, seed + 1)


def cache_of(m, host):
    return m.KVCache.of(cu(host[0]), cu(host[2]), cu(host[1]), cu(host[3]))


def check(got, want, err, what):
    """As R.check, and infinities have to be where they are wanted, with their sign."""
    R.check(got, want, err, what)
    far = torch.isinf(want)
    assert torch.equal(got.double().cpu()[far], want[far]), what + ": infinities"


def place(step, b, p):
    """Page and row of place p of sequence b."""
    return int(step.table[b, p // step.page]), p % step.page


# ------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(2, 1), (4, 1), (6, 4), (2, 90)])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_infinite_values_that_every_row_sees(m, D, G, n, fmt):
    """Infinities and NaN among the values of keys far from a sequence's end, which all
    rows see (of codes: infinite scales, NaN codes): each reaches its own column, with its
    sign, of few rows and of many."""
    L = 340
    step = A.Step([(n, L), (1, 70)], 16, seed=3)
    host = contents(step, 1, D, fmt, 8)
    k, ks, v, vs = host
    # (keys alike: probabilities within a factor of 2^4 or so of each other)
    for p, col, x in ((5, 3, math.inf), (40, 7, -math.inf), (70, 9, math.nan), (100, 11, math.inf),
                      (131, 11, math.inf), (132, 13, math.inf), (133, 13, -math.inf), (200, 3, math.inf)):
        page, row = place(step, 0, p)
        if fmt == "bf16":
            v[page, 0, row, col] = x
        elif fmt == "fp8" and math.isnan(x):
            v.view(torch.uint8)[page, 0, row, col] = 0x7f
    if fmt != "bf16":
        page, row = place(step, 0, 260)
        vs[page, 0, row] = math.inf
        raw = v.view(torch.uint8)[page, 0, row]
        raw[torch.arange(D) % 4 == 1] = 0
    q = randn(step.T, G * D, seed=4).to(BF)
    want, err = A.attention(q, *host, step, G, D ** -0.5)
    if fmt != "int8":
        assert bool(torch.isnan(want[:n]).any())
    assert bool((want == math.inf).any()) and bool((want == -math.inf).any())
    got = m.paged_attention(cu(q), cache_of(m, host), step.batch(m))
    check(got, want, err, "attention")


# ------------------------------------------------------------------------ windows
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,lens", [(1, [(6, 2), (3, 40)]), (2, [(300, 250), (5, 1), (80, 80)])])
def test_window_past_every_place(m, fmt, causal, G, lens):
    """The widest window, with tokens of negative place (fewer keys than new tokens): as
    none at all."""
    step = A.Step(lens, 16, seed=3)
    host = contents(step, 1, 64, fmt, 8)
    cache = cache_of(m, host)
    q = randn(step.T, G * 64, seed=4).to(BF)
    want, err = A.attention(q, *host, step, G, 64 ** -0.5, causal, 0)
    none = m.paged_attention(cu(q), cache, step.batch(m), causal=causal)
    check(none, want, err, "without a window")
    for window in ((1 << 31) - 1, (1 << 31) - 2, (1 << 31) - 300, 1 << 30):
        got = m.paged_attention(cu(q), cache, step.batch(m), causal=causal, window=window)
        assert torch.equal(got.view(torch.int16), none.view(torch.int16)), window


# --------------------------------------------------------------- infinite scores
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("lens", [[(1, 1), (1, 40), (1, 3000), (2, 3000)],
                                  [(90, 90), (70, 1500), (1, 200), (3, 3)]])
def test_scores_of_minus_infinity(m, D, G, lens):
    """Keys whose score is -inf have no weight; a row that sees keys and whose every score is
    -inf has a softmax of NaN, one that sees no key is zero (pages that do not exist among
    them, pieces of a long sequence that hold nothing else)."""
    step = A.Step(lens, 16, seed=3)
    if lens[2][1] > 2000:
        step.table[3] = -1                              # sequence 3: sees nothing
        step.table[2, 64:] = -1                         # sequence 2: 1024 keys, all -inf
        gone = {0: lambda p: True, 1: lambda p: p != 7, 2: lambda p: True, 3: lambda p: True}
    else:
        step.table[1, 4:] = -1                          # (its first 64 places exist, all -inf)
        gone = {0: lambda p: p < 37 or p % 3 == 0, 1: lambda p: True, 2: lambda p: p < 199,
                3: lambda p: p < 2}
    host = contents(step, 1, D, "bf16", 8)
    k = host[0]
    k[..., 0] = 0.0
    low = torch.zeros(k.shape[:3], dtype=torch.bool)
    for b, (n, L) in enumerate(lens):
        for p in range(L):
            page, row = place(step, b, p)
            if 0 <= page < step.num_pages and gone[b](p):
                low[page, 0, row] = True
    q = randn(step.T, G, D, seed=4).to(BF)
    q[..., 0] = 1.5
    q = q.reshape(step.T, G * D)
    # wanted: the weight of a key 60 below the others, 10^-26, is none
    k[..., 0] = torch.where(low, torch.tensor(-40.0 * D ** 0.5), torch.tensor(0.0)).to(BF)
    want, err = A.attention(q, *host, step, G, D ** -0.5)
    for b, (n, L) in enumerate(lens):
        for i in range(n):
            sees = [place(step, b, p) for p in range(L - n + i + 1)]
            sees = [bool(low[x[0], 0, x[1]]) for x in sees if 0 <= x[0] < step.num_pages]
            if sees and all(sees):
                want[step.cu[b] + i] = math.nan
    assert bool(torch.isnan(want).any()) and bool(torch.isfinite(want).any())
    k[..., 0] = torch.where(low, torch.tensor(-math.inf), torch.tensor(0.0)).to(BF)
    got = m.paged_attention(cu(q), cache_of(m, host), step.batch(m))
    check(got, want, err, "attention")


@pytest.mark.parametrize("x", [math.inf, math.nan])
@pytest.mark.parametrize("D,G,lens", [(64, 2, [(1, 40), (2, 3000), (1, 9)]), (128, 4, [(90, 1500), (3, 70)]),
                                      (256, 8, [(1, 2000), (40, 600)])])
def test_scores_of_infinity_and_nan(m, x, D, G, lens):
    """A key with an infinite or NaN score in the middle of each sequence: NaN for the rows
    that see it, in whatever piece it lies, and nothing for those that do not."""
    step = A.Step(lens, 16, seed=3)
    host = contents(step, 1, D, "bf16", 8)
    q = randn(step.T, G, D, seed=4).to(BF)
    q[..., 0] = 1.5
    q = q.reshape(step.T, G * D)
    want, err = A.attention(q, *host, step, G, D ** -0.5, True, 30)
    whole, werr = A.attention(q, *host, step, G, D ** -0.5)
    for b, (n, L) in enumerate(lens):
        p = max(0, L - n // 2 - 20)
        page, row = place(step, b, p)
        host[0][page, 0, row, 0] = x
        for i in range(n):
            at = L - n + i
            if p <= at:
                whole[step.cu[b] + i] = math.nan
                if p > at - 30:
                    want[step.cu[b] + i] = math.nan
    cache = cache_of(m, host)
    check(m.paged_attention(cu(q), cache, step.batch(m), window=30), want, err, "window")
    check(m.paged_attention(cu(q), cache, step.batch(m)), whole, werr, "whole")


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,L,gone", [(1, 150, 150, 3), (4, 100, 100, 5), (2, 300, 900, 45), (3, 5, 20, 1),
                                        (2, 1300, 1300, 70)])
def test_rows_whose_first_pages_do_not_exist(m, fmt, D, G, n, L, gone):
    """Rows that see places but no page (zeros) beside rows of the same block that see keys,
    with and without a window."""
    step = A.Step([(n, L), (2, 30)], 16, seed=3)
    step.table[0, :gone] = -1
    host = contents(step, 1, D, fmt, 8)
    cache = cache_of(m, host)
    q = randn(step.T, G * D, seed=4).to(BF)
    for window in (0, 21):
        want, err = A.attention(q, *host, step, G, D ** -0.5, True, window)
        assert bool((want[:n] == 0).all(1).any()) == (L - n < 16 * gone)
        check(m.paged_attention(cu(q), cache, step.batch(m), window=window), want, err, "attention")


# ------------------------------------------------- precision of sequences of few rows
def two_terms(q, host, step, heads, scale, err):
    """The bound of A.attention, `err`, with the probabilities' rounding to one bf16 term
    (2^-8 of the sum of |p v|, the result's rounding on top of it) exchanged for that to
    two: 2^-17, a rest of half a step at most and half a step of that."""
    k, ks, v, vs = host
    size = (v.float().abs() if v.dtype != torch.int8 else v.abs().to(torch.int8)).to(v.dtype)
    total, _ = A.attention(q, k, ks, size, vs, step, heads, scale)
    return err - (A.HALF - 2.0 ** -17) * total * (1 + A.HALF) ** 2


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("D,G,lens,T,most", [
    (128, 4, [(1, 300)], 512, 512),             # one token in a step captured for chunks
    (64, 2, [(16, 700)], 64, 64),
    (256, 4, [(4, 200)], 300, 300),
    (128, 4, [(1, 300), (2, 90), (8, 64)], 900, 300),     # rows behind the last sequence
    (64, 1, [(32, 200), (1, 1), (9, 400)], 120, 40),
    (128, 4, [(1, 300), (200, 300), (8, 64)], 209, 200),  # beside a chunk
])
def test_few_rows_keep_their_precision_in_any_batch(m, fmt, D, G, lens, T, most):
    """Sequences of up to 32 query rows of a kv head (16 of 256-wide heads) have two terms of
    each probability, whatever the step has room for."""
    step = A.Step(lens, 16, seed=3, T=T)
    host = contents(step, 1, D, fmt, 8)
    q = randn(T, G * D, seed=4).to(BF)
    scale = D ** -0.5
    want, err = A.attention(q, *host, step, G, scale)
    tight = two_terms(q, host, step, G, scale, err)
    got = m.paged_attention(cu(q), cache_of(m, host), step.batch(m, most=most))
    for b, (n, _) in enumerate(lens):
        few = n * G <= (16 if D == 256 else 32)
        rows = slice(step.cu[b], step.cu[b] + n)
        check(got[rows], want[rows], (tight if few else err)[rows], "sequence %d" % b)


# ----------------------------------------------- windows without the causal limit
@pytest.mark.parametrize("D,fmt,n,L,window", [(64, "bf16", 2300, 2300, 64), (128, "int8", 1100, 1900, 200),
                                              (256, "bf16", 700, 1500, 33), (64, "fp8", 130, 4000, 5)])
def test_windows_of_tokens_that_see_what_follows(m, D, fmt, n, L, window):
    """Without the causal limit a token sees the window before it and all behind it: the
    first row blocks see the most keys and are cut into pieces, the last ones may see none."""
    step = A.Step([(n, L), (3, 50), (0, 10), (40, 400)], 16, seed=3)
    host = contents(step, 1, D, fmt, 8)
    q = (1.5 * randn(step.T, 2 * D, seed=4)).to(BF)
    want, err = A.attention(q, *host, step, 2, D ** -0.5, False, window)
    got = m.paged_attention(cu(q), cache_of(m, host), step.batch(m), causal=False, window=window)
    check(got, want, err, "attention")


# --------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("D,n,L,B", [(128, 40, 1500, 1), (64, 1, 5000, 3), (256, 90, 1100, 2),
                                     (128, 3, 129, 2), (128, 200, 513, 2)])
@pytest.mark.parametrize("again", [False, True])
def test_workspace_of_the_stated_size(m, D, n, L, B, again):
    """Nothing is written behind the workspace's end; also where the sequences' rows are given
    more than once (ends that go back)."""
    step = A.Step([(n, L)] * B, 16, seed=3)
    host = contents(step, 2, D, "bf16", 8)
    cache = cache_of(m, host)
    T, G = step.T, 4
    q = cu(randn(T, 2 * G * D, seed=4).to(BF))
    ends = [0, T] * B if again else step.cu
    seqs = len(ends) - 1
    table = cu(step.table).repeat(-(-seqs // B), 1)[:seqs]
    batch = m.SequenceBatch(i32(*ends), i32(*[L] * seqs), table, T if again else n, L)
    size = m.moe_w8a8_paged_attention_workspace_size(cache.struct, batch.struct, 2 * G, T)
    room = torch.full((size + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.zeros(T, 2 * G * D, dtype=BF, device="cuda")
    a = m.moe_w8a8_attention_args(2 * G, 1, 0, D ** -0.5, q.data_ptr(), 2 * G * D, out.data_ptr(),
                                  2 * G * D)
    assert m.moe_w8a8_paged_attention(a, cache.struct, batch.struct, T, room.data_ptr(), size,
                                      stream=torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert bool((room[size:] == 0x5a).all())
    if not again:
        want, err = A.attention(q.cpu(), *host, step, 2 * G, D ** -0.5)
        check(out, want, err, "attention")


# ------------------------------------------------------------------ norms of heads
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size,eps", [(1e-20, 16.0), (1e-20, 1e30), (1e-18, 5.0), (1e-30, 1e-3),
                                      (1e-39, 0.0), (9.2e-41, 0.0), (1e-39, 1e-44), (1e-33, 1e-30),
                                      (1e-39, 1e-20), (3e38, 1e30), (1e20, 1e38)])
def test_norms_of_tiny_rows(m, D, size, eps):
    """Head rows far from 1 against every eps: neither what the squares lose nor what eps
    becomes when the row is lifted leaves fp32. (One element of each head is not zero, or
    all of them are.)"""
    step = A.Step([(4, 20)], 16, seed=1)
    x = torch.ones(4, 4, D)
    x[1::2, :, 1:] = 0.0
    x = (size * x).to(BF)
    host = contents(step, 1, D, "bf16", 8)
    q = m.qk_norm_rope(cu(x.view(4, -1)), cache_of(m, host), step.batch(m), 2, norm=True, eps=eps)
    eps = float(torch.tensor(eps, dtype=F32))
    y, e = A.rope(x[:, :2], None, eps, True, None, None, False)
    # (2^-134: half a step of the smallest bf16 numbers)
    check(q, y.reshape(4, -1), (e + A.HALF * (y.abs() + e)).reshape(4, -1) + 2.0 ** -134, "queries")
