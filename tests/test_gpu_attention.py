"""qk_norm_rope, paged_attention and token_logprobs on the GPU against plain 64-bit
forms, within bounds that count the kernels' roundings (tests/attention_ref.py)."""
import math
import sys

import pytest
import torch

import attention_ref as A
import block_ref as R

pytestmark = pytest.mark.gpu
BF, F32, F64, E4, I8 = A.BF, A.F32, A.F64, A.E4, A.I8


@pytest.fixture(scope="module", autouse=True)
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_int8_expert_amd as mod
    mod.load_library()
    return mod


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def cu(t):
    return None if t is None else t.cuda()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def setup(m, step, Hkv, D, fmt, seed):
    shape = (step.num_pages, Hkv, step.page, D)
    k, ks = A.cached(shape, fmt, seed)
    v, vs = A.cached(shape, fmt, seed + 1)
    return (k, ks, v, vs), m.KVCache.of(cu(k), cu(v), cu(ks), cu(vs))


def check_attention(m, step, host, cache, q, heads, out=None, batch=None, **kw):
    D = cache.head_dim
    scale = kw.pop("scale", None)
    want, err = A.attention(q, *host, step, heads, D ** -0.5 if scale is None else scale,
                            kw.get("causal", True), kw.get("window", 0))
    got = m.paged_attention(cu(q), cache, batch or step.batch(m), scale=scale, out=out, **kw)
    torch.cuda.synchronize()
    rows = step.cu[-1]
    R.check(got[:rows], want[:rows], err[:rows], "attention")
    return got


# --------------------------------------------------------------- attention
MIXED = [(1, 1), (5, 37), (0, 50), (3, 3), (1, 0), (70, 200), (4, 2), (33, 33), (2, 129)]


@pytest.mark.parametrize("D,fmt,Hkv,G,page,lens,causal,window", [
    (128, "bf16", 2, 4, 64, [(1, 300), (1, 1), (1, 64), (1, 0), (1, 1031)], True, 0),
    (128, "int8", 2, 8, 32, [(1, 300), (1, 1), (1, 64), (1, 0), (1, 1031)], True, 0),
    (128, "fp8", 1, 16, 16, [(1, 300), (1, 17), (1, 96), (1, 2500)], True, 0),
    (64, "bf16", 3, 1, 16, [(1, 300), (1, 15), (2, 96), (4, 2500)], True, 0),
    (64, "int8", 1, 7, 64, [(1, 300), (1, 15), (2, 96), (2, 2500)], True, 0),
    (64, "fp8", 2, 2, 256, [(1, 300), (0, 15), (2, 96), (1, 2500)], True, 100),
    (256, "bf16", 1, 8, 16, [(1, 300), (1, 15), (2, 96), (1, 700)], True, 0),
    (256, "int8", 2, 3, 32, [(1, 300), (1, 15), (2, 96), (5, 700)], True, 0),
    (256, "fp8", 1, 1, 128, [(1, 300), (1, 15), (2, 96), (5, 700)], True, 33),
    (128, "bf16", 2, 3, 16, MIXED, True, 0),
    (128, "int8", 1, 4, 64, MIXED, True, 19),
    (128, "fp8", 2, 1, 32, MIXED, False, 0),
    (64, "bf16", 2, 4, 128, MIXED, True, 0),
    (64, "int8", 2, 7, 16, MIXED, False, 40),
    (64, "fp8", 1, 5, 32, MIXED, True, 0),
    (256, "bf16", 1, 4, 16, MIXED, True, 0),
    (256, "int8", 1, 2, 64, MIXED, True, 0),
    (256, "fp8", 2, 2, 16, MIXED, True, 7),
    (128, "bf16", 1, 64, 64, [(1, 400), (1, 33)], True, 0),
    (128, "fp8", 1, 24, 64, [(2, 400), (1, 33)], True, 0),
    (128, "bf16", 1, 5, 64, [(300, 300), (200, 1100), (1, 900)], True, 0),
    (128, "int8", 2, 1, 32, [(257, 513), (64, 64), (1, 1)], True, 0),
    (64, "bf16", 1, 2, 64, [(511, 800)], True, 200),
    (256, "bf16", 1, 1, 64, [(130, 400), (129, 129)], True, 0),
    (256, "fp8", 1, 2, 256, [(130, 400), (129, 129)], False, 0),
])
def test_attention(m, D, fmt, Hkv, G, page, lens, causal, window):
    say("attention", D, fmt, Hkv, G, page, lens, causal, window)
    step = A.Step(lens, page, seed=D + G)
    host, cache = setup(m, step, Hkv, D, fmt, 5)
    q = (1.5 * randn(step.T, Hkv * G * D, seed=9)).to(BF)
    check_attention(m, step, host, cache, q, Hkv * G, causal=causal, window=window)


def test_attention_many_sequences(m):
    """More sequences than a wavefront has lanes, many of them without tokens."""
    g = torch.Generator().manual_seed(1)
    lens = [(int(n), int(n) + int(c)) for n, c in zip(
        torch.randint(0, 3, (333,), generator=g), torch.randint(0, 150, (333,), generator=g))]
    step = A.Step(lens, 16, seed=3)
    host, cache = setup(m, step, 1, 64, "bf16", 6)
    q = randn(step.T, 2 * 64, seed=2).to(BF)
    check_attention(m, step, host, cache, q, 2)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("lens", [[(1, 40001)], [(2, 20000), (1, 9000), (1, 3)]])
def test_attention_long(m, fmt, lens):
    """Keys split over many blocks."""
    step = A.Step(lens, 64, seed=3)
    host, cache = setup(m, step, 2, 128, fmt, 7)
    q = (2 * randn(step.T, 8 * 128, seed=4)).to(BF)
    check_attention(m, step, host, cache, q, 8)
    # bounds that say little size the launch differently, the result is as exact
    check_attention(m, step, host, cache, q, 8, batch=step.batch(m, longest=16))
    check_attention(m, step, host, cache, q, 8, batch=step.batch(m, longest=1 << 20, most=9))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[(1, 100), (1, 33)], [(90, 300), (1, 70), (17, 40)]])
def test_attention_pages_that_do_not_exist(m, fmt, lens):
    step = A.Step(lens, 16, seed=3)
    step.table[0, 1] = -1
    step.table[0, 4] = step.num_pages
    step.table[1, :3] = 1 << 30
    host, cache = setup(m, step, 2, 128, fmt, 8)
    q = randn(step.T, 4 * 128, seed=4).to(BF)
    check_attention(m, step, host, cache, q, 4)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,lens", [(4, [(1, 100), (3, 33)]), (2, [(90, 300), (1, 70), (40, 40)])])
def test_attention_unseen_keys_hold_anything(m, D, G, lens):
    """NaN and infinities in places that hold no key, and in keys and values of tokens
    that come later: no part in what does not see them; all of it in what does."""
    step = A.Step(lens, 16, seed=3)
    host, cache = setup(m, step, 1, D, "bf16", 8)
    k, _, v, _ = host
    at = lambda b, p: (int(step.table[b, p // 16]), 0, p % 16)  # noqa: E731
    for b, (n, L) in enumerate(lens):       # behind the last key, to the page's end
        for p in range(L, -(-L // 16) * 16):
            k[at(b, p)] = math.nan
            v[at(b, p)] = math.nan if p % 2 else math.inf
    n, L = lens[-1]
    v[at(len(lens) - 1, L - 1)][0] = math.inf
    v[at(len(lens) - 1, L - 1)][3] = math.nan
    v[at(len(lens) - 1, L - n // 2)][5] = -math.inf
    n, L = lens[0]
    v[at(0, L - 1)][::7] = math.nan
    k[at(0, L - 1)] = 1.0                   # (a key of later tokens: finite scores)
    free = set(range(step.num_pages)) - set(step.table.flatten().tolist())
    for p in free:
        k[p] = math.nan
        v[p] = math.nan
    cache.k.copy_(k)
    cache.v.copy_(v)
    q = randn(step.T, G * D, seed=4).to(BF)
    check_attention(m, step, host, cache, q, G)
    # keys that are NaN: only rows that see them
    kn = k.clone()
    kn[at(0, lens[0][1] - 1)] = math.nan
    cache.k.copy_(kn)
    got = m.paged_attention(cu(q), cache, step.batch(m)).cpu()
    n = lens[0][0]
    assert torch.isnan(got[n - 1].float()).all()
    if n > 1:
        want, err = A.attention(q, *host, step, G, D ** -0.5)
        R.check(got[:n - 1], want[:n - 1], err[:n - 1], "rows that do not see it")


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_attention_scales_of_unseen_keys(m, fmt):
    lens = [(3, 30), (50, 90)]
    step = A.Step(lens, 16, seed=3)
    host, cache = setup(m, step, 2, 64, fmt, 8)
    for b, (n, L) in enumerate(lens):
        for p in range(L, -(-L // 16) * 16):
            cache.k_scale[int(step.table[b, p // 16]), :, p % 16] = math.inf
            cache.v_scale[int(step.table[b, p // 16]), :, p % 16] = math.nan
    # the last token's value: a NaN scale reaches that token alone
    b, p = 1, 89
    cache.v_scale[int(step.table[b, p // 16]), :, p % 16] = math.nan
    host[3][int(step.table[b, p // 16]), :, p % 16] = math.nan
    q = randn(step.T, 6 * 64, seed=4).to(BF)
    check_attention(m, step, host, cache, q, 6)


@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.3, 2.0), (1.0, 30.0), (1e-3, 1.0)])
def test_attention_scales_and_sizes(m, scale, size):
    step = A.Step([(1, 500), (70, 150)], 32, seed=3)
    host, cache = setup(m, step, 1, 128, "bf16", 8)
    q = (size * randn(step.T, 4 * 128, seed=4)).to(BF)
    check_attention(m, step, host, cache, q, 4, scale=scale)


@pytest.mark.parametrize("lens", [[(1, 200), (2, 31)], [(80, 200), (2, 31)]])
def test_attention_strides_and_rows_behind(m, lens):
    """Rows at odd addresses inside wider buffers; what is not the result's stays."""
    T = sum(n for n, _ in lens) + 5
    step = A.Step(lens, 32, seed=3, T=T)
    host, cache = setup(m, step, 2, 64, "bf16", 8)
    W = 6 * 64
    qb = randn(T, W + 37, seed=4).to(BF).cuda()
    ob = torch.full((T, W + 51), 3.0, dtype=BF, device="cuda")
    q, out = qb[:, 5:5 + W], ob[:, 9:9 + W]
    want, err = A.attention(q.cpu(), *host, step, 6, 64 ** -0.5)
    assert m.paged_attention(q, cache, step.batch(m), out=out) is out
    n = step.cu[-1]
    R.check(out[:n], want[:n], err[:n], "attention")
    rest = ob.clone()
    rest[:n, 9:9 + W] = 3.0
    assert bool((rest == 3.0).all())


def test_attention_layers_of_one_buffer(m):
    """Caches whose pages lie apart: the layers of one buffer."""
    step = A.Step([(1, 200), (40, 90)], 16, seed=3)
    shape = (step.num_pages, 3, 2, 16, 128)
    kb, ksb = A.cached(shape, "int8", 1)
    vb, vsb = A.cached(shape, "int8", 2)
    dev = [cu(t) for t in (kb, vb, ksb, vsb)]
    for layer in (0, 2):
        cache = m.KVCache.of(*(t[:, layer] for t in dev))
        host = (kb[:, layer], ksb[:, layer], vb[:, layer], vsb[:, layer])
        q = randn(step.T, 4 * 128, seed=layer).to(BF)
        check_attention(m, step, host, cache, q, 4)


def test_attention_far_pages(m):
    """Pages past 2^32 bytes of a cache."""
    D, page, pages = 128, 256, 70000                # 4.6 GB of int8 keys
    step = A.Step([(1, 600), (20, 300)], page, seed=3)
    host, _ = setup(m, step, 2, D, "int8", 8)
    k = torch.empty(pages, 2, page, D, dtype=I8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty(pages, 2, page, dtype=F32, device="cuda")
    vs = torch.empty_like(ks)
    base = pages - step.num_pages
    for t, x in ((k, 0), (ks, 1), (v, 2), (vs, 3)):
        t[base:] = host[x].cuda()
    q = randn(step.T, 4 * D, seed=4).to(BF)
    want, err = A.attention(q, *host, step, 4, D ** -0.5)
    step.table += base * (step.table >= 0)
    got = m.paged_attention(cu(q), m.KVCache.of(k, v, ks, vs), step.batch(m))
    R.check(got, want, err, "attention")


def test_attention_follows_the_batch_in_a_graph(m):
    """A captured call reads lengths and pages when it is replayed, beside eager calls."""
    lens0 = [(1, 2000), (1, 5), (1, 130)]
    steps = [A.Step(l, 32, seed=i, spare=80 - sum(-(-x[1] // 32) for x in l)) for i, l in enumerate(
        (lens0, [(1, 30), (1, 2100), (1, 1)], [(1, 0), (0, 9), (1, 700)]))]
    width = max(s.table.shape[1] for s in steps)
    host, cache = setup(m, steps[0], 2, 128, "fp8", 8)
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    cuv = torch.zeros(4, dtype=torch.int32, device="cuda")
    length = torch.zeros(3, dtype=torch.int32, device="cuda")
    batch = m.SequenceBatch(cuv, length, table, 1, 2100)
    q = torch.zeros(3, 8 * 128, dtype=BF, device="cuda")

    def load(i):
        s = steps[i]
        table.fill_(-1)
        table[:, :s.table.shape[1]] = s.table.cuda()
        cuv.copy_(torch.tensor(s.cu, dtype=torch.int32))
        length.copy_(torch.tensor([l for _, l in s.lens], dtype=torch.int32))
        q.copy_(randn(3, 8 * 128, seed=20 + i).to(BF))

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.paged_attention(q, cache, batch)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.paged_attention(q, cache, batch)
    for i in (0, 1, 2, 1, 0):
        load(i)
        eager = m.paged_attention(q, cache, batch)
        graph.replay()
        torch.cuda.synchronize()
        s = steps[i]
        want, err = A.attention(q.cpu()[:s.cu[-1]], *host, s, 8, 128 ** -0.5)
        R.check(out[:s.cu[-1]], want, err, "replay %d" % i)
        assert torch.equal(out[:s.cu[-1]].view(torch.int16), eager[:s.cu[-1]].view(torch.int16))


def test_attention_two_streams(m):
    """Calls on two streams over one cache at once, each against its own batch."""
    steps = [A.Step([(1, 3000), (1, 70)], 64, seed=1), A.Step([(90, 700)], 64, seed=2)]
    host, cache = setup(m, steps[0], 2, 128, "bf16", 8)
    qs = [randn(s.T, 4 * 128, seed=i).to(BF) for i, s in enumerate(steps)]
    batches = [s.batch(m) for s in steps]
    dev = [cu(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(m.paged_attention(dev[i], cache, batches[i]))
    torch.cuda.synchronize()
    for i, s in enumerate(steps):
        want, err = A.attention(qs[i], *host, s, 4, 128 ** -0.5)
        for g in got[i]:
            R.check(g, want, err, "stream %d" % i)


# ------------------------------------------------------------------- rope
def check_rope(m, step, Hq, Hkv, D, fmt, norm, rot, pairs, seed=0, size=1.0, qkv=None, eps=1e-6,
               positions=None, weights=True, in_place=False):
    qkv = (size * randn(step.T, (Hq + 2 * Hkv) * D, seed=seed)).to(BF) if qkv is None else qkv
    g = torch.Generator().manual_seed(seed + 1)
    qw = 1 + 0.2 * torch.randn(D, generator=g) if norm and weights else None
    kw = 1 + 0.2 * torch.randn(D, generator=g) if norm and weights else None
    freq = 1e4 ** (-torch.arange(0, rot, 2, dtype=F64) / rot) if rot else None
    host, cache = setup(m, step, Hkv, D, fmt, seed + 2)
    before = [t.clone() if t is not None else None for t in host]
    dev = qkv.cuda()
    out = dev[:, :Hq * D] if in_place else None
    q = m.qk_norm_rope(dev, cache, step.batch(m), Hq, norm=norm, q_weight=cu(qw), k_weight=cu(kw),
                       eps=eps, inv_freq=cu(freq), interleaved=pairs, positions=cu(positions),
                       out=out)
    torch.cuda.synchronize()
    x = qkv.view(step.T, Hq + 2 * Hkv, D)
    k, ks, v, vs = before
    bound = {n: torch.zeros(t.shape, dtype=F64) for n, t in (("k", k), ("v", v))}
    want = {"k": k.float().double(), "v": v.float().double()}
    swant = {"k": None if ks is None else ks.double(), "v": None if vs is None else vs.double()}
    sbound = {n: None if ks is None else torch.zeros(ks.shape, dtype=F64) for n in ("k", "v")}
    for b, (n, L) in enumerate(step.lens):
        if n == 0:
            continue
        rows = slice(step.cu[b], step.cu[b] + n)
        place = torch.arange(L - n, L)
        pos = place if positions is None else positions[rows]
        y, e = A.rope(x[rows, :Hq], qw, eps, norm, pos, freq, pairs)
        R.check(q[rows], y.reshape(n, -1), (e + A.HALF * (y.abs() + e)).reshape(n, -1) + 1e-40, "q")
        y, e = A.rope(x[rows, Hq:Hq + Hkv], kw, eps, norm, pos, freq, pairs)
        for name, yy, ee in (("k", y, e), ("v", x[rows, Hq + Hkv:].double(), torch.zeros_like(e))):
            page = step.table[b][(place.clamp_min(0) // step.page)].long()
            ok = (place >= 0) & (page >= 0) & (page < step.num_pages)
            at = (page[ok], slice(None), (place % step.page)[ok])
            yy, ee = yy[ok], ee[ok]
            if fmt == "bf16":
                want[name][at] = yy
                bound[name][at] = (ee + A.HALF * (yy.abs() + ee) + 1e-40) if name == "k" else 0.0
                continue
            q8, s, off, rel = R.requantised(yy.reshape(-1, D), ee.reshape(-1, D), fmt == "fp8")
            want[name][at] = q8.reshape(yy.shape)
            bound[name][at] = off.reshape(yy.shape)
            swant[name][at] = s.reshape(yy.shape[:2])
            sbound[name][at] = (s * (rel + 4 * R.U)).reshape(yy.shape[:2])
    for name, t, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        R.check(t.float().reshape(-1, D), want[name].reshape(-1, D), bound[name].reshape(-1, D), name)
        if s is not None:
            R.check(s.reshape(-1, step.page), swant[name].reshape(-1, step.page),
                    sbound[name].reshape(-1, step.page), name + " scales")
    return q, cache


@pytest.mark.parametrize("D,fmt,Hq,Hkv,page,norm,rot,pairs", [
    (128, "bf16", 8, 2, 64, True, 128, False),
    (128, "int8", 7, 1, 16, True, 64, True),
    (128, "fp8", 5, 5, 32, False, 128, True),
    (64, "bf16", 3, 3, 16, True, 32, False),
    (64, "int8", 14, 2, 128, False, 16, True),
    (64, "fp8", 1, 1, 16, True, 64, False),
    (256, "bf16", 2, 1, 16, True, 64, True),
    (256, "int8", 3, 3, 256, True, 256, False),
    (256, "fp8", 6, 2, 32, False, 0, False),
    (128, "bf16", 4, 4, 16, False, 112, False),
])
def test_rope(m, D, fmt, Hq, Hkv, page, norm, rot, pairs):
    say("rope", D, fmt, Hq, Hkv, page, norm, rot, pairs)
    step = A.Step([(1, 1), (5, 37), (0, 50), (40, 200), (4, 2), (3, 3)], page, seed=D)
    check_rope(m, step, Hq, Hkv, D, fmt, norm, rot, pairs, seed=3)


def test_rope_far_places_and_positions(m):
    step = A.Step([(3, 1000003), (2, 5)], 256, seed=1)
    check_rope(m, step, 2, 1, 64, "bf16", False, 64, False)
    pos = torch.tensor([1 << 40, 7, 0, -3, 123456789])
    check_rope(m, step, 2, 1, 64, "int8", True, 64, True, positions=pos)


def test_rope_pages_that_do_not_exist(m):
    step = A.Step([(40, 60), (3, 20)], 16, seed=1)
    step.table[0, 2] = -1
    step.table[0, 3] = step.num_pages
    step.table[1, 1] = 1 << 30
    check_rope(m, step, 4, 2, 128, "fp8", True, 128, False)


@pytest.mark.parametrize("size", [1e-30, 1e-19, 1e18, 1e37])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_rope_extreme_rows(m, size, fmt):
    step = A.Step([(9, 20)], 16, seed=1)
    check_rope(m, step, 4, 2, 128, fmt, True, 128, False, size=size, eps=0.0)
    check_rope(m, step, 4, 2, 64, fmt, True, 64, True, size=size, weights=False)


def test_rope_rows_that_are_not_finite(m):
    """A head with a NaN or an infinity: that head of that token alone."""
    step = A.Step([(6, 6)], 16, seed=1)
    D, Hq, Hkv = 64, 2, 2
    clean = randn(6, (Hq + 2 * Hkv) * D, seed=1).to(BF)
    dirty = clean.clone()
    dirty[1, 3] = math.nan               # query head 0
    dirty[2, (Hq + 1) * D + 5] = math.inf   # key head 1
    dirty[4, (Hq + Hkv) * D + 9] = math.nan  # value head 0
    for fmt in ("bf16", "int8"):
        _, c0 = setup(m, step, Hkv, D, fmt, 4)
        _, c1 = setup(m, step, Hkv, D, fmt, 4)
        f = cu(1e4 ** (-torch.arange(0, D, 2, dtype=F64) / D))
        q0 = m.qk_norm_rope(cu(clean), c0, step.batch(m), Hq, norm=True, inv_freq=f)
        q1 = m.qk_norm_rope(cu(dirty), c1, step.batch(m), Hq, norm=True, inv_freq=f)
        assert torch.isnan(q1[1, :D].float()).all()
        q1[1, :D] = q0[1, :D]
        assert torch.equal(q0.view(torch.int16), q1.view(torch.int16))
        page = int(step.table[0, 0])
        for n, tok, head in (("k", 2, 1), ("v", 4, 0)):
            a, b = getattr(c0, n), getattr(c1, n)
            if fmt == "bf16":
                assert torch.isnan(b[page, head, tok].float()).any()
            else:
                sa, sb = getattr(c0, n + "_scale"), getattr(c1, n + "_scale")
                assert math.isnan(float(sb[page, head, tok])) and int(b[page, head, tok].abs().sum()) == 0
                sb[page, head, tok] = sa[page, head, tok]
                assert torch.equal(sa, sb)
            b[page, head, tok] = a[page, head, tok]
            assert torch.equal(a, b)


def test_rope_in_place_and_strides(m):
    step = A.Step([(5, 37), (3, 3)], 16, seed=1, T=11)
    step.T = 8
    q0, c0 = check_rope(m, step, 6, 2, 64, "bf16", True, 64, False)
    q1, c1 = check_rope(m, step, 6, 2, 64, "bf16", True, 64, False, in_place=True)
    assert torch.equal(q0.view(torch.int16), q1.view(torch.int16))
    # a wider buffer at an odd address, rows behind the last sequence
    W = 10 * 64
    src = randn(8, W, seed=0).to(BF).cuda()
    wide = torch.full((11, W + 13), 5.0, dtype=BF, device="cuda")
    wide[:8, 3:3 + W] = src
    out = torch.full((11, 6 * 64 + 7), 5.0, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    qw = (1 + 0.2 * torch.randn(64, generator=g)).cuda()
    kw = (1 + 0.2 * torch.randn(64, generator=g)).cuda()
    f = cu(1e4 ** (-torch.arange(0, 64, 2, dtype=F64) / 64))
    _, c2 = setup(m, step, 2, 64, "bf16", 2)
    m.qk_norm_rope(wide[:, 3:3 + W], c2, step.batch(m), 6, norm=True, q_weight=qw, k_weight=kw,
                   inv_freq=f, out=out[:, 1:1 + 6 * 64])
    assert torch.equal(out[:8, 1:1 + 384].contiguous().view(torch.int16), q0.view(torch.int16))
    assert torch.equal(c2.k.view(torch.int16), c0.k.view(torch.int16))
    out[:8, 1:1 + 384] = 5.0
    assert bool((out == 5.0).all())


# --------------------------------------------------------------- logprobs
def check_logprobs(m, x, tokens, top, steps=None):
    T, V = x.shape
    lp, dlp, ent, dent, tt, tl, dtl = A.logprobs(x, tokens, top, V / 256 + 128)
    r = m.token_logprobs(cu(x), cu(tokens), top=top)
    col = lambda t: t.reshape(T, -1)  # noqa: E731
    if tokens is not None:
        R.check(col(r.logprobs), col(lp), col(dlp), "logprobs")
    R.check(col(r.entropy), col(ent), col(dent), "entropy")
    if top:
        assert torch.equal(r.top_tokens.cpu(), tt), "top tokens"
        R.check(r.top_logprobs, tl, dtl, "top logprobs")
    return r


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (3, 7, 7), (2, 64, 64), (5, 1000, 5), (1, 4097, 20),
                                     (33, 8191, 1), (4, 32003, 20), (2, 131072, 64), (1, 151937, 0),
                                     (300, 513, 3), (1, 1 << 20, 8), (700, 5000, 2)])
def test_logprobs(m, dtype, T, V, top):
    say("logprobs", dtype, T, V, top)
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(T, V, generator=g) * (1 + 3 * torch.rand(T, 1, generator=g))).to(dtype)
    tokens = torch.randint(0, V, (T,), generator=g)
    tokens[0] = V - 1
    check_logprobs(m, x, tokens, top)


@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two", "peak", "late", "offset",
                                  "zeros"])
@pytest.mark.parametrize("V", [1000, 40000, 150001])
def test_logprobs_orders(m, kind, V):
    """Ties and orders in which every element, or none, is a new largest one."""
    i = torch.arange(V, dtype=F32)
    x = {"equal": torch.full((V,), 2.5), "rising": i / 1024, "falling": -i / 1024,
         "two": (i % 2), "peak": torch.where(i == V // 3, 80.0, -20.0),
         "late": torch.where(i >= V - 70, 3.0, 1.0), "offset": 3e4 + (i * 7 % 13),
         "zeros": torch.where(i % 3 == 0, -0.0, 0.0)}[kind]
    x = torch.stack([x, x.flip(0)])
    for dtype in (F32, BF):
        check_logprobs(m, x.to(dtype), torch.tensor([V // 3, 0]), 33)


def test_logprobs_masked_and_not_finite(m):
    V = 5000
    x = randn(7, V, seed=1)
    x[0, ::2] = -math.inf
    x[1, 5:] = torch.finfo(F32).min      # masked by the lowest value
    x[2, :] = -math.inf
    x[3, 77] = math.nan
    x[4, 88] = math.inf
    x[5, :] = -math.inf
    x[5, 9] = 1.0
    tokens = torch.tensor([1, 2, 3, 4, 5, 9, V])
    r = m.token_logprobs(cu(x), cu(tokens), top=4)
    for t in (0, 1, 5):
        lp, dlp, ent, dent, tt, tl, dtl = A.logprobs(x[t:t + 1], tokens[t:t + 1], 4, V / 256 + 128)
        one = lambda v: v[t:t + 1].reshape(1, -1)  # noqa: E731
        if t != 0:
            assert torch.equal(r.top_tokens[t].cpu()[:1], tt[0, :1])
        else:
            assert torch.equal(r.top_tokens[t].cpu(), tt[0])
        R.check(one(r.logprobs), lp.reshape(1, -1), dlp.reshape(1, -1), "logprobs")
        ent = ent if t == 1 else None
        if ent is not None:
            R.check(one(r.entropy), ent.reshape(1, -1), dent.reshape(1, -1), "entropy")
    # (the reference's entropy of rows with -inf is 0 * inf: computed here without them)
    keep = x[0, 1::2].double()
    p = torch.softmax(keep, 0)
    assert abs(float(r.entropy[0]) + float((p * torch.log(p)).sum())) < 1e-5
    assert float(r.entropy[5]) == 0.0 and float(r.logprobs[5]) == 0.0
    for t in (2, 3, 4):
        assert math.isnan(float(r.logprobs[t])) and math.isnan(float(r.entropy[t]))
        assert torch.isnan(r.top_logprobs[t]).all()
    assert r.top_tokens[2].tolist() == [0, 1, 2, 3]
    assert int(r.top_tokens[3, 0]) == 77 and int(r.top_tokens[4, 0]) == 88
    assert math.isnan(float(r.logprobs[6])) and math.isfinite(float(r.entropy[6]))
    assert r.top_tokens[5].tolist() == [9, 0, 1, 2]


def test_logprobs_strides_parts_and_graph(m):
    wide = randn(9, 3010, seed=1).cuda()
    x = wide[:, 5:3006]
    tokens = torch.arange(9).cuda()
    a = m.token_logprobs(x, tokens, top=5)
    b = m.token_logprobs(x.contiguous(), tokens, top=5)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    c = m.token_logprobs(x, top=5, entropy=False)
    assert c.logprobs is None and c.entropy is None and torch.equal(c.top_tokens, a.top_tokens)
    d = m.token_logprobs(x, tokens, entropy=False)
    assert d.top_tokens is None and torch.equal(d.logprobs, a.logprobs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.token_logprobs(x, tokens, top=5)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = m.token_logprobs(x, tokens, top=5)
    for i in range(4):
        wide.copy_(randn(9, 3010, seed=10 + i))
        e = m.token_logprobs(x, tokens, top=5)
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(r, e):
            assert torch.equal(u, v)


# --------------------------------------------------------------- together
class Decoder:
    """Two decoder layers and an LM head as a user of the W8A8 blocks builds them."""
    H, F, V, Hq, Hkv, D, PAGE = 320, 200, 333, 6, 2, 64, 16

    def __init__(self, m, fp8, fmt, pages):
        self.m, self.fmt = m, "fp8" if fp8 else "int8"
        H, F, V, D = self.H, self.F, self.V, self.D
        W = (self.Hq + 2 * self.Hkv) * D

        def linear(k, n, seed):
            p = m.W8A8Linear(k, n, fp8=fp8)
            p.quantise(cu(randn(n, k, seed=seed) / math.sqrt(k)))
            return p

        self.layers = []
        for i in range(2):
            ffn = m.W8A8FFN(H, F, fp8=fp8)
            ffn.quantise(cu(randn(2 * F, H, seed=40 + i) / math.sqrt(H)),
                         cu(randn(H, F, seed=50 + i) / math.sqrt(F)))
            self.layers.append(dict(
                qkv=linear(H, W, 10 + i), proj=linear(self.Hq * D, H, 20 + i), ffn=ffn,
                cache=m.KVCache(pages, self.PAGE, self.Hkv, D, fmt),
                norms=[cu(1 + 0.1 * randn(H, seed=30 + 2 * i + j)) for j in range(2)],
                qw=cu(1 + 0.1 * randn(D, seed=60 + i)), kw=cu(1 + 0.1 * randn(D, seed=70 + i))))
        self.head, self.last = linear(H, V, 99), cu(1 + 0.1 * randn(H, seed=98))
        self.freq = cu(1e4 ** (-torch.arange(0, D, 2, dtype=F64) / D))

    def __call__(self, x, batch, tokens):
        m, seen, y, res = self.m, [], x, None
        for layer in self.layers:
            a = m.add_norm(y, res, weight=layer["norms"][0], codes=self.fmt, normed=False)
            q = m.qk_norm_rope(layer["qkv"](codes=(a.codes, a.scales)), layer["cache"], batch,
                               self.Hq, norm=True, q_weight=layer["qw"], k_weight=layer["kw"],
                               inv_freq=self.freq)
            o = m.paged_attention(q, layer["cache"], batch)
            seen.append((q, o))
            b = m.add_norm(layer["proj"](o), a.residual, weight=layer["norms"][1],
                           codes=self.fmt, normed=False)
            y, res = layer["ffn"](codes=(b.codes, b.scales)), b.residual
        c = m.add_norm(y, res, weight=self.last, codes=self.fmt, normed=False, residual_out=False)
        logits = self.head(codes=(c.codes, c.scales), out_dtype=F32)
        return seen, logits, m.token_logprobs(logits, tokens, top=5)


def check_run(run, step, tokens, result):
    """Attention and answers of a run against the plain forms of their actual operands."""
    seen, logits, r = result
    T = step.cu[-1]
    for layer, (q, o) in zip(run.layers, seen):
        c = layer["cache"]
        host = [None if t is None else t.cpu() for t in (c.k, c.k_scale, c.v, c.v_scale)]
        want, err = A.attention(q.cpu(), *host, step, run.Hq, run.D ** -0.5)
        R.check(o[:T], want[:T], err[:T], "attention")
    lp, dlp, ent, dent, tt, tl, dtl = A.logprobs(logits.cpu(), tokens, 5, run.V / 256 + 128)
    R.check(r.logprobs[:, None], lp[:, None], dlp[:, None], "logprobs")
    R.check(r.entropy[:, None], ent[:, None], dent[:, None], "entropy")
    assert torch.equal(r.top_tokens.cpu(), tt)
    R.check(r.top_logprobs, tl, dtl, "top logprobs")


def same(a, b):
    seen_a, logits_a, ra = a
    seen_b, logits_b, rb = b
    for u, v in zip(seen_a, seen_b):
        for x, y in zip(u, v):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(logits_a, logits_b)
    for x, y in zip(ra, rb):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fp8,fmt", [(False, "int8"), (True, "fp8"), (False, "bf16")])
def test_decoder_prefill_then_steps_in_a_graph(m, fp8, fmt):
    """A ragged prefill, then steps of one token: eager on another stream, and captured once
    and replayed, with the same results. With INT8 weights, whose sums are exact, keys and
    values of the first layer, which no attention precedes, are those of one prefill."""
    lens = [37, 5, 0, 64, 1]
    steps = 3
    every = A.Step([(n, n + steps) for n in lens], Decoder.PAGE, seed=4)
    run = Decoder(m, fp8, fmt, every.num_pages)
    B, V = len(lens), run.V
    words = [randn(n + steps, run.H, seed=80 + b).to(BF) for b, n in enumerate(lens)]

    def part(new, length):
        s = A.Step(list(zip(new, length)), Decoder.PAGE)
        s.table, s.num_pages = every.table, every.num_pages
        x = torch.cat([words[b][l - n:l] for b, (n, l) in enumerate(zip(new, length))])
        return s, x

    s, x = part(lens, lens)
    tokens = torch.arange(s.T) * 7 % V
    say("prefill", fp8, fmt)
    check_run(run, s, tokens, run(cu(x), s.batch(m), cu(tokens)))

    # steps of one token over fixed buffers
    cuv = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    length = torch.zeros(B, dtype=torch.int32, device="cuda")
    batch = m.SequenceBatch(cuv, length, every.table.cuda(), 1, every.longest)
    xs, ts = torch.zeros(B, run.H, dtype=BF, device="cuda"), cu(torch.arange(B) * 11 % V)
    graph, out = None, None
    side = torch.cuda.Stream()
    for i in range(steps):
        s, x = part([1] * B, [n + i + 1 for n in lens])
        length.copy_(torch.tensor([n + i + 1 for n in lens], dtype=torch.int32))
        xs.copy_(x)
        say("step", i)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            eager = run(xs, batch, ts)
        torch.cuda.synchronize()
        check_run(run, s, ts.cpu(), eager)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = run(xs, batch, ts)
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            same(out, eager)

    # one prefill of everything writes the same keys and values in the first layer
    c = run.layers[0]["cache"]
    before = [t.clone() for t in (c.k, c.v)]
    s, x = part([n + steps for n in lens], [n + steps for n in lens])
    tokens = torch.arange(s.T) % V
    say("whole")
    check_run(run, s, tokens, run(cu(x), s.batch(m), cu(tokens)))
    if not fp8:  # (sums of FP8 products are rounded, in an order of each kernel of the product)
        for u, v in zip(before, (c.k, c.v)):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_rope_follows_the_batch_in_a_graph(m):
    """A captured call writes where lengths and pages say when it is replayed."""
    cases = [A.Step([(2, 30), (1, 9)], 16, seed=1, spare=3), A.Step([(1, 3), (2, 40)], 16, seed=2)]
    pages = max(s.num_pages for s in cases)
    width = max(s.table.shape[1] for s in cases)
    D, Hq, Hkv = 128, 4, 2
    cuv = torch.zeros(3, dtype=torch.int32, device="cuda")
    length = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    batch = m.SequenceBatch(cuv, length, table, 2, 40)
    x = torch.zeros(3, (Hq + 2 * Hkv) * D, dtype=BF, device="cuda")
    f = cu(1e4 ** (-torch.arange(0, D, 2, dtype=F64) / D))
    caches = [m.KVCache(pages, 16, Hkv, D, "int8") for _ in range(2)]

    def load(i):
        s = cases[i]
        cuv.copy_(torch.tensor(s.cu, dtype=torch.int32))
        length.copy_(torch.tensor([n for _, n in s.lens], dtype=torch.int32))
        table.fill_(-1)
        table[:, :s.table.shape[1]] = s.table.cuda()
        x.copy_(randn(3, x.shape[1], seed=5 + i).to(BF))

    load(0)
    call = lambda c: m.qk_norm_rope(x, c, batch, Hq, norm=True, inv_freq=f)  # noqa: E731
    call(caches[0])
    for c in caches:
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call(caches[0])
    for i in (0, 1, 0, 1):
        load(i)
        graph.replay()
        e = call(caches[1])
        torch.cuda.synchronize()
        assert torch.equal(q.view(torch.int16), e.view(torch.int16))
        for n in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)), n


# ------------------------------------------------------------------ edges
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_attention_last_places(m, n, fmt):
    """A sequence as long as places are counted (2^31 - 1024 keys), a window over its end:
    its last pages alone exist."""
    D, page, W = 64, 256, 300
    L = (1 << 31) - 1024
    width = L // page
    step = A.Step([(n, n + W)], page, seed=3)
    step.table = step.table[:, :-(-(n + W) // page)]
    host, cache = setup(m, step, 1, D, fmt, 8)
    q = randn(n, 2 * D, seed=4).to(BF)
    # the same keys at the end of a long sequence: places differ by a multiple of a page
    short = -(-(n + W) // page) * page
    ref = A.Step([(n, short)], page, seed=3)
    ref.table, ref.num_pages = step.table, step.num_pages
    want, err = A.attention(q, *host, ref, 2, D ** -0.5, True, W)
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, width - short // page:] = cu(ref.table[0])
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    for length in (width * page, (1 << 31) - 1):  # (past the table: as far as it goes)
        batch = m.SequenceBatch(i32(0, n), i32(length), table, n, 1 << 20)
        got = m.paged_attention(cu(q), cache, batch, window=W)
        torch.cuda.synchronize()
        R.check(got, want, err, "last places")


def test_nothing_to_do(m):
    """No rows, no sequences, sequences without tokens or without pages."""
    _, cache = setup(m, A.Step([(1, 20)], 16), 1, 64, "bf16", 3)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    for T, cuv, lens, width in ((0, (0, 0), (7,), 1), (0, (0,), (), 2), (2, (0,), (), 0),
                                (2, (0, 0, 0), (5, 0), 1), (2, (0, 2), (2,), 0)):
        batch = m.SequenceBatch(i32(*cuv), i32(*lens),
                                torch.zeros(len(lens), width, dtype=torch.int32, device="cuda"),
                                2, 20)
        before = cache.k.clone()
        x = randn(T, 4 * 64, seed=1).to(BF).cuda()
        out = torch.full((T, 128), 5.0, dtype=BF, device="cuda")
        m.qk_norm_rope(x, cache, batch, 2, norm=True, out=out)
        there = cuv[-1]
        assert bool((out[there:] == 5.0).all()) and torch.equal(before, cache.k)
        out.fill_(5.0)
        m.paged_attention(x[:, :128], cache, batch, out=out)
        assert bool((out[there:] == 5.0).all()) and bool((out[:there] == 0).all())
    r = m.token_logprobs(torch.zeros(0, 77, device="cuda"), torch.zeros(0, dtype=torch.int64).cuda(),
                         top=3)
    assert r.logprobs.shape == (0,) and r.top_tokens.shape == (0, 3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 90])
def test_attention_scores_far_below_zero(m, D, n):
    """Scores of -10^31 and less, far apart: the largest have all the weight."""
    L, big = 200, 2.0 ** 52
    step = A.Step([(n, L)], 16, seed=1)
    _, cache = setup(m, step, 1, D, "bf16", 3)
    j = torch.arange(L)
    for p in range(L):
        cache.k[int(step.table[0, p // 16]), 0, p % 16] = -big * (3 + 37 * p % 101)
    # (places 0 and 101 have the same key: half the weight each)
    at = torch.nonzero(37 * j[:L - n + 1] % 101 == 0).flatten().tolist()
    assert at == [0, 101]
    q = torch.full((n, 2 * D), big, dtype=BF, device="cuda")
    got = m.paged_attention(q, cache, step.batch(m))
    want = (sum(cache.v[int(step.table[0, p // 16]), 0, p % 16].float() for p in at) / 2).to(BF)
    assert torch.equal(got[0, :D], want) and torch.equal(got[0, D:], want)
    assert bool(torch.isfinite(got.float()).all())
