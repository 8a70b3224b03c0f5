"""Refusals of qk_norm_rope, paged_attention and token_logprobs, on the host: the C ABI
validates its arguments before anything is enqueued, the binding checks every tensor
before it hands out a pointer (no GPU is touched by these cases)."""
import os

import pytest
import torch

import w8a8_int8_expert_amd as m

FAKE = 0x10000000   # never dereferenced
OK, INV, UNS, WS = (m.MOE_W8A8_OK, m.MOE_W8A8_ERR_INVALID, m.MOE_W8A8_ERR_UNSUPPORTED,
                    m.MOE_W8A8_ERR_WORKSPACE)
BF, F32, F64, I8, I32, I64, E4 = (torch.bfloat16, torch.float32, torch.float64, torch.int8,
                                  torch.int32, torch.int64, torch.float8_e4m3fn)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(m.LIB_PATH):
        from w8a8_int8_expert_amd import build
        build.build()
    return m.load_library()


def far(i):  # places that overlap nothing
    return FAKE + (i << 44)


def cache(pages=8, page=64, heads=2, D=128, fmt=0, k=far(1), v=far(2), stride=None, ks=far(3),
          vs=far(4), sstride=None):
    return m.moe_w8a8_kv_cache(pages, page, heads, D, fmt, k, v,
                               page * heads * D if stride is None else stride, ks, vs,
                               page * heads if sstride is None else sstride)


def batch(n=3, most=4, longest=500, width=8, cu=far(5), lengths=far(6), table=far(7), ld=8):
    return m.moe_w8a8_batch(n, most, longest, width, cu, lengths, table, ld)


def rope(heads=4, norm=1, rotary=128, pairs=0, eps=1e-6, qkv=far(8), ld=1024, q=far(9), ld_q=512,
         qw=far(10), kw=far(11), freq=far(12), pos=None, c=None, b=None, T=0):
    a = m.moe_w8a8_qk_norm_rope_args(heads, norm, rotary, pairs, eps, qkv, ld, q, ld_q, qw, kw, freq,
                                     pos)
    return m.moe_w8a8_qk_norm_rope(a, c or cache(), b or batch(), T, stream=0)


def attend(heads=4, causal=1, window=0, scale=0.1, q=far(8), ld_q=512, out=far(9), ld_o=512, c=None,
           b=None, T=5, ws=far(13), n=0):
    a = m.moe_w8a8_attention_args(heads, causal, window, scale, q, ld_q, out, ld_o)
    return m.moe_w8a8_paged_attention(a, c or cache(), b or batch(), T, ws, n, stream=0)


def answer(V=100, t=1, top=3, x=far(1), ld=100, tok=far(2), lp=far(3), ent=far(4), tt=far(5),
           tl=far(6), T=0, ws=None, n=0):
    a = m.moe_w8a8_logprobs_args(V, t, top, x, ld, tok, lp, ent, tt, tl)
    return m.moe_w8a8_token_logprobs(a, T, ws, n, stream=0)


def test_empty_calls():
    assert rope() == OK and rope(T=3, b=batch(n=0)) == OK and rope(qkv=None, q=None) == OK
    assert attend(T=0) == OK and attend(b=batch(n=0)) == OK and attend(b=batch(most=0)) == OK
    assert answer() == OK and answer(x=None, tok=None, lp=None, tt=None, tl=None) == OK


@pytest.mark.parametrize("call", [rope, attend])
def test_caches_that_are_refused(call):
    kw = dict(T=4)
    if call is attend:
        kw["n"] = 1 << 60
    bad = [(INV, dict(pages=0)), (INV, dict(heads=0)), (INV, dict(fmt=3)), (INV, dict(k=None)),
           (INV, dict(v=None)), (INV, dict(k=far(1) + 8)), (INV, dict(stride=64 * 256 - 16)),
           (INV, dict(stride=64 * 256 + 8)), (INV, dict(stride=1 << 41)), (INV, dict(ks=None)),
           (INV, dict(vs=far(4) + 4)), (INV, dict(sstride=64)), (INV, dict(sstride=130)),
           (INV, dict(fmt=2)), (UNS, dict(D=96)), (UNS, dict(D=512)), (UNS, dict(page=8)),
           (UNS, dict(page=48)), (UNS, dict(page=512)), (UNS, dict(heads=1025)), (INV, dict(D=0)),
           (INV, dict(page=0))]
    for code, c in bad:
        assert call(c=cache(**c), **kw) == code, c
    bad = [dict(n=-1), dict(most=-1), dict(longest=-1), dict(width=-1), dict(cu=None),
           dict(lengths=None), dict(table=None), dict(cu=far(5) + 2), dict(lengths=far(6) + 1),
           dict(table=far(7) + 2), dict(ld=7), dict(ld=(1 << 26) + 1)]
    for b in bad:
        assert call(b=batch(**b), **kw) == INV, b
    assert call(b=batch(n=(1 << 20) + 1), **kw) == UNS
    for T in (-1, 1 << 22):
        assert call(**{**kw, "T": T}) == INV


def test_rope_refusals():
    bad = [(INV, dict(heads=0)), (INV, dict(rotary=-16)), (INV, dict(eps=-1.0)),
           (INV, dict(eps=float("nan"))), (INV, dict(norm=0)), (INV, dict(qkv=None)),
           (INV, dict(q=None)), (INV, dict(qkv=far(8) + 1)), (INV, dict(ld=1023)),
           (INV, dict(ld_q=511)), (INV, dict(freq=None)), (INV, dict(freq=far(12) + 4)),
           (INV, dict(pos=far(14) + 4)), (INV, dict(qw=far(10) + 2)), (UNS, dict(rotary=8)),
           (UNS, dict(rotary=144)), (UNS, dict(heads=513, ld=1 << 20, ld_q=1 << 20)),
           (INV, dict(ld=(1 << 26) + 1)),
           # results over inputs, the cache and the batch's arrays
           (INV, dict(q=far(8) + 2)), (INV, dict(q=far(10))), (INV, dict(q=far(1))),
           (INV, dict(q=far(3))), (INV, dict(q=far(7))), (INV, dict(qkv=far(2))),
           (INV, dict(kw=far(4))), (INV, dict(pos=far(2) + 16)), (INV, dict(freq=far(1)))]
    for code, kw in bad:
        assert rope(T=4, **kw) == code, kw
    assert rope(T=4, c=cache(v=far(1))) == INV
    assert rope(T=4, c=cache(vs=far(3) + 16)) == INV
    assert rope(T=4, b=batch(lengths=far(2))) == INV
    assert rope(T=4, b=batch(table=far(4))) == INV


def test_attention_refusals():
    n = 1 << 60
    bad = [(INV, dict(window=-1)), (INV, dict(scale=float("inf"))), (INV, dict(heads=0)),
           (UNS, dict(heads=5)), (UNS, dict(heads=514)), (INV, dict(q=None)), (INV, dict(out=None)),
           (INV, dict(q=far(8) + 1)), (INV, dict(ld_q=511)), (INV, dict(ld_o=511)),
           (INV, dict(out=far(8))), (INV, dict(out=far(1) + 256)), (INV, dict(out=far(4))),
           (INV, dict(out=far(6))), (INV, dict(ws=far(13) + 16)), (INV, dict(ws=far(9))),
           (INV, dict(ws=far(2)))]
    for code, kw in bad:
        assert attend(n=n, **kw) == code, kw
    # many rows over a long context: partial results need room
    b = batch(n=1, most=1, longest=1 << 16, width=1 << 10, ld=1 << 10)
    need = m.moe_w8a8_paged_attention_workspace_size(cache(), b, 4, 1)
    assert need > 0 and need % 256 == 0
    assert attend(b=b, T=1, ws=None, n=0) == WS and attend(b=b, T=1, n=need - 256) == WS
    size = m.moe_w8a8_paged_attention_workspace_size
    assert size(cache(D=96), b, 4, 1) == 0 and size(cache(), b, 5, 1) == 0
    assert size(cache(), b, 4, 1 << 22) == 0 and size(cache(), b, 4, 0) == 0


def test_logprob_refusals():
    bad = [(INV, dict(V=0)), (INV, dict(top=-1)), (INV, dict(top=101)), (INV, dict(t=2)),
           (UNS, dict(V=(1 << 20) + 1, ld=1 << 21)), (UNS, dict(top=65)), (INV, dict(x=None)),
           (INV, dict(x=far(1) + 2)), (INV, dict(ld=99)), (INV, dict(tok=None)),
           (INV, dict(lp=None)), (INV, dict(tt=None)), (INV, dict(tl=None)), (INV, dict(top=0)),
           (INV, dict(tok=far(2) + 4)), (INV, dict(ent=far(4) + 2)), (INV, dict(tt=far(5) + 4)),
           (INV, dict(lp=far(1))), (INV, dict(tl=far(2))), (INV, dict(ent=far(3))),
           (INV, dict(tok=None, lp=None, ent=None, tt=None, tl=None, top=0))]
    for code, kw in bad:
        assert answer(T=4, **kw) == code, kw
    for T in (-1, 1 << 22):
        assert answer(T=T) == INV


def refuses(f, *a, **kw):
    with pytest.raises(m.MoEW8A8Error):
        f(*a, **kw)


def cpu_cache(fmt=I8, pages=4, heads=2, page=16, D=64):
    k = torch.zeros(pages, heads, page, D, dtype=fmt)
    s = None if fmt == BF else torch.zeros(pages, heads, page)
    return m.KVCache.of(k, k.clone(), s, None if s is None else s.clone())


def cpu_batch(B=2, most=3, longest=40, width=4):
    z = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    return m.SequenceBatch(z(B + 1), z(B), z(B, width), most, longest)


def test_binding_caches():
    k = torch.zeros(4, 2, 16, 64, dtype=I8)
    s = torch.zeros(4, 2, 16)
    for a in ((k.float(), k, s, s), (k[0], k[0], s, s), (k, k.view(torch.uint8), s, s), (k, k[:3], s, s),
              (k, k, None, s), (k, k, s, s.double()), (k, k, s, s[:, :1]), (k.to(BF), k.to(BF), s, s),
              (k.transpose(1, 2), k.transpose(1, 2), s, s), (k, [k], s, s)):
        refuses(m.KVCache.of, *a)
    for shape in ((4, 2, 16, 96), (4, 2, 24, 64), (4, 2, 8, 64), (4, 1025, 16, 64), (0, 2, 16, 64)):
        z = torch.zeros(shape, dtype=BF)
        refuses(m.KVCache.of, z, z)
    b = torch.zeros(4, 2, 16, 64, dtype=BF)
    big = torch.zeros(4, 2 * 16 * 64 + 8, dtype=BF)
    refuses(m.KVCache.of, big[:, :2048].view(4, 2, 16, 64), b)      # pages 8 elements further apart
    shifted = torch.zeros(4 * 2048 + 4, dtype=BF)[4:].view(4, 2, 16, 64)
    refuses(m.KVCache.of, shifted, shifted)
    layers = torch.zeros(4, 3, 2, 16, 64, dtype=BF)
    c = m.KVCache.of(layers[:, 1], layers[:, 2])
    assert c.struct.page_stride == 3 * 2048 and c.num_pages == 4
    refuses(m.KVCache.of, layers[:, 1], b)
    refuses(m.KVCache, 4, 16, 2, 64, format="fp16", device="cpu")
    refuses(m.KVCache, 0, 16, 2, 64, device="cpu")
    c = m.KVCache(4, 16, 2, 64, format="fp8", device="cpu")
    assert c.k.dtype == E4 and c.k_scale.shape == (4, 2, 16) and c.page_size == 16


def test_binding_batches():
    z = lambda *s, t=I32: torch.zeros(*s, dtype=t)  # noqa: E731
    for a in ((z(3), z(2), z(2, 4), -1, 9), (z(3), z(2), z(2, 4), 1, 1 << 31), (z(2), z(2), z(2, 4), 1, 9),
              (z(3), z(3), z(2, 4), 1, 9), (z(3, t=I64), z(2), z(2, 4), 1, 9), (z(3), z(2), z(2), 1, 9),
              (z(3), z(2, t=F32), z(2, 4), 1, 9), (z(6)[::2], z(2), z(2, 4), 1, 9),
              (z(3), z(2), z(4, 2).t(), 1, 9), (z(3), z(2), z(1, 4).expand(2, 4), 1, 9),
              ([0, 1], z(1), z(1, 4), 1, 9)):
        refuses(m.SequenceBatch, *a)
    m.SequenceBatch(z(3), z(2), z(2, 9)[:, :4], 1, 9)
    m.SequenceBatch(z(1), z(0), z(0, 4), 0, 0)


def test_binding_rope():
    c, b = cpu_cache(), cpu_batch()
    x = torch.zeros(3, 8 * 64, dtype=BF)
    f = torch.zeros(32, dtype=F64)
    w = torch.ones(64)
    r = m.qk_norm_rope
    refuses(r, x.float(), c, b, 4)
    refuses(r, x, c, b, 5)
    refuses(r, x, c, b, 0)
    refuses(r, x, None, b, 4)
    refuses(r, x, c, (1, 2), 4)
    refuses(r, x[0], c, b, 4)
    refuses(r, x, c, b, 4, q_weight=w)
    refuses(r, x, c, b, 4, norm=True, q_weight=w[:32])
    refuses(r, x, c, b, 4, norm=True, k_weight=w.double())
    refuses(r, x, c, b, 4, inv_freq=f.float())
    refuses(r, x, c, b, 4, inv_freq=f[:4])
    refuses(r, x, c, b, 4, inv_freq=torch.zeros(40, dtype=F64))
    refuses(r, x, c, b, 4, inv_freq=f, positions=torch.zeros(2, dtype=I64))
    refuses(r, x, c, b, 4, inv_freq=f, positions=torch.zeros(3, dtype=I32))
    refuses(r, x, c, b, 4, out=torch.zeros(3, 5 * 64, dtype=BF))
    refuses(r, x, c, b, 4, inv_freq=f)  # all in order, but not on a GPU


def test_binding_attention():
    c, b = cpu_cache(), cpu_batch()
    q = torch.zeros(3, 4 * 64, dtype=BF)
    a = m.paged_attention
    refuses(a, q.float(), c, b)
    refuses(a, q[:, :3 * 64], c, b)
    refuses(a, q[:, :100], c, b)
    refuses(a, q[:, :0], c, b)
    refuses(a, q, c, b, window=-1)
    refuses(a, q, c, b, window=1 << 31)
    refuses(a, q, c, b, out=torch.zeros(2, 4 * 64, dtype=BF))
    refuses(a, q, c, b, out=torch.zeros(3, 4 * 64))
    refuses(a, q, b, c)
    refuses(a, q[0], c, b)
    refuses(a, q, c, b)


def test_binding_logprobs():
    x, t = torch.zeros(3, 50), torch.zeros(3, dtype=I64)
    f = m.token_logprobs
    refuses(f, x.double(), t)
    refuses(f, x[0], t)
    refuses(f, x, t[:2])
    refuses(f, x, t.int())
    refuses(f, x, t, top=51)
    refuses(f, x, t, top=-1)
    refuses(f, torch.zeros(3, 100), t, top=65)
    refuses(f, x, entropy=False)
    refuses(f, x[:, :0], t)
    refuses(f, x.t(), None)
    refuses(f, x, t)
