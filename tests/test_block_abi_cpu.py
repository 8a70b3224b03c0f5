"""Refusals of the block operators, on the host: the C ABI validates its
arguments before anything is enqueued, the binding checks every tensor before
it hands out a pointer (no GPU is touched by these cases)."""
import os

import pytest
import torch

import w8a8_int8_expert_amd as m

FAKE, FAR = 0x100000, 1 << 40   # never dereferenced; FAR overlaps nothing near FAKE
OK, INV, UNS, WS = (m.MOE_W8A8_OK, m.MOE_W8A8_ERR_INVALID, m.MOE_W8A8_ERR_UNSUPPORTED,
                    m.MOE_W8A8_ERR_WORKSPACE)
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(m.LIB_PATH):
        from w8a8_int8_expert_amd import build
        build.build()
    return m.load_library()


def weights(K=300, N=70, fmt=0, gated=0, w=FAKE, scale=FAKE, inv=None, bias=None):
    return m.moe_w8a8_linear_weights(K, N, fmt, gated, w, scale, inv, bias)


def act(x=FAKE, ld=300, q=None, s=None):
    return m.moe_w8a8_act(x, ld, q, s)


def result(out=FAR, ld=70, t=0, gate=None, add=None, ld_add=70):
    return m.moe_w8a8_result(out, ld, t, gate, add, ld_add)


def linear(w=None, a=None, T=4, r=None, ws=2 * FAR, n=1 << 40):
    return m.moe_w8a8_linear(w or weights(), a or act(), T, r or result(), ws, n, stream=0)


def test_sizes():
    assert [m.moe_w8a8_row_pitch(k) for k in (1, 128, 129, 65536)] == [128, 128, 256, 65536]
    assert [m.moe_w8a8_row_pitch(k) for k in (0, -1, 65537)] == [0, 0, 0]
    assert m.moe_w8a8_linear_scales(17) == 32 and m.moe_w8a8_linear_scales(66, 1) == 128
    assert m.moe_w8a8_linear_scales(0) == 0 and m.moe_w8a8_linear_scales(65, 1) == 0
    assert m.moe_w8a8_linear_codes_bytes(17, 129) == 32 * 256
    assert m.moe_w8a8_linear_codes_bytes(66, 129, 1) == 128 * 256
    assert m.moe_w8a8_linear_codes_bytes(17, 0) == 0
    assert m.moe_w8a8_linear_codes_bytes((1 << 20) + 1, 1) == 0
    assert m.moe_w8a8_linear_codes_bytes(1 << 20, 65536) == 1 << 36
    for f in (lambda T: m.moe_w8a8_linear_workspace_size(1000, 4096, T),
              lambda T: m.moe_w8a8_ffn_workspace_size(4096, 1000, 70, T)):
        sizes = [f(T) for T in list(range(0, 600)) + [1023, 1024, 1025, 4096, 100000]]
        assert sizes[0] == 0 and all(b >= a for a, b in zip(sizes, sizes[1:])) and sizes[8] > 0
        assert f(-1) == 0 and f(1 << 22) == 0 and f((1 << 22) - 1) > 0
    assert m.moe_w8a8_linear_workspace_size(0, 1, 1) == 0
    assert m.moe_w8a8_ffn_workspace_size(1, 65537, 1, 1) == 0


def test_linear_refusals():
    assert linear(T=-1) == INV and linear(T=1 << 22) == INV and linear(T=(1 << 63) - 1) == INV
    for w in (weights(K=0), weights(N=-1), weights(fmt=2), weights(gated=1), weights(gated=2),
              weights(w=None), weights(scale=None), weights(w=FAKE + 8), weights(scale=FAKE + 2),
              weights(inv=FAKE + 1), weights(bias=FAKE + 2)):
        assert linear(w=w) == INV
    assert linear(w=weights(K=65537), a=act(ld=65537)) == UNS
    assert linear(w=weights(N=(1 << 20) + 1), r=result(ld=1 << 21)) == UNS
    for a in (act(x=None), act(x=FAKE + 1), act(ld=299), act(ld=(1 << 26) + 1),
              act(q=FAKE, s=FAKE), act(x=None, q=FAKE), act(x=None, s=FAKE),
              act(x=None, q=FAKE + 8, s=FAKE), act(x=None, q=FAKE, s=FAKE + 2)):
        assert linear(a=a) == INV
    for r in (result(out=None), result(out=FAR + 1), result(t=2), result(out=FAR + 2, t=1),
              result(ld=69), result(gate=FAKE + 1), result(add=FAKE + 1),
              result(add=FAKE, ld_add=69), result(add=FAR, ld_add=71),   # over out, another pitch
              result(add=FAR, t=1),                                     # over an fp32 out
              result(add=FAR + 2), result(out=FAKE + 64),               # over add, over x
              result(gate=FAR + 8)):                                    # the gate inside out
        assert linear(r=r) == INV
    need = m.moe_w8a8_linear_workspace_size(70, 300, 50)
    assert linear(T=50, ws=None) == WS and linear(T=50, n=need - 1) == WS
    assert linear(T=50, ws=2 * FAR + 128) == INV
    assert linear(T=0, a=m.moe_w8a8_act(), r=m.moe_w8a8_result(), ws=None, n=0) == OK
    assert linear(w=weights(K=0), T=0) == INV


def test_ffn_refusals():
    gu, dn = weights(K=300, N=64, gated=1), weights(K=32, N=70)

    def ffn(g=gu, d=dn, a=None, T=4, r=None, ws=2 * FAR, n=1 << 40):
        return m.moe_w8a8_ffn(g, d, a or act(), T, r or result(), ws, n, stream=0)
    assert ffn(T=-1) == INV
    assert ffn(g=weights(K=300, N=64)) == INV                 # not gated
    assert ffn(g=weights(K=300, N=63, gated=1)) == INV        # odd
    assert ffn(g=weights(K=300, N=64, gated=1, bias=FAKE)) == INV
    assert ffn(g=weights(K=300, N=66, gated=1)) == INV        # F differs
    assert ffn(d=weights(K=32, N=70, fmt=1)) == INV           # formats differ
    assert ffn(d=weights(K=32, N=70, inv=FAKE)) == INV
    assert ffn(d=weights(K=32, N=70, gated=1)) == INV
    assert ffn(a=act(ld=299)) == INV and ffn(r=result(ld=69)) == INV
    assert ffn(ws=None) == WS
    assert ffn(n=m.moe_w8a8_ffn_workspace_size(300, 32, 70, 4) - 1) == WS
    assert ffn(T=0, a=m.moe_w8a8_act(), r=m.moe_w8a8_result(), ws=None, n=0) == OK


def test_weight_refusals():
    def quantise(w=None, src=FAR, t=1, ld=300, sm=None):
        return m.moe_w8a8_linear_quantise(w or weights(), src, t, ld, sm, stream=0)
    assert quantise(w=weights(w=None)) == INV and quantise(src=None) == INV
    assert quantise(t=2) == INV and quantise(src=FAR + 2) == INV and quantise(ld=299) == INV
    assert quantise(src=FAR + 1, t=0) == INV and quantise(sm=FAKE + 2) == INV
    assert quantise(w=weights(K=65537), ld=65537) == UNS

    def pack(w=None, src=FAR, ld=300, s=2 * FAR):
        return m.moe_w8a8_linear_pack(w or weights(), src, ld, s, stream=0)
    assert pack(src=None) == INV and pack(s=None) == INV and pack(s=2 * FAR + 2) == INV
    assert pack(ld=299) == INV and pack(src=FAKE) == INV and pack(s=FAKE) == INV


def test_act_quant_refusals():
    def aq(K=300, fmt=0, x=FAKE, ld=300, T=4, inv=None, q=FAR, s=2 * FAR):
        return m.moe_w8a8_act_quant(K, fmt, x, ld, T, inv, q, s, stream=0)
    for kw in (dict(K=0), dict(fmt=2), dict(x=None), dict(x=FAKE + 1), dict(ld=299), dict(T=-1),
               dict(T=1 << 22), dict(inv=FAKE + 2), dict(q=None), dict(s=None), dict(q=FAR + 8),
               dict(s=2 * FAR + 2), dict(q=FAKE), dict(s=FAKE + 4), dict(s=FAR + 4)):
        assert aq(**kw) == INV, kw
    assert aq(K=65537, ld=65537) == UNS
    assert aq(T=0, x=None, q=None, s=None) == OK


def test_add_norm_refusals():
    def an(T=4, **kw):
        a = m.moe_w8a8_add_norm_args()
        base = dict(hidden=300, pre_norm=1, post_norm=0, eps=1e-6, residual_scale=1.0,
                    block_scale=1.0, y=FAKE, ld_y=300, normed=FAR, ld_normed=300)
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return m.moe_w8a8_add_norm(a, T, stream=0)
    for kw in (dict(T=-1), dict(T=1 << 22), dict(hidden=0), dict(pre_norm=3), dict(post_norm=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(residual_scale=float("inf")), dict(block_scale=float("nan")),
               dict(residual_type=2), dict(format=2), dict(y=None), dict(y=FAKE + 1),
               dict(ld_y=299), dict(normed=None), dict(normed=FAR + 1), dict(ld_normed=299),
               dict(pre_norm=0, pre_weight=FAKE), dict(post_weight=FAKE), dict(post_bias=FAKE),
               dict(q=3 * FAR), dict(s=3 * FAR), dict(q=3 * FAR + 8, s=4 * FAR),
               dict(q=3 * FAR, s=4 * FAR + 2), dict(residual=2 * FAR, ld_residual=299),
               dict(residual=2 * FAR + 2, ld_residual=300, residual_type=1),
               dict(residual_out=2 * FAR + 1, ld_residual_out=300),
               dict(gate_token=FAKE + 1), dict(gate_token=3 * FAR, gate_rows=2 * FAR, ld_gate=300,
                                               gate_group=1),
               dict(gate_rows=2 * FAR, ld_gate=300, gate_group=0),
               dict(gate_rows=2 * FAR, ld_gate=299, gate_group=1), dict(inv_smooth=FAKE + 2),
               # overlaps the header does not allow
               dict(normed=FAKE + 2), dict(normed=FAKE, ld_normed=301),
               dict(residual=FAR, ld_residual=300),
               dict(residual_out=FAR, ld_residual_out=300),
               dict(residual=2 * FAR, ld_residual=300, residual_out=2 * FAR, ld_residual_out=302),
               dict(q=FAR, s=4 * FAR), dict(q=3 * FAR, s=3 * FAR + 16),
               dict(gate_rows=FAR, ld_gate=300, gate_group=4),
               dict(pre_weight=FAR + 4)):
        assert an(**kw) == INV, kw
    assert an(hidden=65537, ld_y=65537, ld_normed=65537) == UNS
    assert an(T=0, y=None, normed=None) == OK


def test_binding_refusals():
    """CPU tensors on CPU-placed operators: every case is refused before the
    library is called."""
    lin = m.W8A8Linear(70, 30, device="cpu")
    ffn = m.W8A8FFN(70, 30, device="cpu")
    T = 5
    x = torch.zeros(T, 70, dtype=BF)
    q, s = torch.zeros(T, 128, dtype=torch.int8), torch.zeros(T)
    for op, N in ((lin, 30), (ffn, 70)):
        for kw in (dict(), dict(x=x, codes=(q, s)), dict(x=x.float()), dict(x=x[:, :69]),
                   dict(x=x.t()), dict(x=x[0]), dict(x=x[:1].expand(T, 70)),
                   dict(codes=(q[:, :70], s)), dict(codes=(q, s[:4])), dict(codes=(q, None)),
                   dict(codes=(q.float(), s)), dict(codes=(q, s.double())),
                   dict(x=x, out=torch.zeros(T, N)[:4]), dict(x=x, out=torch.zeros(T, N).double()),
                   dict(x=x, out=torch.zeros(T, N), out_dtype=BF),
                   dict(x=x, add=torch.zeros(T, N)), dict(x=x, add=torch.zeros(T, N + 1, dtype=BF)),
                   dict(x=x, gate=torch.zeros(T + 1)), dict(x=x, gate=torch.zeros(T, dtype=BF)),
                   dict(x=x, out_dtype=torch.float16)):
            with pytest.raises(m.MoEW8A8Error):
                op.forward(**kw)
        with pytest.raises(m.MoEW8A8Error, match="GPU"):   # nothing else is wrong
            op.forward(x)
    with pytest.raises(m.MoEW8A8Error):
        lin.load_quantized(torch.zeros(30, 69, dtype=torch.int8), torch.zeros(30))
    with pytest.raises(m.MoEW8A8Error):
        lin.load_quantized(torch.zeros(30, 70), torch.zeros(30))
    with pytest.raises(m.MoEW8A8Error):
        lin.quantise(torch.zeros(30, 70, dtype=torch.float16))
    for shape in ((0, 1), (1, 0), (65537, 1), (1, (1 << 20) + 1)):
        with pytest.raises(m.MoEW8A8Error):
            m.W8A8Linear(*shape, device="cpu")
    with pytest.raises(m.MoEW8A8Error):
        m.act_quant(x.float())
    with pytest.raises(m.MoEW8A8Error):
        m.act_quant(x, torch.zeros(71))
    w = torch.ones(70)
    for kw in (dict(y=x.float()), dict(y=x[0]), dict(residual=x[:4]), dict(residual=x.double()),
               dict(norm="l2"), dict(post_norm="x"), dict(weight=w[:69]), dict(weight=w.to(BF)),
               dict(bias=w[:1]), dict(codes="int4"), dict(gate=torch.zeros(3)),
               dict(gate=torch.zeros(T, 70)), dict(gate=torch.zeros(0, 70, dtype=BF)),
               dict(gate=torch.zeros(2, 70, dtype=BF), gate_group=2), dict(gate=w.to(BF)),
               dict(gate=torch.zeros(2, 70, dtype=BF), gate_group=0), dict(normed=x[:4]),
               dict(residual=x, residual_out=torch.zeros(T, 70)), dict(codes="int8",
                                                                      inv_smooth=w[:3])):
        with pytest.raises(m.MoEW8A8Error):
            m.add_norm(**{"y": x, **kw})


def test_header_from_c(tmp_path):
    """The block operators' declarations link from a C99 program, which gets the
    sizes the binding gets and the refusal of a NULL argument."""
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    libdir = os.path.dirname(m.LIB_PATH)
    src = tmp_path / "client.c"
    src.write_text(
        "#include <stdio.h>\n#include \"moe_w8a8.h\"\n"
        "int main(void) {\n"
        "  printf(\"%lld %zu %lld %zu %zu\\n\", (long long)moe_w8a8_row_pitch(300),\n"
        "         moe_w8a8_linear_codes_bytes(70, 300, 1),\n"
        "         (long long)moe_w8a8_linear_scales(70, 1),\n"
        "         moe_w8a8_linear_workspace_size(70, 300, 90),\n"
        "         moe_w8a8_ffn_workspace_size(300, 35, 70, 90));\n"
        "  printf(\"%d %d %d %d %d %d\\n\", moe_w8a8_linear_quantise(0, 0, 0, 0, 0, 0),\n"
        "         moe_w8a8_linear_pack(0, 0, 0, 0, 0),\n"
        "         moe_w8a8_act_quant(8, 0, 0, 8, 1, 0, 0, 0, 0),\n"
        "         moe_w8a8_linear(0, 0, 1, 0, 0, 0, 0),\n"
        "         moe_w8a8_ffn(0, 0, 0, 1, 0, 0, 0, 0), moe_w8a8_add_norm(0, 1, 0));\n"
        "  return 0;\n}\n")
    exe = tmp_path / "client"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I", os.path.join(root, "include"), str(src), "-L", libdir, "-lmoe_w8a8",
                    "-Wl,-rpath," + libdir, "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60)
    sizes, codes = r.stdout.splitlines()
    assert [int(v) for v in sizes.split()] == [
        384, m.moe_w8a8_linear_codes_bytes(70, 300, 1), m.moe_w8a8_linear_scales(70, 1),
        m.moe_w8a8_linear_workspace_size(70, 300, 90), m.moe_w8a8_ffn_workspace_size(300, 35, 70, 90)]
    assert [int(v) for v in codes.split()] == [INV] * 6


def test_codes_of_the_other_format_are_refused():
    """INT8 token codes given to an FP8 product would be read as e4m3 bytes."""
    T = 5
    s = torch.zeros(T)
    i8 = torch.zeros(T, 128, dtype=torch.int8)
    for fp8 in (False, True):
        right, wrong = (i8.view(torch.float8_e4m3fn), i8) if fp8 else \
            (i8, i8.view(torch.float8_e4m3fn))
        for op in (m.W8A8Linear(70, 30, device="cpu", fp8=fp8),
                   m.W8A8FFN(70, 30, device="cpu", fp8=fp8)):
            with pytest.raises(m.MoEW8A8Error, match="codes must be"):
                op.forward(codes=(wrong, s))
            with pytest.raises(m.MoEW8A8Error, match="GPU"):   # nothing else is wrong
                op.forward(codes=(right, s))


def test_weight_sources_over_their_destination_are_refused():
    """Filling a weight matrix reads its source twice and in another order than it
    writes: no source may share a byte with the codes or the scales filled."""
    N, K = 70, 300
    w = weights(w=FAR, scale=2 * FAR)
    codes, scales = m.moe_w8a8_linear_codes_bytes(N, K), 4 * m.moe_w8a8_linear_scales(N)
    for t, size in ((0, 2), (1, 4)):
        span = N * K * size
        for src in (FAR, FAR + codes - size, FAR - span + size, 2 * FAR, 2 * FAR + scales - size,
                    2 * FAR - span + size):
            assert m.moe_w8a8_linear_quantise(w, src, t, K, None, stream=0) == INV
    for sm in (FAR, FAR + codes - 4, 2 * FAR - K * 4 + 4):
        assert m.moe_w8a8_linear_quantise(w, 3 * FAR, 1, K, sm, stream=0) == INV
    for src in (FAR, FAR + codes - 1, 2 * FAR - N * K + 1, 2 * FAR + scales - 1):
        assert m.moe_w8a8_linear_pack(w, src, K, 3 * FAR, stream=0) == INV
    for s in (FAR, FAR + codes - 4, 2 * FAR + scales - 4):
        assert m.moe_w8a8_linear_pack(w, 3 * FAR, K, s, stream=0) == INV


def test_results_over_the_weights_are_refused():
    """A result that shares a byte with a buffer of the weights would change the
    weights while other blocks still read them."""
    N, K = 70, 300
    codes, scales = m.moe_w8a8_linear_codes_bytes(N, K), 4 * m.moe_w8a8_linear_scales(N)
    at = [(8 + i) * FAR for i in range(4)]
    w = weights(w=at[0], scale=at[1], inv=at[2], bias=at[3])
    ends = [(at[0], codes), (at[1], scales), (at[2], 4 * K), (at[3], 4 * N)]
    out_bytes = 4 * N * 2                                   # T = 4 rows of bf16
    for p, size in ends:
        for o in (p, p + size - 2, p - out_bytes + 2):
            assert linear(w=w, r=result(out=o)) == INV
    gu, dn = weights(K=K, N=64, gated=1), weights(K=32, N=N, w=at[0], scale=at[1], bias=at[3])
    gu2 = weights(K=K, N=64, gated=1, w=at[0], scale=at[1], inv=at[2])
    plain = weights(K=32, N=N)
    for g, d, ps in ((gu, dn, (at[0], at[1], at[3])), (gu2, plain, (at[0], at[1], at[2]))):
        for p in ps:
            assert m.moe_w8a8_ffn(g, d, act(), 4, result(out=p), 2 * FAR, 1 << 40, stream=0) == INV
    for q, s in ((FAR, 2 * FAR), (FAR - 4 * 384 + 16, 2 * FAR), (3 * FAR, FAR + 4 * K - 4)):
        assert m.moe_w8a8_act_quant(K, 0, FAKE, K, 4, FAR, q, s, stream=0) == INV


def far_rows(rows, width, dtype=torch.float32):
    """A matrix whose rows lie further apart than the library takes (a view of a
    storage that is never touched)."""
    store = torch.empty(0, dtype=dtype, device="meta")
    return store.new_empty((1,)).as_strided((rows, width), ((1 << 26) + 1, 1))


def test_every_operand_is_checked_before_weights_change(monkeypatch):
    """A pitch past the library's limit is refused with the other checks, before a
    call that loads two matrices has filled the first."""
    from w8a8_int8_expert_amd import block
    called = []
    monkeypatch.setattr(block, "_call", lambda name, *a, **k: called.append(name))
    H, F, N = 64, 32, 5
    meta = torch.device("meta")
    lin, ffn = m.W8A8Linear(H, N, device=meta), m.W8A8FFN(H, F, device=meta, out_features=N)
    z = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device=meta)  # noqa: E731
    i8 = torch.int8
    for call in (lambda: lin.quantise(far_rows(N, H)),
                 lambda: lin.load_quantized(far_rows(N, H, i8), z(N)),
                 lambda: ffn.quantise(z(2 * F, H), far_rows(N, F)),
                 lambda: ffn.quantise(far_rows(2 * F, H), z(N, F)),
                 lambda: ffn.load_quantized(z(2 * F, H, d=i8), z(2 * F), far_rows(N, F, i8), z(N)),
                 lambda: lin(far_rows(3, H, BF)),
                 lambda: ffn(z(3, H, d=BF), out=far_rows(3, N, BF)),
                 lambda: m.add_norm(z(3, H, d=BF), far_rows(3, H, BF))):
        with pytest.raises(m.MoEW8A8Error, match="too far apart"):
            call()
        assert not called
    ffn.quantise(z(2 * F, H), z(N, F))
    assert called == ["moe_w8a8_linear_quantise"] * 2


def test_gate_group_of_any_size(monkeypatch):
    """The group that reaches the library needs no more gate rows than there are,
    whatever number was given: one past 64 bits does not wrap to a small one."""
    from w8a8_int8_expert_amd import block
    seen = []
    monkeypatch.setattr(block, "_call", lambda name, dev, a, T, **k: seen.append(a._obj.gate_group))
    T = 5
    y, gate = torch.zeros(T, 70, dtype=BF), torch.zeros(1, 70, dtype=BF)
    for group in (None, T, T + 1, 1 << 40, (1 << 64) + 1, (1 << 65) + 2):
        m.add_norm(y, gate=gate, gate_group=group)
        assert -(-T // seen[-1]) == 1, group
