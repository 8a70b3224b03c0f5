"""What lies between a decoder block's QKV projection and its output projection,
and behind its LM head: what is measured.

Three operators:
  rope    norms of queries and keys for each head and the position rotation, in one
          pass over the QKV projection's rows; queries go to bf16 rows, keys and
          values into a paged cache (bf16, or INT8 / FP8 codes with a scale for
          each token and head);
  attend  attention of the batch's new tokens (chunks of a prefill, or one token for
          each sequence) over that cache: grouped heads, causal, optional window;
  answer  from LM-head logits: log probabilities of given tokens, the entropy of
          each row, and the top alternatives.

A cache is k, v [pages][kv heads][page size][D]; codes have scales fp32 [pages]
[kv heads][page size]. Sequence b's new tokens are rows cu[b] .. cu[b+1], the last
ones of its length[b]; place p of it lies in page table[b][p // page size]. Codes of
a key are decided in fp32: rint(fl(v * fl(qmax / max|v|))).
"""
import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"int8": 127.0, "fp8": 448.0}
SCORES = 32 * 8192 * 8192          # scores of the largest listed attention
CACHED = 8 * 65536 * 8 * 128       # cached elements of the largest listed one


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch of a block with 32 heads over 8: latency; FP8 cache
        dict(name="rope decode fp8", op="rope", B=32, q=1, kv=4096, ragged=3, Hq=32, Hkv=8, D=128,
             page=64, fmt="fp8", norm=True, rot=128, pairs=False),
        # ragged chunks at far places; 64-wide heads, half of each rotated, in pairs, no norm
        dict(name="rope odd partial", op="rope", B=7, q=701, kv=100003, ragged=5, Hq=14, Hkv=2,
             D=64, page=16, fmt="bf16", norm=False, rot=32, pairs=True),
        # a whole prefill of 32 x 512 tokens
        dict(name="rope prefill", op="rope", B=32, q=512, kv=512, ragged=0, Hq=32, Hkv=8, D=128,
             page=64, fmt="bf16", norm=True, rot=128, pairs=False),
        # one request's next token: latency
        dict(name="attend 1 token", op="attend", B=1, q=1, kv=1031, ragged=0, Hq=32, Hkv=8, D=128,
             page=64, fmt="bf16", causal=True, window=0),
        # a decode batch of 32 requests of mixed lengths, INT8 cache
        dict(name="attend decode int8", op="attend", B=32, q=1, kv=8192, ragged=11, Hq=32, Hkv=8,
             D=128, page=64, fmt="int8", causal=True, window=0),
        # long contexts, 64 heads over 8, FP8 cache: the most that is read
        dict(name="attend decode long", op="attend", B=8, q=1, kv=65536, ragged=0, Hq=64, Hkv=8,
             D=128, page=64, fmt="fp8", causal=True, window=0),
        # a chunk of one long prompt beside the decode steps of others
        dict(name="attend chunk mixed", op="attend", B=12, q=512, kv=16384, ragged=2, Hq=32, Hkv=8,
             D=128, page=32, fmt="bf16", causal=True, window=0),
        # ragged batch, seven heads share one, 64-wide, window, small pages, INT8
        dict(name="attend odd window", op="attend", B=9, q=613, kv=5003, ragged=7, Hq=28, Hkv=4,
             D=64, page=16, fmt="int8", causal=True, window=1000),
        # one prompt of 8192 tokens from its start: the largest product
        dict(name="attend prefill", op="attend", B=1, q=8192, kv=8192, ragged=0, Hq=32, Hkv=8,
             D=128, page=64, fmt="bf16", causal=True, window=0),
        # a decode step's fp32 logits of an odd vocabulary: sampled tokens and 20 alternatives
        dict(name="answer decode", op="answer", T=32, V=32003, dtype="fp32", top=20),
        # one token of a large vocabulary, bf16 logits with many ties
        dict(name="answer 1 token", op="answer", T=1, V=131072, dtype="bf16", top=5),
        # log probabilities of a whole prompt
        dict(name="answer prompt", op="answer", T=4096, V=32003, dtype="fp32", top=1),
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
    op = rng.choice(["rope", "attend", "attend", "attend", "answer"])
    if op == "answer":
        V = _size(rng, 512, 160000)
        return dict(op=op, T=max(1, min(_size(rng, 1, 4096), 4096 * 32003 // V)), V=V,
                    dtype=rng.choice(["fp32", "bf16"]), top=rng.choice([0, 1, 5, 20, 64]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    page, fmt = rng.choice([16, 32, 64, 128, 256]), rng.choice(["bf16", "int8", "fp8"])
    ragged = rng.choice([0, rng.randrange(1, 1000)])
    B, q = _size(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 8), _size(rng, 9, 4096)])
    if op == "rope":
        B = max(1, min(B, 16384 * 48 * 128 // (q * (Hq + 2 * Hkv) * D)))
        return dict(op=op, B=B, q=q, kv=q + _size(rng, 1, 100000), ragged=ragged, Hq=Hq, Hkv=Hkv,
                    D=D, page=page, fmt=fmt, norm=rng.random() < 0.6,
                    rot=rng.choice([D, D, D // 2, D // 4]), pairs=rng.random() < 0.4)
    kv = max(q, _size(rng, 16, 65536))
    while B > 1 and (B * kv * Hkv * D > CACHED // 2 or B * Hq * q * kv * D > SCORES * 64):
        B = max(1, B // 2)
    while Hq * q * kv * D > SCORES * 64 and q > 1:
        q = max(1, q // 2)
        kv = max(q, kv * 3 // 4)
    return dict(op=op, B=B, q=q, kv=kv, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, page=page, fmt=fmt,
                causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))


def _lengths(case):
    """(new tokens, whole length) of each sequence. ragged 0: all alike; else the
    first is the longest chunk, the second the longest context, and now and then a
    sequence has nothing new."""
    c = case
    if not c["ragged"]:
        return [(c["q"], c["kv"])] * c["B"]
    r, got = random.Random(c["ragged"]), []
    for b in range(c["B"]):
        n = c["q"] if b == 0 else 0 if b > 1 and r.random() < 0.1 else _log(r, 1, c["q"])
        ctx = c["kv"] - c["q"]
        got.append((n, n + (ctx if b == 1 else int(ctx * r.random() ** 1.5))))
    return got


# -------------------------------------------------------------------- inputs
def _cached(g, shape, fmt):
    """Cached keys or values as a cache holds them: (elements, scales or None)."""
    x = torch.randn(shape, generator=g, device=DEV)
    if fmt == "bf16":
        return x.bfloat16(), None
    s = torch.exp(0.2 * torch.randn(shape[:-1], generator=g, device=DEV))
    if fmt == "int8":
        return x.mul_(38).round_().clamp_(-127, 127).to(torch.int8), s.mul_(1 / 38)
    return x.mul_(110).clamp_(-448, 448).to(torch.float8_e4m3fn), s.mul_(1 / 110)


def _inputs(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "answer":
        T, V = c["T"], c["V"]
        x = torch.randn(T, V, generator=g, device=DEV)
        x *= 1 + 3 * torch.rand(T, 1, generator=g, device=DEV)  # flat rows and peaked ones
        s["logits"] = x.to(torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)
        s["tokens"] = torch.randint(0, V, (T,), generator=g, device=DEV)
        return s
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    lens = _lengths(c)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    s["T"], s["most"], s["longest"] = cu[-1], max(n for n, _ in lens), max(t for _, t in lens)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s["lengths"] = torch.tensor([t for _, t in lens], dtype=torch.int32, device=DEV)
    # the pages lie anywhere in the cache; of a batch whose keys are only written, the
    # pages of the new tokens are there and the others are not
    first = [(t - n) // page if c["op"] == "rope" else 0 for n, t in lens]
    need = [-(-t // page) - f if t else 0 for (_, t), f in zip(lens, first)]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
    width = -(-s["longest"] // page)
    rows, at = [], 0
    for f, n in zip(first, need):
        rows.append([-1] * f + order[at:at + n] + [-1] * (width - f - n))
        at += n
    s["table"] = torch.tensor(rows, dtype=torch.int32, device=DEV)
    s["k"], s["ks"] = _cached(g, (pages, Hkv, page, D), c["fmt"])
    s["v"], s["vs"] = _cached(g, (pages, Hkv, page, D), c["fmt"])
    if c["op"] == "attend":
        s["q"] = (1.5 * torch.randn(s["T"], Hq * D, generator=g, device=DEV)).bfloat16()
        return s
    x = torch.randn(s["T"], (Hq + 2 * Hkv) * D, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(s["T"], 1, generator=g, device=DEV))
    s["qkv"] = x.bfloat16()
    s["qw"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if c["norm"] else None
    s["kw"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if c["norm"] else None
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV)
    s["freq"] = 1e6 ** (-i / c["rot"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] != "answer":
        # the cache's handle and the step's batch, which a program makes once and
        # takes through every block
        import w8a8_int8_expert_amd as m
        s["cache"] = m.KVCache.of(s["k"], s["v"], s["ks"], s["vs"])
        s["batch"] = m.SequenceBatch(s["cu"], s["lengths"], s["table"], s["most"], s["longest"])
    return s


# --------------------------------------------------------- the framework's own
def _run_own(s):
    import w8a8_int8_expert_amd as m
    c = s["case"]
    if c["op"] == "answer":
        r = m.token_logprobs(s["logits"], s["tokens"], top=c["top"])
        out = {"logprobs": r.logprobs, "entropy": r.entropy}
        if c["top"]:
            out["top_tokens"], out["top_logprobs"] = r.top_tokens, r.top_logprobs
        return out
    if c["op"] == "attend":
        return m.paged_attention(s["q"], s["cache"], s["batch"], causal=c["causal"],
                                 window=c["window"])
    q = m.qk_norm_rope(s["qkv"], s["cache"], s["batch"], c["Hq"], norm=c["norm"],
                       q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, inv_freq=s["freq"],
                       interleaved=c["pairs"])
    return _written(s, q)


def _written(s, q):
    """The queries and the whole cache after the call; INT8 codes as the numbers they
    stand for (e4m3 codes are numbers already)."""
    out = {"q": q}
    for n in ("k", "v"):
        out[n] = s[n].bfloat16() if s["case"]["fmt"] == "int8" else s[n]
        if s[n + "s"] is not None:
            out[n + "_scale"] = s[n + "s"]
    return out


# ---------------------------------------------------------------- plain forms
def _places(s):
    """Of each new token: its sequence, and its place in it."""
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"].long()[b + 1] + s["lengths"].long()[b]


def _codes(v, fmt):
    """Codes (as fp32 numbers) and scales of fp32 rows along the last axis."""
    a = v.abs().amax(-1, keepdim=True)
    top = torch.full_like(a, QMAX[fmt])  # a tensor: a quotient with a number is not a division here
    rr = torch.where(a > 0, top / a, torch.zeros_like(a))
    p = (v * rr).clamp(-QMAX[fmt], QMAX[fmt])
    return p.round() if fmt == "int8" else p.to(torch.float8_e4m3fn).float(), (a / top)[..., 0]


def _rope(s):
    c = s["case"]
    T, Hq, Hkv, D, R = s["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    qk, v = x[:, :Hq + Hkv], x[:, Hq + Hkv:]
    if c["norm"]:
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-6)
        qk = torch.cat([qk[:, :Hq] * s["qw"], qk[:, Hq:] * s["kw"]], 1)
    b, place = _places(s)
    angle = place.double()[:, None] * s["freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["pairs"]:
        x0, x1 = qk[..., 0:R:2], qk[..., 1:R:2]
    else:
        x0, x1 = qk[..., :R // 2], qk[..., R // 2:R]
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    turned = torch.stack([y0, y1], -1).flatten(2) if c["pairs"] else torch.cat([y0, y1], -1)
    qk = torch.cat([turned, qk[..., R:]], -1)
    page = s["table"][b, place // c["page"]].long()
    at = place % c["page"]
    _put(s["k"], s["ks"], page, at, qk[:, Hq:], c["fmt"])
    _put(s["v"], s["vs"], page, at, v, c["fmt"])
    return _written(s, qk[:, :Hq].bfloat16().view(T, Hq * D))


def _put(to, scales, page, at, x, fmt):
    if fmt == "bf16":
        to[page, :, at] = x.bfloat16()
        return
    codes, scale = _codes(x, fmt)
    scales[page, :, at] = scale
    codes = codes.to(torch.int8) if fmt == "int8" else codes.to(torch.float8_e4m3fn).view(torch.int8)
    to.view(torch.int8)[page, :, at] = codes


def _dense(x, scales, table, page):
    """Cached rows of every sequence, [B][kv heads][places][D] in fp32."""
    at = table.clamp_min(0).long()
    y = x.view(torch.int8)[at].view(x.dtype).float() if x.dtype == torch.float8_e4m3fn \
        else x[at].float()
    if scales is not None:
        y = y * scales[at][..., None]
    B, P, H, _, D = y.shape
    return y.transpose(1, 2).reshape(B, H, P * page, D)


def _attend(s):
    c = s["case"]
    Hq, Hkv, D, N, T = c["Hq"], c["Hkv"], c["D"], s["most"], s["T"]
    B, G = c["B"], Hq // Hkv
    k = _dense(s["k"], s["ks"], s["table"], c["page"])
    v = _dense(s["v"], s["vs"], s["table"], c["page"])
    cu, length = s["cu"].long(), s["lengths"].long()
    i = torch.arange(N, device=DEV)
    row = (cu[:-1, None] + i).clamp_max(T - 1)               # [B][N]
    q = s["q"].float()[row].view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).view(B, Hkv, G, N, -1)
    scores *= 1 / math.sqrt(D)
    key = torch.arange(scores.shape[-1], device=DEV)
    place = (length - (cu[1:] - cu[:-1]))[:, None] + i       # [B][N]
    seen = (key < length[:, None, None]).expand(B, N, -1)
    if c["causal"]:
        seen = seen & (key <= place[:, :, None])
    if c["window"]:
        seen = seen & (key > place[:, :, None] - c["window"])
    seen = seen[:, None, None]
    scores = torch.where(seen, scores, torch.full((), -math.inf, device=DEV))
    scores -= scores.amax(-1, keepdim=True).clamp_min(-1e30)
    p = scores.exp_()
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros((), device=DEV))
    o = torch.matmul(p.view(B, Hkv, G * N, -1), v).view(B, Hkv, G, N, D)
    b, place = _places(s)
    n = torch.arange(T, device=DEV) - cu[b]
    return o.permute(0, 3, 1, 2, 4)[b, n].reshape(T, Hq * D).bfloat16()


def _answer(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    log = total.log()
    out = {"logprobs": ((x.gather(1, s["tokens"][:, None]) - top) - log)[:, 0],
           "entropy": (log - (e * (x - top)).sum(1, keepdim=True) / total)[:, 0]}
    if c["top"]:
        best, at = torch.sort(x, dim=1, descending=True, stable=True)  # ties: lowest index first
        out["top_tokens"] = at[:, :c["top"]].contiguous()
        out["top_logprobs"] = (best[:, :c["top"]] - top) - log
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _rope(state) if op == "rope" else _attend(state) if op == "attend" else _answer(state)


# ------------------------------------------------------------------ 64 bits
def _decided(v, fmt):
    """Codes of rows whose values are fp32 numbers, decided in fp32."""
    v = v.to(torch.float32)
    big = torch.maximum(v.max(-1).values, -v.min(-1).values)
    step = torch.div(torch.full_like(big, QMAX[fmt]), big)
    step[big == 0] = 0
    q = torch.mul(v, step.unsqueeze(-1)).clamp(-QMAX[fmt], QMAX[fmt])
    q = torch.round(q) if fmt == "int8" else q.to(torch.float8_e4m3fn)
    return q.to(torch.float64), big.to(torch.float64) / QMAX[fmt]


def _exact_rope(case, s):
    c, F = case, torch.float64
    Hq, Hkv, D, R = c["Hq"], c["Hkv"], c["D"], c["rot"]
    out = {"q": torch.empty(s["T"], Hq * D, dtype=F, device=DEV)}
    for n in ("k", "v"):
        out[n] = s[n].to(torch.float32).to(F)
        if s[n + "s"] is not None:
            out[n + "_scale"] = s[n + "s"].to(F)

    def turned(x, w, place):
        x = x.to(F)
        if c["norm"]:
            x = x / torch.sqrt(torch.mean(x * x, dim=-1, keepdim=True) + 1e-6) * w.to(F)
        a = torch.outer(place.to(F), s["freq"]).unsqueeze(1)
        z = torch.complex(torch.cos(a), torch.sin(a))
        head, tail = x[..., :R], x[..., R:]
        if c["pairs"]:
            w2 = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * z
            head = torch.view_as_real(w2).reshape(head.shape)
        else:
            lo, hi = head.chunk(2, dim=-1)
            w2 = torch.complex(lo.contiguous(), hi.contiguous()) * z
            head = torch.cat((w2.real, w2.imag), dim=-1)
        return torch.cat((head, tail), dim=-1)

    row = 0
    for b, (n, length) in enumerate(_lengths(c)):
        if n == 0:
            continue
        x = s["qkv"][row:row + n].reshape(n, Hq + 2 * Hkv, D)
        place = torch.arange(length - n, length, device=DEV)
        out["q"][row:row + n] = turned(x[:, :Hq], s["qw"], place).reshape(n, -1)
        for name, y in (("k", turned(x[:, Hq:Hq + Hkv], s["kw"], place)), ("v", x[:, Hq + Hkv:])):
            page, at = s["table"][b].long()[place // c["page"]], place % c["page"]
            y = y.to(F)
            if c["fmt"] != "bf16":
                y, scale = _decided(y, c["fmt"])
                out[name + "_scale"][page, :, at] = scale
            out[name][page, :, at] = y
        row += n
    return out


def _exact_attend(case, s):
    c, F = case, torch.float64
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.zeros(s["T"], Hq, D, dtype=F, device=DEV)
    row = 0
    for b, (n, length) in enumerate(_lengths(c)):
        if n == 0 or length == 0:
            continue
        pages = s["table"][b][:-(-length // c["page"])].long().tolist()
        for h in range(Hkv):
            def cached(x, scale):
                y = torch.cat([x[p, h] for p in pages])[:length].to(torch.float32).to(F)
                if scale is not None:
                    y = y * torch.cat([scale[p, h] for p in pages])[:length].to(F).unsqueeze(1)
                return y
            k, v = cached(s["k"], s["ks"]), cached(s["v"], s["vs"])
            key = torch.arange(length, device=DEV)
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                x = s["q"][row + i:row + i + m].view(m, Hq, D)[:, h * G:(h + 1) * G].to(F)
                z = torch.matmul(x.reshape(m * G, D), k.t()).view(m, G, length) / math.sqrt(D)
                place = (length - n + i + torch.arange(m, device=DEV)).view(m, 1, 1)
                gone = torch.zeros(m, 1, length, dtype=torch.bool, device=DEV)
                if c["causal"]:
                    gone = gone | (key > place)
                if c["window"]:
                    gone = gone | (key <= place - c["window"])
                z = torch.softmax(z.masked_fill(gone, -math.inf), dim=-1)
                z = torch.nan_to_num(z, nan=0.0)  # (a row that sees nothing)
                out[row + i:row + i + m, h * G:(h + 1) * G] = torch.matmul(
                    z.view(m * G, length), v).view(m, G, D)
        row += n
    return out.view(s["T"], Hq * D)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    logits, F = s["logits"], torch.float64
    T, top = logits.shape[0], case["top"]
    out = {"logprobs": torch.empty(T, dtype=F, device=DEV),
           "entropy": torch.empty(T, dtype=F, device=DEV)}
    if top:
        out["top_tokens"] = None
        out["top_logprobs"] = torch.empty(T, top, dtype=F, device=DEV)
    for i in range(0, T, 512):
        lp = torch.log_softmax(logits[i:i + 512].to(F), dim=1)
        out["logprobs"][i:i + 512] = lp[torch.arange(lp.shape[0]), s["tokens"][i:i + 512]]
        out["entropy"][i:i + 512] = -(torch.exp(lp) * lp).sum(1)
        if top:
            out["top_logprobs"][i:i + 512] = torch.topk(lp, top, dim=1).values
    return out


# --------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "answer":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["T"] * (c["V"] * size + 16 + 12 * c["top"]),
                "flops": 5 * c["T"] * c["V"]}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    row = (2 * D if c["fmt"] == "bf16" else D + 4) * 2 * Hkv  # a token's keys and values
    lens = _lengths(c)
    T = sum(n for n, _ in lens)
    if c["op"] == "rope":
        return {"bytes": T * ((2 * Hq + 2 * Hkv) * D * 2 + row),
                "flops": T * (Hq + 2 * Hkv) * D * 8}
    pairs = keys = 0
    for n, length in lens:
        if n == 0:
            continue
        start, w = length - n, c["window"] or length + n
        if c["causal"]:   # token i sees min(start + i + 1, window) keys
            full = max(0, min(n, w - start))        # tokens whose window is not full yet
            pairs += full * start + full * (full + 1) // 2 + (n - full) * w
        else:
            pairs += sum(length - max(0, start + i + 1 - w) for i in range(n))
        keys += min(length, n - 1 + w)
    return {"bytes": keys * row + T * Hq * D * 4, "flops": 4 * pairs * Hq * D}
