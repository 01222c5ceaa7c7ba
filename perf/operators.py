"""The quantised-cache serving operators, as they are measured.

Five operators that follow each other in a serving step over a paged cache of
8-bit rows: the rotary positions of q and k, the cache write that quantises
each (token, KV head) row with a power-of-two scale of its own, the attention
of single tokens and of chunks of new tokens over that cache, and the read of
whole sequences back out of it.

A case is a dict of plain values; its sequence lengths come from its own
"lens_seed", so the work of a case is known without its inputs.  A cache of
8-bit rows ("fp8row") is uint8 [num_blocks][num_kv_heads][bs * (D + 1)]: bs
rows of D E4M3 codes, then the bs rows' scale bytes b, each standing for
2^(b - 127); a cached element is code * 2^(b - 127).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # rotary positions of one decode step of a 13B-shaped layer: 64 sequences, small and latency-bound
        dict(name="rotary step f16", op="rotary", dtype="f16", tokens=64, heads=40, kv_heads=40, head=128,
             rot=128, interleaved=False, far=2048),
        # the same for the packed prompts of a 7B-shaped layer, half of each head rotated, neighbouring pairs
        dict(name="rotary prompts bf16", op="rotary", dtype="bf16", tokens=21569, heads=32, kv_heads=32, head=128,
             rot=64, interleaved=True, far=131072),
        # quantising write alone, no positions: one step of the tiny fp32 shape
        dict(name="write step f32", op="write", dtype="f32", tokens=4, heads=0, kv_heads=4, head=64, block=16,
             rot=0, interleaved=False, far=0),
        # rotary and quantising write of one decode step: 256 sequences, 32 heads
        dict(name="rotary write step bf16", op="write", dtype="bf16", tokens=256, heads=32, kv_heads=32, head=128,
             block=16, rot=128, interleaved=False, far=4096),
        # the same for 16 chunks of 512 tokens with 64 query heads over 8 KV heads
        dict(name="rotary write chunks f16", op="write", dtype="f16", tokens=8192, heads=64, kv_heads=8, head=128,
             block=32, rot=128, interleaved=True, far=131072),
        # a few short sequences read back (a prefix handed on)
        dict(name="read short bf16", op="read", dtype="bf16", seqs=7, lo=1, hi=300, lens_seed=11, kv_heads=2, head=64,
             block=16),
        # the caches of a 13B-shaped batch read back
        dict(name="read batch f16", op="read", dtype="f16", seqs=64, lo=256, hi=2048, lens_seed=12, kv_heads=40,
             head=128, block=16),
        # decode of one short sequence in fp32: latency
        dict(name="decode one f32", op="decode", dtype="f32", seqs=1, lo=33, hi=33, lens_seed=13, heads=4, kv_heads=4,
             head=64, block=16),
        # decode of a 13B-shaped batch, one query head per KV head
        dict(name="decode batch f16", op="decode", dtype="f16", seqs=64, lo=256, hi=2048, lens_seed=14, heads=40,
             kv_heads=40, head=128, block=16),
        # decode of long contexts, 8 query heads per KV head
        dict(name="decode long bf16", op="decode", dtype="bf16", seqs=16, lo=16384, hi=32768, lens_seed=15, heads=64,
             kv_heads=8, head=128, block=16),
        # whole prompts of different lengths
        dict(name="prompts f16", op="prefill", dtype="f16", seqs=8, lo=100, hi=1000, qlo=0, qhi=0, lens_seed=16, heads=16,
             kv_heads=16, head=64, block=16),
        # chunks of 512 new tokens over long contexts, 8 query heads per KV head
        dict(name="chunks bf16", op="prefill", dtype="bf16", seqs=8, lo=2048, hi=8192, qlo=512, qhi=512, lens_seed=17,
             heads=64, kv_heads=8, head=128, block=16),
    ]


def _log(rng, lo, hi):
    """A whole number, evenly spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "decode", "prefill"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    c = dict(op=op, dtype=dtype, head=rng.choice([64, 128]))
    group = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    kv = _log(rng, 1, max(1, 40 // group))
    if op == "rotary":
        c["head"] = rng.choice([64, 80, 96, 128, 256])
        per = (kv * group + kv) * c["head"] * BYTES[dtype]
        c.update(tokens=_log(rng, 1, max(2, min(40000, 350_000_000 // per))), heads=kv * group, kv_heads=kv,
                 rot=rng.choice([c["head"], c["head"] // 2, 2 * rng.randint(1, c["head"] // 2)]),
                 interleaved=rng.random() < 0.5, far=_log(rng, 16, 1 << 20))
        return c
    c["block"] = rng.choice([16, 32])
    if op == "write":
        rot = rng.choice([0, c["head"], c["head"], c["head"] // 2, 2 * rng.randint(1, c["head"] // 2)])
        c.update(tokens=_log(rng, 1, max(2, min(20000, 300_000_000 // ((group + 2) * kv * c["head"] * BYTES[dtype])))),
                 heads=kv * group if rot else 0, kv_heads=kv, rot=rot, interleaved=rng.random() < 0.5,
                 far=_log(rng, 16, 1 << 20))
        return c
    c["lens_seed"] = rng.randrange(1 << 30)
    c["kv_heads"] = kv
    if op == "read":
        hi = _log(rng, 1, 4096)
        c.update(seqs=_log(rng, 1, max(1, min(256, 300_000_000 // (hi * kv * c["head"])))), hi=hi, lo=rng.randint(0, hi))
        return c
    c["heads"] = kv * group
    if op == "decode":
        hi = _log(rng, 1, 32768)
        c.update(seqs=_log(rng, 1, max(1, min(256, 400_000_000 // (hi * kv * c["head"])))), hi=hi, lo=rng.randint(0, hi))
        return c
    c["dtype"] = rng.choice(["f16", "bf16"])
    hi = _log(rng, 2, 8192)
    q = _log(rng, 1, min(hi, 1024))
    c.update(seqs=_log(rng, 1, max(1, min(16, 1_500_000_000 // (hi * q * c["heads"])))), hi=hi, lo=rng.randint(q, hi),
             qlo=rng.randint(1, q), qhi=q)
    if rng.random() < 0.3:
        c.update(qlo=0, qhi=0, hi=min(hi, 1500), lo=min(c["lo"], 1500))
        c["seqs"] = max(1, min(c["seqs"], 1_500_000_000 // (c["hi"] ** 2 * c["heads"])))
    return c


def _lens(case):
    r = random.Random(case["lens_seed"])
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    ctx[0] = max(ctx[0], 1)
    if case["op"] != "prefill":
        return ctx, None
    if case["qhi"] == 0:            # whole prompts
        return ctx, list(ctx)
    return ctx, [min(n, r.randint(case["qlo"], case["qhi"])) for n in ctx]


def work(case):
    op, D, es = case["op"], case["head"], BYTES[case["dtype"]]
    if op == "rotary":
        rows = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * rows * D * es + case["tokens"] * 8, "flops": 3 * rows * case["rot"]}
    if op == "write":
        q, kv = case["tokens"] * case["heads"], 2 * case["tokens"] * case["kv_heads"]
        return {"bytes": 2 * q * D * es + kv * (D * es + D + 1) + 16 * case["tokens"], "flops": 3 * q * case["rot"] + 4 * kv * D}
    ctx, qs = _lens(case)
    blocks = sum(-(-n // case["block"]) for n in ctx)
    rows = 2 * sum(ctx) * case["kv_heads"]
    if op == "read":
        return {"bytes": rows * (D + 1 + D * es) + 4 * blocks, "flops": rows * D}
    if op == "decode":
        return {"bytes": rows * (D + 1) + 4 * blocks + 2 * case["seqs"] * case["heads"] * D * es,
                "flops": 4 * D * sum(ctx) * case["heads"]}
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(ctx, qs))
    return {"bytes": rows * (D + 1) + 4 * blocks + 2 * sum(qs) * case["heads"] * D * es,
            "flops": 4 * D * pairs * case["heads"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _frequencies(rot, far):
    """Frequencies 10000^(-2i / rot) in fp32; for far positions the slow ones
    are divided by 8 (a context stretched eightfold), the fast ones kept."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / max(rot, 1))
    if far > 8192:
        turns = far / 8 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 8.0)
    return f.float().cuda()


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """Rows of fp32 -> (E4M3 codes, whole exponents): the smallest e in
    [-60, 60] with max|row| <= 448 * 2^e, codes round to nearest even."""
    m, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, ex - 9 + (m > 0.875).to(ex.dtype), torch.full_like(ex, -60)).clamp(-60, 60)
    codes = (x * _pow2(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, e


def _new_cache(case, blocks):
    return torch.zeros((blocks, case["kv_heads"], case["block"] * (case["head"] + 1)), dtype=torch.uint8, device="cuda")


def _codes(cache, case):
    return cache[:, :, :case["block"] * case["head"]].unflatten(2, (case["block"], case["head"]))


def _scales(cache, case):
    return cache[:, :, case["block"] * case["head"]:]


def _store(cache, case, x, blk, off):
    codes, e = _quantise(x.float())
    _codes(cache, case)[blk, :, off] = codes.view(torch.uint8)
    _scales(cache, case)[blk, :, off] = (e + 127).to(torch.uint8)


def _filled(case, x):
    """A cache that holds the values x [blocks, Hkv, bs, D]."""
    cache = _new_cache(case, x.shape[0])
    codes, e = _quantise(x)
    _codes(cache, case).copy_(codes.view(torch.uint8))
    _scales(cache, case).copy_(e + 127)
    return cache


def _paged(case, gen):
    """A block table over a pool in random order, both caches filled, and the lengths."""
    ctx, qs = _lens(case)
    bs = case["block"]
    L = torch.tensor(ctx, device="cuda")
    nblk = (L + bs - 1) // bs
    width = max(1, int(max(-(-n // bs) for n in ctx)))
    pool = int(sum(-(-n // bs) for n in ctx)) + 3
    owned = torch.arange(width, device="cuda")[None, :] < nblk[:, None]
    tables = torch.full(owned.shape, -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    tables[owned] = order[:int(owned.sum())]
    st = dict(case=case, tables=tables, lens=L.to(torch.int32), L=L, ctx=ctx, qs=qs)
    # channel-dependent spread for keys, smaller values for V, as projections give
    spread = torch.exp(0.5 * torch.randn(case["head"], generator=gen, device="cuda"))
    shape = pool, case["kv_heads"], bs, case["head"]
    st["k_cache"] = _filled(case, torch.randn(shape, generator=gen, device="cuda") * spread)
    st["v_cache"] = _filled(case, torch.randn(shape, generator=gen, device="cuda") * 0.5)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt, D = case["op"], DTYPES[case["dtype"]], case["head"]
    if op in ("rotary", "write"):
        T, H, Hkv = case["tokens"], case["heads"], case["kv_heads"]
        st = dict(case=case, freq=_frequencies(case["rot"], case["far"]))
        # one projection's output: q, k and v of a token side by side
        both = _randn(gen, (T, (H + 2 * Hkv) * D), dt)
        st["q"] = both[:, :H * D].view(T, H, D)
        st["k"] = both[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
        st["v"] = both[:, (H + Hkv) * D:].view(T, Hkv, D)
        st["pos"] = torch.randint(0, max(case["far"], 1), (T,), generator=gen, device="cuda")
        st["q_out"] = torch.empty((T, H, D), dtype=dt, device="cuda")
        if op == "rotary":
            st["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda")
            return st
        bs = case["block"]
        pool = -(-T // bs) + 2
        st["slots"] = torch.randperm(pool * bs, generator=gen, device="cuda")[:T].contiguous()
        st["k_cache"], st["v_cache"] = _new_cache(case, pool), _new_cache(case, pool)
        return st
    st = _paged(case, gen)
    S = case["seqs"]
    if op == "decode":
        st["q"] = _randn(gen, (S, case["heads"], D), dt)
        st["out"] = torch.empty_like(st["q"])
        return st
    counts = st["ctx"] if op == "read" else st["qs"]
    st["start"] = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    T = sum(counts)
    if op == "read":
        st["k_out"] = torch.empty((T, case["kv_heads"], D), dtype=dt, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
    else:
        st["q"] = _randn(gen, (T, case["heads"], D), dt)
        st["out"] = torch.empty_like(st["q"])
        st["most_q"] = max(counts)
    return st


# ---------------------------------------------------------------------------
# the operators: plain forms, and the framework's calls
# ---------------------------------------------------------------------------
def _rotated(x, pos, freq, rot, interleaved):
    """x [T, heads, D] in fp32 with its first `rot` dims rotated."""
    a = pos.double()[:, None] * freq.double()[None, :]
    cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    x = x.float()
    y = x.clone()
    if interleaved:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = u * cos - v * sin
        y[..., 1:rot:2] = v * cos + u * sin
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = u * cos - v * sin
        y[..., rot // 2:rot] = v * cos + u * sin
    return y


def _read(cache, case, blk, off):
    """Rows (blk, off) of a cache as fp32 [..., Hkv, D]."""
    codes = _codes(cache, case)[blk, :, off].view(torch.float8_e4m3fn).float()
    e = _scales(cache, case)[blk, :, off].to(torch.int32) - 127
    return codes * _pow2(e).unsqueeze(-1)


def _sequences(cache, st):
    """Every sequence's rows as fp32 [S, Hkv, width * bs, D] (rows past a length: whatever the pool holds)."""
    case = st["case"]
    blk = st["tables"].clamp(min=0).long()
    codes = _codes(cache, case)[blk].view(torch.float8_e4m3fn).float()
    codes *= _pow2(_scales(cache, case)[blk].to(torch.int32) - 127).unsqueeze(-1)
    return codes.transpose(1, 2).flatten(2, 3)


def _weights(z):
    """Softmax over the last axis; a row without a finite value has all weights zero."""
    z -= z.amax(-1, keepdim=True).clamp(min=-1e30)
    z.exp_()
    z /= z.sum(-1, keepdim=True).clamp(min=1e-30)
    return z


def _plain_rotary(st):
    c = st["case"]
    args = st["pos"], st["freq"], c["rot"], c["interleaved"]
    dt = st["q"].dtype
    return {"q": _rotated(st["q"], *args).to(dt), "k": _rotated(st["k"], *args).to(dt)}


def _plain_write(st):
    c = st["case"]
    args = st["pos"], st["freq"], c["rot"], c["interleaved"]
    k = _rotated(st["k"], *args) if c["rot"] else st["k"]
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    _store(st["k_cache"], c, k, blk, off)
    _store(st["v_cache"], c, st["v"], blk, off)
    return _written(st, _rotated(st["q"], *args).to(st["q"].dtype) if c["rot"] else None)


def _written(st, q):
    """The caches as the values their bytes stand for: codes and scales."""
    c = st["case"]
    return ({} if q is None else {"q": q}) | {
        "k_cache": _codes(st["k_cache"], c).view(torch.float8_e4m3fn),
        "k_cache_scales": _scales(st["k_cache"], c).view(torch.float8_e8m0fnu),
        "v_cache": _codes(st["v_cache"], c).view(torch.float8_e4m3fn),
        "v_cache_scales": _scales(st["v_cache"], c).view(torch.float8_e8m0fnu)}


def _plain_read(st):
    c = st["case"]
    at = torch.arange(st["k_out"].shape[0], device="cuda")
    s = torch.searchsorted(st["start"], at, right=True) - 1
    t = at - st["start"][s]
    blk = st["tables"][s, t // c["block"]].long()
    dt = DTYPES[c["dtype"]]
    return {n: _read(st[n + "_cache"], c, blk, t % c["block"]).to(dt) for n in ("k", "v")}


def _plain_decode(st):
    c = st["case"]
    S, H, D = st["q"].shape
    K, V = _sequences(st["k_cache"], st), _sequences(st["v_cache"], st)
    q = st["q"].float().view(S, c["kv_heads"], H // c["kv_heads"], D)
    z = torch.matmul(q, K.transpose(2, 3)) * D ** -0.5
    seen = torch.arange(z.shape[3], device="cuda")[None, :] < st["L"][:, None]
    z.masked_fill_(~seen[:, None, None, :], -math.inf)
    return torch.matmul(_weights(z), V).view(S, H, D).to(st["q"].dtype)


def _plain_prefill(st):
    c = st["case"]
    T, H, D = st["q"].shape
    S, Hkv, n = c["seqs"], c["kv_heads"], st["most_q"]
    start = st["start"].long()
    counts = start[1:] - start[:-1]
    at = torch.arange(T, device="cuda")
    s = torch.searchsorted(start, at, right=True) - 1
    i = at - start[s]
    q = torch.zeros((S, n, H, D), device="cuda")
    q[s, i] = st["q"].float()
    q = q.view(S, n, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)
    z = torch.matmul(q, _sequences(st["k_cache"], st).transpose(2, 3))
    z *= D ** -0.5
    keys = torch.arange(z.shape[3], device="cuda")
    last = (st["L"] - counts)[:, None] + torch.arange(n, device="cuda")[None, :]     # each query's position
    hidden = keys[None, None, :] > last[:, :, None]
    z.view(S, Hkv, H // Hkv, n, -1).masked_fill_(hidden[:, None, None], -math.inf)
    o = torch.matmul(_weights(z), _sequences(st["v_cache"], st)).view(S, Hkv, H // Hkv, n, D)
    return o.permute(0, 3, 1, 2, 4).reshape(S, n, H, D)[s, i].to(st["q"].dtype)


def _own(st):
    import paged_kv_cache_480_b200 as pkv
    c = st["case"]
    op, scale = c["op"], c["head"] ** -0.5
    if op == "rotary":
        pkv.rotary_embedding(st["q_out"], st["k_out"], st["q"], st["k"], st["pos"], st["freq"],
                             interleaved=c["interleaved"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "write":
        if not c["rot"]:
            pkv.reshape_and_cache_fp8row(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"])
            return _written(st, None)
        pkv.rotary_reshape_and_cache_fp8row(st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                            st["pos"], st["slots"], st["freq"], interleaved=c["interleaved"])
        return _written(st, st["q_out"])
    if op == "read":
        pkv.gather_cache_fp8row(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["tables"], st["start"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if op == "decode":
        return pkv.paged_attention_decode_fp8row(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                                 st["lens"], scale)
    return pkv.paged_attention_prefill_fp8row(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                              st["lens"], st["start"], scale, max_query_len=st["most_q"])


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "write": _plain_write, "read": _plain_read, "decode": _plain_decode,
            "prefill": _plain_prefill}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------
def _values(cache, case, blk):
    """Blocks `blk` of one cache as fp64 tokens [len(blk) * bs, Hkv, D]."""
    bs, D = case["block"], case["head"]
    raw = cache[blk.long()]
    n, Hkv = raw.shape[:2]
    codes = raw[..., :bs * D].reshape(n, Hkv, bs, D).to(torch.int64)
    e, m, sign = (codes >> 3) & 15, codes & 7, codes >> 7
    v = torch.where(e > 0, (8 + m).double() * torch.pow(2.0, (e - 10).double()), m.double() * 2.0 ** -9)
    v = torch.where(sign > 0, -v, v)
    p = torch.pow(2.0, raw[..., bs * D:].reshape(n, Hkv, bs, 1).double() - 127.0)
    return (v * p).transpose(1, 2).reshape(n * bs, Hkv, D)


def _turned(x, st):
    """x rotated in fp64, as a complex product."""
    c = st["case"]
    rot = c["rot"]
    x = x.double()
    a = st["pos"].double()[:, None, None] * st["freq"].double()
    w = torch.polar(torch.ones_like(a), a)
    pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
        x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    y = y.flatten(-2) if c["interleaved"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _e4m3(x):
    """fp64 values within +-448 rounded to the nearest E4M3 value, ties to even."""
    step = torch.pow(2.0, torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return {"q": _turned(st["q"], st), "k": _turned(st["k"], st)}
    if op == "write":
        out = {"q": _turned(st["q"], st)} if case["rot"] else {}
        bs = case["block"]
        for name, x in (("k_cache", st["k"]), ("v_cache", st["v"])):
            x = _turned(x, st) if case["rot"] and name == "k_cache" else x.double()
            e = torch.ceil(torch.log2(x.abs().amax(-1).clamp(min=1e-300) / 448.0)).clamp(-60.0, 60.0)
            p = torch.pow(2.0, e)
            pool, Hkv = st[name].shape[:2]
            codes = torch.zeros((pool, Hkv, bs, case["head"]), dtype=torch.float64, device="cuda")
            scales = torch.full((pool, Hkv, bs), 2.0 ** -127, dtype=torch.float64, device="cuda")
            blk, off = st["slots"] // bs, st["slots"] % bs
            codes[blk, :, off] = _e4m3(x / p[..., None])
            scales[blk, :, off] = p
            out[name], out[name + "_scales"] = codes, scales
        return out
    scale, D = case["head"] ** -0.5, case["head"]
    if op == "read":
        got = {"k": [], "v": []}
        for s, n in enumerate(st["ctx"]):
            blk = st["tables"][s, :-(-n // case["block"])]
            for name in got:
                got[name].append(_values(st[name + "_cache"], case, blk)[:n])
        return {name: torch.cat(v) for name, v in got.items()}
    H, Hkv = case["heads"], case["kv_heads"]
    counts = st["qs"] or [1] * case["seqs"]
    out, at = [], 0
    for s, (L, n) in enumerate(zip(st["ctx"], counts)):
        q = st["q"][at:at + n].double()
        at += n
        if L == 0:
            out.append(torch.zeros_like(q))
            continue
        blk = st["tables"][s, :-(-L // case["block"])]
        k = _values(st["k_cache"], case, blk)[:L]
        v = _values(st["v_cache"], case, blk)[:L]
        o = torch.empty_like(q)
        bias = torch.zeros((n, L), dtype=torch.float64, device="cuda")
        bias.masked_fill_(torch.ones_like(bias).triu(L - n + 1) > 0, -math.inf)
        for h in range(H):
            g = h * Hkv // H
            o[:, h] = torch.softmax(q[:, h] @ k[:, g].T * scale + bias, -1) @ v[:, g]
        out.append(o)
    return torch.cat(out)
