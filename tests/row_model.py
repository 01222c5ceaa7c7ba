"""Plain 64-bit forms of the rotary, 8-bit row cache and read-back operators,
and the error bounds that the tests of their kernels use.

Bounds count roundings: one is off by at most eps / 2 of the value (bf16 2^-8,
fp16 2^-11, fp32 2^-24, E4M3 2^-4).
"""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---- rotary ---------------------------------------------------------------
def rotate(x, positions, inv_freq, interleaved, att=1.0):
    """x [T, heads, D] rotated in fp64."""
    R = 2 * inv_freq.numel()
    a = positions.double()[:, None, None] * inv_freq.double()
    c, s = a.cos() * att, a.sin() * att
    x = x.double()
    y = x.clone()
    i = torch.arange(R // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def rotate_slack(x, inv_freq, interleaved, att=1.0):
    """fp32 error of a rotation: cos and sin are off by at most 2^-21 (the
    fraction's rounding, 2 pi 2^-26, and a few ulp of sincospi), the products
    and the sum by 2^-23 more of (|x| + |y|)."""
    ones = rotate(x.double().abs(), torch.zeros(x.shape[0], device=x.device), inv_freq, interleaved)
    R = 2 * inv_freq.numel()
    i = torch.arange(R // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    both = ones[..., first] + ones[..., second]
    slack = torch.zeros_like(ones)
    slack[..., first] = both
    slack[..., second] = both
    return slack * abs(att) * 2.0 ** -20


# ---- row quantisation -----------------------------------------------------
def quantise(x):
    """Rows [..., D] -> (E4M3 code bytes, scale bytes), from the definition."""
    x = x.double()
    amax = x.abs().amax(-1)
    nan = x.isnan().any(-1)
    e = torch.full_like(amax, 60.0)
    for k in range(59, -61, -1):                 # the smallest k with amax <= 448 * 2^k
        e = torch.where(amax <= 448.0 * 2.0 ** k, torch.full_like(e, k), e)
    y = (x * torch.pow(2.0, -e)[..., None]).clamp(-448.0, 448.0)
    codes = y.float().to(torch.float8_e4m3fn).view(torch.uint8)   # (y is exact in fp32 wherever it rounds to a code > 0)
    codes = torch.where(nan[..., None], torch.full_like(codes, 0x7f), codes)
    b = torch.where(nan, torch.full_like(e, 255.0), e + 127.0).to(torch.uint8)
    return codes, b


def value(codes, b):
    """fp64 values of code bytes [..., D] with scale bytes [...]."""
    p = torch.pow(2.0, b.double() - 127.0)
    p = torch.where(b == 255, torch.full_like(p, math.nan), p)
    return codes.view(torch.float8_e4m3fn).double() * p[..., None]


def codes_of(cache, bs, D):
    """Views of a row cache [NB, Hkv, bs * (D + 1)]: codes [NB, Hkv, bs, D], scales [NB, Hkv, bs]."""
    return cache[..., :bs * D].unflatten(2, (bs, D)), cache[..., bs * D:]


def put(cache, bs, D, blk, off, x):
    """Rows x [n, Hkv, D] into (blk, off) of a row cache."""
    c, s = codes_of(cache, bs, D)
    codes, b = quantise(x)
    c[blk, :, off] = codes
    s[blk, :, off] = b


def pages(lens, bs, gen, spare=2, device="cuda"):
    """A block table (unused entries -1) over a pool in random order."""
    n = [-(-L // bs) for L in lens]
    order = torch.randperm(sum(n) + spare, generator=gen)
    width = max(max(n), 1)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, k in enumerate(n):
        tables[s, :k] = order[at:at + k].to(torch.int32)
        at += k
    return tables.to(device), sum(n) + spare


def fill_rows(cache, bs, D, tables, lens, x):
    """x: one [L, Hkv, D] per sequence, into its pages."""
    for s, L in enumerate(lens):
        if L:
            t = torch.arange(L, device=cache.device)
            put(cache, bs, D, tables[s, t // bs].long(), t % bs, x[s])


def sequence(cache, bs, D, tables, s, L):
    """fp64 rows [L, Hkv, D] of sequence s."""
    t = torch.arange(L, device=cache.device)
    c, b = codes_of(cache, bs, D)
    blk = tables[s, t // bs].long()
    return value(c[blk, :, t % bs], b[blk, :, t % bs])


# ---- attention ------------------------------------------------------------
def attend(q, K, V, scale):
    """q [n, H, D], the last n of L tokens; K, V [L, Hkv, D] fp64.  Returns the
    output and a bound of what rounding may change: `logit` the error of a
    logit that fp32 sums of D products allow (D 2^-24 of the sum of magnitudes,
    twice: the weight and the softmax sum), `top` the largest |V| of the head."""
    n, H, D = q.shape
    L, Hkv, _ = K.shape
    G = H // Hkv
    if L == 0:
        z = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        return z, z, z
    q = q.double().view(n, Hkv, G, D)
    z = torch.einsum("ngad,lgd->ngal", q, K) * scale
    mag = torch.einsum("ngad,lgd->ngal", q.abs(), K.abs()) * abs(scale)
    hidden = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)[:, None, None, :]
    z = z.masked_fill(hidden, -math.inf)
    o = torch.einsum("ngal,lgd->ngad", torch.softmax(z, -1), V).reshape(n, H, D)
    logit = (2 * D * 2.0 ** -24 * mag.masked_fill(hidden, 0.0).amax(-1)).reshape(n, H, 1).expand(n, H, D)
    top = V.abs().amax((0, 2))[None, :, None, None].expand(n, Hkv, G, D).reshape(n, H, D)
    return o, logit, top


def attention_bound(ref, logit, top, dtype, weight_dtype, L):
    """Rounding of the output; of each weight to weight_dtype; logit errors; the
    exponential (2^-20); and, for fp16 weights, their floor: a weight below
    2^-25 of the largest contribution is lost, L 2^-24 of the largest |V|."""
    w = 0.0 if weight_dtype is None else half_step(weight_dtype)
    floor = L * 2.0 ** -24 if weight_dtype == torch.float16 else 0.0
    return half_step(dtype) * ref.abs() + (w + logit + 2.0 ** -20 + floor) * top


def close(got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape
    assert torch.equal(got.isnan(), ref.isnan()), "NaNs in other places"
    ok = ref.isfinite()
    assert torch.equal(got[~ok & ~ref.isnan()], ref[~ok & ~ref.isnan()])
    err = (got - ref).abs()[ok]
    over = err > bound[ok]
    assert not over.any(), f"{int(over.sum())} of {over.numel()} off by up to {float((err / bound[ok].clamp(min=1e-300)).max()):.3g} bounds"
