"""Decode and chunk attention over 8-bit row caches, element by element: the bound
of an output is made of the contributions p_t |V_t| that it is the sum of, so one
that is lost, or weighed by another row's scale, shows wherever it is the largest
of its dim."""
import math

import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from test_gpu_row_cache import paged_rows

pytestmark = pytest.mark.gpu


def spread(lo, hi):
    return lambda x, g: x * torch.exp2(torch.randint(lo, hi + 1, x.shape[:2] + (1,), generator=g, device="cuda").float())


def own_dims(lo, hi):
    """Row t has its elements in the dims d = t (mod 8) alone, rows of very different scales."""
    def f(x, g):
        t, d = torch.arange(x.shape[0], device="cuda"), torch.arange(x.shape[2], device="cuda")
        return spread(lo, hi)(x, g) * ((d[None, :] - t[:, None]) % 8 == 0)[:, None, :]
    return f


def reference(q, K, codes, e, scale, dtype, weights, fp16_floor):
    """(output, bound) of q [n, H, D], the last n of L tokens; V = codes 2^e [L, Hkv, D] and [L, Hkv].
    Per contribution: the rounding of its weight, twice the error of a logit (its own
    and the sum's), and the exponentials' 2^-20.  fp16 weights are taken relative to
    the largest p 2^e of the head: half a step, 2^-25, of that an element."""
    n, H, D = q.shape
    L, Hkv, _ = K.shape
    q = q.double().view(n, Hkv, H // Hkv, D)
    hidden = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)[:, None, None, :]
    z = (torch.einsum("ngad,lgd->ngal", q, K) * scale).masked_fill(hidden, -math.inf)
    mag = torch.einsum("ngad,lgd->ngal", q.abs(), K.abs()).masked_fill(hidden, 0.0).amax(-1, keepdim=True) * abs(scale)
    p, V = torch.softmax(z, -1), codes * torch.pow(2.0, e)[..., None]
    out, parts = torch.einsum("ngal,lgd->ngad", p, V), torch.einsum("ngal,lgd->ngad", p, V.abs())
    w = 0.0 if weights is None else rm.half_step(weights)
    bound = rm.half_step(dtype) * out.abs() + parts * (w + 2 * D * 2.0 ** -24 * mag + 2.0 ** -20)
    if fp16_floor:
        top = (p * torch.pow(2.0, e).T[None, :, None, :]).amax(-1, keepdim=True)
        bound = bound + 2.0 ** -25 * top * codes.abs().sum(0)[None, :, None, :]
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25              # an output below 2^-14
    return out.reshape(n, H, D), bound.reshape(n, H, D)


def stored(cache, bs, D, bt, s, L):
    t = torch.arange(L, device="cuda")
    c, b = rm.codes_of(cache, bs, D)
    blk = bt[s, t // bs].long()
    return c[blk, :, t % bs].view(torch.float8_e4m3fn).double(), b[blk, :, t % bs].double() - 127.0


@pytest.mark.parametrize("dt,G,D,bs", [("f16", 1, 128, 16), ("f16", 8, 64, 32), ("bf16", 1, 64, 16), ("bf16", 4, 128, 32),
                                       ("bf16", 8, 128, 16), ("bf16", 20, 128, 16), ("f32", 1, 64, 16), ("f32", 8, 128, 32)])
@pytest.mark.parametrize("values", [spread, own_dims])
def test_decode(dt, G, D, bs, values):
    lens, dtype, wide = [5, 40, 300, 900], rm.DT[dt], 12 if dt == "f16" else 30
    kc, vc, bt, cl, gc = paged_rows(lens, 2 * G, 2, D, bs, dt, 95, kscale=spread(-10, 2), vscale=values(-wide, min(wide, 12)))
    q = torch.randn(4, 2 * G, D, generator=gc, device="cuda").to(dtype)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, D ** -0.5)
    for s, L in enumerate(lens):
        K = rm.sequence(kc, bs, D, bt, s, L)
        weights = None if dt == "f32" else dtype if G >= 17 else torch.float16
        rm.close(out[s:s + 1], *reference(q[s:s + 1], K, *stored(vc, bs, D, bt, s, L), D ** -0.5, dtype, weights,
                                          dt != "f32" and G < 17))
    assert pkv.read_device_errors() == 0


@pytest.mark.parametrize("G,D,bs", [(1, 128, 16), (8, 64, 32), (3, 128, 32)])
@pytest.mark.parametrize("values", [spread, own_dims])
def test_chunks(G, D, bs, values):
    lens, counts = [300, 50, 700], [200, 50, 130]
    kc, vc, bt, cl, gc = paged_rows(lens, 2 * G, 2, D, bs, "bf16", 96, kscale=spread(-10, 2), vscale=values(-30, 12))
    start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    q = torch.randn(sum(counts), 2 * G, D, generator=gc, device="cuda").bfloat16()
    out = torch.empty_like(q)
    pkv.paged_attention_prefill_fp8row(out, q, kc, vc, bt, cl, start, D ** -0.5, max_query_len=200)
    for s, (L, n) in enumerate(zip(lens, counts)):
        a = int(start[s])
        rm.close(out[a:a + n], *reference(q[a:a + n], rm.sequence(kc, bs, D, bt, s, L), *stored(vc, bs, D, bt, s, L),
                                          D ** -0.5, torch.bfloat16, torch.bfloat16, False))
    assert pkv.read_device_errors() == 0
