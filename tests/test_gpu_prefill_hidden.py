"""Chunk attention over E4M3 caches where K or V hold elements that q's type has
not: NaN, and with f16 q what lies beyond +-65504.  A query sees them from their
token on, none before it."""
import math

import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from test_gpu_rotary import gen_of
from test_gpu_row_cache import paged_rows

pytestmark = pytest.mark.gpu


def masked_reference(q, K, V, scale, dtype):
    """attend() with V's NaN and (f16) overflowing elements taken out, and put
    back where a query sees them: an infinity of either sign, NaN for both or a
    NaN.  K's overflowing elements count as +-65504."""
    n, H, D = q.shape
    L, Hkv, _ = V.shape
    most = 65504.0 if dtype == torch.float16 else math.inf
    K = torch.where(K.isnan(), K, K.clamp(-most, most))
    out_of = V.isnan() | (V.abs() > most)
    ref, logit, top = rm.attend(q, K, torch.where(out_of, torch.zeros_like(V), V), scale)
    ref = ref.view(n, Hkv, H // Hkv, D).clone()
    pos = torch.arange(L - n, L, device=V.device)

    def seen(at):                              # [n, Hkv, D]: a query sees one of these elements
        return (at.cumsum(0) > 0)[pos]
    up, down = seen(V.isnan() | (V > most)), seen(V.isnan() | (V < -most))
    for where, x in ((up & ~down, math.inf), (down & ~up, -math.inf), (up & down, math.nan)):
        ref[where[:, :, None, :].expand_as(ref) & ~ref.isnan()] = x
    return ref.view(n, H, D), logit, top


def check(name, lens, counts, H, D, bs, dt, kc, vc, bt, rows, q, scale, extra=()):
    dtype = rm.DT[dt]
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    getattr(pkv, name)(out, q, kc, vc, bt, cl, start, scale, *extra, max_query_len=max(counts))
    assert pkv.read_device_errors() == 0
    tiny = 2.0 ** -25 if dt == "f16" else 0.0
    for s, (L, n) in enumerate(zip(lens, counts)):
        if n == 0:
            continue
        a = int(start[s])
        K, V = (rows(c, s, L) for c in (kc, vc))
        ref, logit, top = masked_reference(q[a:a + n], K, V, scale, dtype)
        rm.close(out[a:a + n], ref, rm.attention_bound(ref, logit, top, dtype, dtype, L) + tiny)
    return out


@pytest.mark.parametrize("dt,G,D,bs", [("bf16", 1, 128, 16), ("f16", 1, 64, 32), ("bf16", 8, 64, 16), ("f16", 3, 128, 32),
                                       ("bf16", 100, 64, 16)])
def test_nan_rows_of_v(dt, G, D, bs):
    """First, last, in the middle of a tile, several of a sequence; some
    sequences without one between those that have them."""
    lens, counts = [300, 140, 129, 700, 5, 128, 33], [300, 140, 100, 257, 5, 1, 33]
    bad = {0: {130: [1], 299: [0, 1]}, 2: {0: [0], 128: [1]}, 3: {600: [0], 520: [0], 130: [1]}, 6: {32: [0]}}
    kc, vc, bt, cl, gc = paged_rows(lens, 2 * G, 2, D, bs, dt, 70)
    for s, rows in bad.items():
        for t, heads in rows.items():
            c, b = rm.codes_of(vc, bs, D)
            for h in heads:
                b[bt[s, t // bs].long(), h, t % bs] = 255
                c[bt[s, t // bs].long(), h, t % bs] = 0x7f
    q = torch.randn(sum(counts), 2 * G, D, generator=gc, device="cuda").to(rm.DT[dt])
    check("paged_attention_prefill_fp8row", lens, counts, 2 * G, D, bs, dt, kc, vc, bt,
          lambda c, s, L: rm.sequence(c, bs, D, bt, s, L), q, D ** -0.5)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_rows_in_many_items_of_a_cta(dt, D):
    """More items than SMs: what one leaves behind is not the next one's."""
    lens = [(37 * i) % 400 + 1 for i in range(40)]
    kc, vc, bt, cl, gc = paged_rows(lens, 16, 16, D, 16, dt, 71)
    c, b = rm.codes_of(vc, 16, D)
    g = torch.Generator()
    g.manual_seed(5)
    for s, L in enumerate(lens):
        if s % 3 == 0:
            t, h = int(torch.randint(L, (1,), generator=g)), int(torch.randint(16, (1,), generator=g))
            b[bt[s, t // 16].long(), h, t % 16] = 255
    q = torch.randn(sum(lens), 16, D, generator=gc, device="cuda").to(rm.DT[dt])
    out = check("paged_attention_prefill_fp8row", lens, lens, 16, D, 16, dt, kc, vc, bt,
                lambda c, s, L: rm.sequence(c, 16, D, bt, s, L), q, D ** -0.5)
    again = torch.empty_like(out)
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    pkv.paged_attention_prefill_fp8row(again, q, kc, vc, bt, cl, start, D ** -0.5, max_query_len=max(lens))
    assert torch.equal(out.nan_to_num(9.0), again.nan_to_num(9.0))


@pytest.mark.parametrize("dt,G,D,bs", [("bf16", 1, 128, 16), ("f16", 1, 64, 32), ("bf16", 8, 64, 16), ("f16", 3, 128, 32)])
def test_nan_codes_of_a_per_tensor_cache(dt, G, D, bs):
    lens, counts = [300, 140, 700, 5], [300, 140, 257, 5]
    g = torch.Generator()
    g.manual_seed(72)
    bt, NB = rm.pages(lens, bs, g)
    gc = gen_of(72)
    kc, vc = (torch.randn(NB, 2, bs, D, generator=gc, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    for s, t, h, d in ((0, 130, 0, 7), (0, 299, 1, D - 1), (0, 5, 1, 0), (1, 139, 0, 40), (2, 0, 0, 33), (2, 520, 1, 63),
                       (2, 699, 1, 62), (2, 300, 0, 1), (3, 3, 1, 17)):
        vc[bt[s, t // bs].long(), h, t % bs, d] = 0xff if t % 2 else 0x7f
    q = torch.randn(sum(counts), 2 * G, D, generator=gc, device="cuda").to(rm.DT[dt])

    def rows(c, s, L):
        t = torch.arange(L, device="cuda")
        return c.view(torch.float8_e4m3fn).double()[bt[s, t // bs].long(), :, t % bs] * 0.5
    check("paged_attention_prefill_fp8kv", lens, counts, 2 * G, D, bs, dt, kc, vc, bt, rows, q, D ** -0.5, (0.5, 0.5))


@pytest.mark.parametrize("D,bs,G", [(64, 16, 1), (128, 32, 4), (128, 16, 8)])
def test_v_rows_from_the_end_of_fp16(D, bs, G):
    """65504 is stored as 65536, which f16 has not: an infinity for the queries
    that see it, both signs together a NaN, and nothing for the others."""
    lens, counts, Hkv = [300, 200], [300, 150], 2
    kc, vc, bt, cl, gc = paged_rows(lens, Hkv * G, Hkv, D, bs, "f16", 73)
    for s, t, h, d, x in ((0, 70, 0, 3, 65504.0), (0, 200, 0, 3, -65504.0), (0, 131, 1, 60, -63488.0), (1, 199, 0, 5, 65504.0),
                          (1, 10, 1, 9, 65504.0)):
        row = torch.randn(1, Hkv, D, generator=gc, device="cuda").half()
        row[0, h, d] = x
        pkv.reshape_and_cache_fp8row(row, row, torch.zeros_like(kc), vc, (bt[s, t // bs].long() * bs + t % bs).view(1))
    q = torch.randn(sum(counts), Hkv * G, D, generator=gc, device="cuda").half()
    out = check("paged_attention_prefill_fp8row", lens, counts, Hkv * G, D, bs, "f16", kc, vc, bt,
                lambda c, s, L: rm.sequence(c, bs, D, bt, s, L), q, D ** -0.5)
    assert out[:70].isfinite().all() and (out[70:200, :G, 3] == math.inf).all() and out[200:300, :G, 3].isnan().all()


def large_keys(x, g):
    x = x * 1000.0
    x[::7, :, 0] = 65504.0                       # stored as 65536
    x[3::7, :, 1] = -63488.0
    x[5::50, :, 2] = 90000.0                     # as a rotated f16 key may be
    return x


@pytest.mark.parametrize("D,bs,G", [(64, 16, 1), (128, 32, 8)])
def test_k_elements_from_the_end_of_fp16_in_chunks(D, bs, G):
    lens, counts, Hkv = [300, 77], [140, 77], 2
    kc, vc, bt, cl, gc = paged_rows(lens, Hkv * G, Hkv, D, bs, "f16", 74, kscale=large_keys)
    q = torch.randn(sum(counts), Hkv * G, D, generator=gc, device="cuda").half()
    check("paged_attention_prefill_fp8row", lens, counts, Hkv * G, D, bs, "f16", kc, vc, bt,
          lambda c, s, L: rm.sequence(c, bs, D, bt, s, L), q, 1e-5)


@pytest.mark.parametrize("D,bs,G", [(64, 16, 20), (128, 32, 64)])
def test_k_elements_from_the_end_of_fp16_in_decode(D, bs, G):
    lens = [300, 77, 1000]
    kc, vc, bt, cl, gc = paged_rows(lens, 2 * G, 2, D, bs, "f16", 75, kscale=large_keys)
    q = torch.randn(3, 2 * G, D, generator=gc, device="cuda").half()
    out = torch.empty_like(q)
    pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, 1e-5)
    for s, L in enumerate(lens):
        K, V = (rm.sequence(c, bs, D, bt, s, L) for c in (kc, vc))
        ref, logit, top = masked_reference(q[s:s + 1], K, V, 1e-5, torch.float16)
        rm.close(out[s:s + 1], ref, rm.attention_bound(ref, logit, top, torch.float16, torch.float16, L) + 2.0 ** -25)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs,G", [(64, 16, 1), (128, 32, 4)])
def test_v_rows_of_large_scales(dt, D, bs, G):
    """Every 50th row 2^8 to 2^50 times as large: bf16 holds all of it, of fp16 a row
    has elements on both sides of its range."""
    def large(x, g):
        x = x.clone()
        n = x[20::50].shape[0]
        x[20::50] *= torch.exp2(torch.randint(8, 51, (n, x.shape[1], 1), generator=g, device="cuda").float())
        if n:
            x[20::50, :, ::3] *= 2.0 ** -16
        return x
    lens, counts, Hkv = [300, 40, 130], [300, 40, 90], 2
    kc, vc, bt, cl, gc = paged_rows(lens, Hkv * G, Hkv, D, bs, dt, 76, vscale=large)
    q = torch.randn(sum(counts), Hkv * G, D, generator=gc, device="cuda").to(rm.DT[dt])
    check("paged_attention_prefill_fp8row", lens, counts, Hkv * G, D, bs, dt, kc, vc, bt,
          lambda c, s, L: rm.sequence(c, bs, D, bt, s, L), q, D ** -0.5)
