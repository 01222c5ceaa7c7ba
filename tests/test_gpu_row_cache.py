"""The 8-bit row cache on the GPU: the quantising write bit for bit, its fused
rotary form, the read-back, and decode and chunk attention over it against the
64-bit form with bounds that count roundings."""
import math

import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from paged_kv_cache_480_b200 import binding
from test_gpu_rotary import gen_of, packed

pytestmark = pytest.mark.gpu


def dirty(NB, Hkv, bs, D, gen):
    """A pool full of arbitrary bytes (NaN codes and any scale among them)."""
    return torch.randint(0, 256, pkv.fp8row_cache_shape(NB, Hkv, bs, D), generator=gen, device="cuda").to(torch.uint8)


# ---- the write ---------------------------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 1, 64, 16), (5, 3, 128, 16), (300, 8, 128, 32), (77, 2, 64, 32), (2050, 1, 64, 16)])
def test_write_is_bit_exact(dt, T, Hkv, D, bs):
    g = gen_of(T + D)
    _, k, v = packed(g, T, 1, Hkv, D, rm.DT[dt], extra=16)
    k.mul_(torch.exp2(torch.randint(-8, 9, (T, Hkv, 1), generator=g, device="cuda").float()).to(k.dtype))
    NB = T // bs + 2
    slots = torch.randperm(NB * bs, generator=g, device="cuda")[:T].contiguous()
    kc, vc = dirty(NB, Hkv, bs, D, g), dirty(NB, Hkv, bs, D, g)
    want = [kc.clone(), vc.clone()]
    on = torch.ones(T, dtype=torch.bool, device="cuda")
    if T > 3:
        on[2] = False
        slots[2] = -7
    for c, x in zip(want, (k, v)):
        rm.put(c, bs, D, slots[on] // bs, slots[on] % bs, x[on])
    pkv.reshape_and_cache_fp8row(k, v, kc, vc, slots)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert pkv.read_device_errors() == 0
    slots[0] = NB * bs + 3
    pkv.reshape_and_cache_fp8row(k, v, kc, vc, slots)
    assert pkv.read_device_errors() == 2
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_write_of_special_rows():
    D, bs = 64, 16
    rows = torch.randn(16, D, generator=gen_of(5), device="cuda")
    rows[0] = 0.0
    rows[1, 5] = math.inf
    rows[2, 7] = math.nan
    rows[3, 63] = -math.inf
    rows[4] *= 1e-38                        # fp32 subnormals among them
    rows[5] *= 3e37
    rows[6] = 0.0
    rows[6, 0] = 448.0 * 2.0 ** 9           # on the border of an exponent,
    rows[7] = rows[6]
    rows[7, 0] = 448.0 * 2.0 ** 9 * (1 + 2.0 ** -23)   # and one step above
    rows[8] = -3.4e38
    rows[9] = 2.0 ** -149
    rows[10, 0] = 448.0 * 2.0 ** 60
    rows[11, :] = math.nan
    k = rows.view(16, 1, D)
    kc, vc = (torch.zeros(pkv.fp8row_cache_shape(1, 1, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(16, device="cuda")
    pkv.reshape_and_cache_fp8row(k, k.flip(0).contiguous(), kc, vc, slots)
    want = torch.zeros_like(kc)
    rm.put(want, bs, D, slots // bs, slots % bs, k)
    assert torch.equal(kc, want)
    out = torch.empty(16, 1, D, device="cuda")
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    pkv.gather_cache_fp8row(out, torch.empty_like(out), kc, vc, bt, torch.tensor([0, 16], dtype=torch.int32, device="cuda"))
    assert out[2].isnan().all() and out[11].isnan().all() and out[[0, 1, 3, 4, 5, 6, 7, 8, 9, 10]].isfinite().all()
    assert out[1, 0, 5] == 448.0 * 2.0 ** 60 and out[3, 0, 63] == -448.0 * 2.0 ** 60 and (out[0] == 0).all()


@pytest.mark.parametrize("dt,T,H,Hkv,D,R,bs,il", [("bf16", 260, 8, 8, 128, 128, 16, False), ("f16", 33, 16, 2, 128, 64, 32, True),
                                                  ("f32", 4, 4, 4, 64, 64, 16, False), ("f32", 50, 0, 3, 128, 20, 16, False),
                                                  ("bf16", 1, 5, 1, 64, 6, 32, False), ("f16", 1030, 1, 1, 64, 64, 16, False),
                                                  ("f32", 21, 2, 1, 128, 126, 32, True), ("bf16", 30, 4, 2, 64, 40, 16, False),
                                                  ("f16", 30, 3, 2, 128, 20, 32, False)])
def test_rotary_write(dt, T, H, Hkv, D, R, bs, il):
    g = gen_of(T + R)
    q, k, v = packed(g, T, H, Hkv, D, rm.DT[dt], extra=16)
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda")
    f, att = pkv.rotary_frequencies(R, scaling="by_index", factor=4.0, original_context=8192)
    f = f.cuda()
    NB = T // bs + 2
    slots = torch.randperm(NB * bs, generator=g, device="cuda")[:T].contiguous()
    kc, vc = dirty(NB, Hkv, bs, D, g), dirty(NB, Hkv, bs, D, g)
    before = [kc.clone(), vc.clone()]
    qo = torch.empty(T, H, D, dtype=q.dtype, device="cuda")
    pkv.rotary_reshape_and_cache_fp8row(qo, q, k, v, kc, vc, pos, slots, f, interleaved=il, attention_scale=att)
    assert pkv.read_device_errors() == 0
    if H:
        ref = rm.rotate(q, pos, f, il, att)
        rm.close(qo, ref, rm.half_step(q.dtype) * ref.abs() + rm.rotate_slack(q, f, il, att) + 2.0 ** -25)
    # V: bit for bit.  K: the scale of the exact row (or, with its largest
    # element within the rotation's error of a border, the neighbour), and each
    # element within half a step of its value
    blk, off = slots // bs, slots % bs
    rm.put(before[1], bs, D, blk, off, v)
    assert torch.equal(vc, before[1])
    c, b = rm.codes_of(kc, bs, D)
    ref, slack = rm.rotate(k, pos, f, il, att), rm.rotate_slack(k, f, il, att)
    e = b[blk, :, off].double() - 127.0
    amax, s = ref.abs().amax(-1), slack.amax(-1)
    assert (amax <= 448.0 * torch.pow(2.0, e) + s).all() and (amax > 224.0 * torch.pow(2.0, e) - s).all()
    step = torch.maximum(ref.abs() * 2.0 ** -4, 2.0 ** -10 * torch.pow(2.0, e)[..., None])
    rm.close(rm.value(c[blk, :, off], b[blk, :, off]), ref, step + 2 * slack)
    if H:                                           # q in place: the same bits
        q2 = q.clone()
        pkv.rotary_reshape_and_cache_fp8row(q2, q2, k, v, kc, vc, pos, slots, f, interleaved=il, attention_scale=att)
        assert torch.equal(q2, qo)
    # every other byte of the K pool stays
    cb, bb = rm.codes_of(before[0], bs, D)
    cb[blk, :, off] = c[blk, :, off]
    bb[blk, :, off] = b[blk, :, off]
    assert torch.equal(kc, before[0])


# ---- the read-back -----------------------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hkv,D,bs,lens", [(1, 64, 16, [1]), (3, 128, 16, [0, 17, 0, 0, 300, 1, 16]), (8, 64, 32, [33, 64, 2000]),
                                           (2, 128, 32, [5] * 70), (40, 128, 16, [700, 0])])
def test_gather_reads_every_token(dt, Hkv, D, bs, lens):
    g = torch.Generator()
    g.manual_seed(len(lens))
    bt, NB = rm.pages(lens, bs, g)
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    T = int(start[-1])
    dtype, gc = rm.DT[dt], gen_of(D)
    s = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)]).cuda().long()
    t = torch.cat([torch.arange(n) for n in lens]).cuda()
    blk, off = bt[s, t // bs].long(), t % bs
    spare = 3                                     # rows behind the last sequence stay as they were
    def outs():
        return [torch.full((T + spare, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    # bits
    caches = [torch.randn(NB, Hkv, bs, D, generator=gc, device="cuda").to(dtype) for _ in range(2)]
    caches[0][0, 0, 0, 0] = math.nan
    for o, c in zip(pkv.gather_cache(*outs(), *caches, bt, start), caches):
        assert torch.equal(o[:T].nan_to_num(3.0), c[blk, :, off].nan_to_num(3.0)) and (o[T:] == 7).all()
    # one scale for all of K and one for all of V
    fp8 = [torch.randint(0, 127, (NB, Hkv, bs, D), generator=gc, device="cuda").to(torch.uint8) for _ in range(2)]
    for o, c, sc in zip(pkv.gather_cache_fp8kv(*outs(), *fp8, bt, start, 0.3, 1.7), fp8, (0.3, 1.7)):
        want = c.view(torch.float8_e4m3fn).float()[blk, :, off] * torch.tensor(sc, device="cuda")
        assert torch.equal(o[:T], want.to(dtype)) and (o[T:] == 7).all()
    # row scales (the exponents reach past fp16's range)
    rows = [dirty(NB, Hkv, bs, D, gc) for _ in range(2)]
    for c in rows:
        cc, b = rm.codes_of(c, bs, D)
        cc[(cc & 127) == 127] = 0
        b.copy_(torch.randint(67, 188, b.shape, generator=gc, device="cuda"))
    for o, c in zip(pkv.gather_cache_fp8row(*outs(), *rows, bt, start), rows):
        cc, b = rm.codes_of(c, bs, D)
        want = rm.value(cc[blk, :, off], b[blk, :, off]).float().to(dtype)
        assert torch.equal(o[:T], want) and (o[T:] == 7).all()
    assert pkv.read_device_errors() == 0


def test_gather_bad_pages_and_lengths():
    Hkv, D, bs, NB = 2, 64, 16, 5
    c = torch.randn(NB, Hkv, bs, D, generator=gen_of(2), device="cuda")
    bt = torch.tensor([[1, NB], [-1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    k, v = torch.full((2, 90, Hkv, D), 7.0, device="cuda")
    pkv.gather_cache(k, v, c, c, bt, torch.tensor([0, 20, 40, 80], dtype=torch.int32, device="cuda"))
    assert pkv.read_device_errors() == 1 | 4
    assert torch.equal(k[:16], c[1].transpose(0, 1)) and (k[16:36] == 0).all()
    assert torch.equal(k[36:40], c[2].transpose(0, 1)[:4]) and torch.equal(v[40:56], c[3].transpose(0, 1))
    assert torch.equal(k[56:72], c[4].transpose(0, 1)) and (k[72:] == 7).all()      # past the table: not written
    # rows before the first sequence stay, too
    k.fill_(7.0)
    pkv.gather_cache(k, v, c, c, bt[2:], torch.tensor([50, 82], dtype=torch.int32, device="cuda"))
    assert pkv.read_device_errors() == 0
    assert (k[:50] == 7).all() and torch.equal(k[50:66], c[3].transpose(0, 1)) and (k[82:] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_of_very_many_heads(dt):
    """A token of more 16-byte units than 2^16."""
    Hkv, D, bs, NB, dtype = 4099, 128, 16, 2, rm.DT[dt]
    g = gen_of(3)
    _, k, v = packed(g, 3, 1, Hkv, D, dtype)
    slots = torch.tensor([17, 3, 16], device="cuda")
    rows = [torch.zeros(pkv.fp8row_cache_shape(NB, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    same = [torch.zeros(NB, Hkv, bs, D, dtype=dtype, device="cuda") for _ in range(2)]
    pkv.reshape_and_cache_fp8row(k, v, *rows, slots)
    pkv.reshape_and_cache(k, v, *same, slots)
    bt = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")    # slots 16, 17 and 0 to 3
    at = torch.tensor([2, 0, 0, 0, 0, 1], device="cuda")                 # the tokens in them
    some = torch.tensor([1, 1, 0, 0, 0, 1], device="cuda", dtype=dtype).view(6, 1, 1)
    outs = lambda: [torch.full((6, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    for o, x in zip(pkv.gather_cache(*outs(), *same, bt, start), (k, v)):
        assert torch.equal(o, x[at] * some)
    for o, c in zip(pkv.gather_cache_fp8row(*outs(), *rows, bt, start), rows):
        cc, b = rm.codes_of(c, bs, D)
        want = rm.value(cc, b)[[1, 1, 0, 0, 0, 0], :, [0, 1, 0, 1, 2, 3]].float().to(dtype)
        assert torch.equal(o, want)
    want = [torch.zeros_like(c) for c in rows]
    for c, x in zip(want, (k, v)):
        rm.put(c, bs, D, slots // bs, slots % bs, x)
    assert torch.equal(rows[0], want[0]) and torch.equal(rows[1], want[1])
    assert pkv.read_device_errors() == 0


# ---- decode --------------------------------------------------------------------
def paged_rows(lens, H, Hkv, D, bs, dt, seed, kscale=None, vscale=None):
    """q, dirty row caches holding the sequences' rows, and tables."""
    g = torch.Generator()
    g.manual_seed(seed)
    bt, NB = rm.pages(lens, bs, g)
    gc = gen_of(seed)
    kc, vc = dirty(NB, Hkv, bs, D, gc), dirty(NB, Hkv, bs, D, gc)
    K = [torch.randn(L, Hkv, D, generator=gc, device="cuda") for L in lens]
    V = [torch.randn(L, Hkv, D, generator=gc, device="cuda") for L in lens]
    if kscale:
        K = [kscale(x, gc) for x in K]
    if vscale:
        V = [vscale(x, gc) for x in V]
    rm.fill_rows(kc, bs, D, bt, lens, K)
    rm.fill_rows(vc, bs, D, bt, lens, V)
    return kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), gc


def check_decode(lens, H, Hkv, D, bs, dt, seed=0, ps=0, scale=None, q=None, **kw):
    kc, vc, bt, cl, gc = paged_rows(lens, H, Hkv, D, bs, dt, seed, **kw)
    dtype = rm.DT[dt]
    if q is None:
        q = torch.randn(len(lens), H, D, generator=gc, device="cuda").to(dtype)
    scale = D ** -0.5 if scale is None else scale
    out = torch.full_like(q, math.nan)
    pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, scale, partition_size=ps)
    assert pkv.read_device_errors() == 0
    for s, L in enumerate(lens):
        K, V = (rm.sequence(c, bs, D, bt, s, L) for c in (kc, vc))
        ref, logit, top = rm.attend(q[s:s + 1], K, V, scale)
        # weights are rounded to fp16, in groups of 17 and more query heads (whose
        # products take the elements in q's type) to q's type
        weights = None if dt == "f32" else dtype if H // Hkv >= 17 and ps == 0 else torch.float16
        rm.close(out[s:s + 1], ref, rm.attention_bound(ref, logit, top, dtype, weights, L))
    return out, (kc, vc, bt, cl, q)


@pytest.mark.parametrize("dt,G,D,bs", [("bf16", 1, 128, 16), ("f16", 1, 64, 32), ("f16", 2, 128, 16), ("bf16", 2, 64, 16),
                                       ("bf16", 4, 64, 32), ("f16", 3, 128, 32), ("bf16", 8, 128, 16), ("f16", 8, 64, 32),
                                       ("bf16", 5, 64, 16), ("f16", 16, 128, 16), ("bf16", 71, 64, 16), ("f16", 130, 64, 32),
                                       ("bf16", 17, 128, 32), ("f16", 64, 64, 16), ("bf16", 64, 128, 16), ("f32", 1, 64, 16),
                                       ("f32", 1, 128, 32), ("f32", 2, 64, 32), ("f32", 4, 128, 16), ("f32", 8, 64, 16),
                                       ("f32", 7, 128, 32), ("f32", 16, 64, 16)])
def test_decode_edge_lengths(dt, G, D, bs):
    check_decode([0, 1, 15, 16, 17, 31, 33, 255, 257, 513, 1000], 2 * G, 2, D, bs, dt, seed=G + D)


@pytest.mark.parametrize("dt,G", [("f16", 1), ("bf16", 8), ("f32", 2)])
def test_decode_long_and_forced_partitions(dt, G):
    check_decode([20000, 3, 8191], 2 * G, 2, 128, 16, dt, seed=3)
    check_decode([1, 47, 700, 2048], 2 * G, 2, 64, 16, dt, seed=4, ps=48)


@pytest.mark.parametrize("dt,H,Hkv,D,bs", [("bf16", 64, 1, 128, 16), ("f16", 40, 2, 128, 32), ("bf16", 18, 1, 64, 16)])
def test_decode_large_groups_long(dt, H, Hkv, D, bs):
    """Units of very different lengths split over the CTAs, empty ones between
    them; more sequences than threads; and the same with partitions, which take
    the other kernel."""
    check_decode([20000, 0, 3, 8191, 0, 128, 129], H, Hkv, D, bs, dt, seed=14)
    check_decode([(13 * i) % 300 for i in range(700)], H, Hkv, 64, bs, dt, seed=15)
    check_decode([500, 77], H, Hkv, D, bs, dt, seed=16, ps=2 * bs)


def test_decode_many_short_sequences():
    check_decode([(7 * i) % 50 for i in range(500)], 4, 1, 64, 16, "bf16", seed=6)


@pytest.mark.parametrize("S", [2, 60, 400])
@pytest.mark.parametrize("G,D,bs", [(3, 128, 32), (6, 64, 32), (8, 128, 32), (8, 128, 16), (12, 64, 16)])
def test_decode_f32_groups_whole_and_in_slices(S, G, D, bs):
    """From calls that leave most warps idle to more items than warps."""
    check_decode([(7 * i) % 70 for i in range(S)], 5 * G, 5, D, bs, "f32", seed=9)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("G", [1, 8])
def test_decode_rows_of_very_different_scales(dt, G):
    """V rows over 2^-30 .. 2^30 and K rows over 2^-10 .. 2^2: the weights are
    relative to the largest contribution, so its neighbours in size keep their
    precision."""
    def spread(lo, hi):
        return lambda x, g: x * torch.exp2(torch.randint(lo, hi + 1, x.shape[:2] + (1,), generator=g, device="cuda").float())
    check_decode([5, 40, 300, 900], 2 * G, 2, 128, 16, dt, seed=8, kscale=spread(-10, 2), vscale=spread(-30, 30) if dt == "f32"
                 else spread(-12, 12))
    if dt == "bf16":                                    # exact in q's type over the whole range of the format
        check_decode([5, 300], 40, 2, 128, 16, dt, seed=8, kscale=spread(-10, 2), vscale=spread(-40, 40))


@pytest.mark.parametrize("dt,size", [("bf16", 1e-12), ("f32", 1e-12), ("bf16", 1e-4), ("f32", 1e-4), ("bf16", 1e4), ("f32", 1e4)])
def test_decode_values_of_any_size(dt, size):
    """Outputs scale with V."""
    check_decode([50, 300], 4, 4, 64, 16, dt, seed=9, vscale=lambda x, g: x * size)


def test_decode_values_near_the_end_of_fp16():
    """fp16 outputs of this size are subnormal (below 2^-14): half their spacing is 2^-25."""
    kc, vc, bt, cl, gc = paged_rows([50, 300], 4, 4, 64, 16, "f16", 9, vscale=lambda x, g: x * 1e-4)
    q = torch.randn(2, 4, 64, generator=gc, device="cuda").half()
    out = torch.empty_like(q)
    pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, 0.125)
    for s, L in enumerate([50, 300]):
        ref, logit, top = rm.attend(q[s:s + 1], *(rm.sequence(c, 16, 64, bt, s, L) for c in (kc, vc)), 0.125)
        rm.close(out[s:s + 1], ref, rm.attention_bound(ref, logit, top, torch.float16, torch.float16, L) + 2.0 ** -25)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_decode_a_row_of_zeros_that_takes_all_weight(dt):
    """A key with by far the largest logit whose V row is zero (scale 2^-60):
    its weight is below fp16's range beside the others', but it is the sum."""
    L, D = 70, 64
    q = torch.zeros(1, 2, D, device="cuda", dtype=rm.DT[dt])
    q[..., 0] = 4.0

    def keys(x, g):
        x = x * 0.1
        x[33, :, 0] = 30.0
        return x

    def values(x, g):
        x = x.clone()
        x[33] = 0.0
        return x
    out, _ = check_decode([L], 2, 2, D, 16, dt, seed=10, q=q, scale=0.1, kscale=keys, vscale=values)
    assert float(out.abs().max()) < 1e-3            # the others hold e^-12 of the weight


def test_decode_nan_rows_stay_in_their_head():
    lens, D, bs = [40, 40], 64, 16
    kc, vc, bt, cl, gc = paged_rows(lens, 4, 2, D, bs, "bf16", 11)
    q = torch.randn(2, 4, D, generator=gc, device="cuda").bfloat16()
    bad = torch.full((1, 2, D), 1.0, device="cuda")
    bad[0, 1, 3] = math.nan
    rm.put(vc, bs, D, bt[0, :1].long(), torch.tensor([5], device="cuda"), bad)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, 0.125)
    assert out[0, 2:].isnan().all() and out[0, :2].isfinite().all() and out[1].isfinite().all()
    for dt in (torch.float32, torch.float16):
        o = torch.empty_like(q, dtype=dt)
        pkv.paged_attention_decode_fp8row(o, q.to(dt), vc, kc, bt, cl, 0.125)       # NaN in K
        assert o[0, 2:].isnan().all() and o[0, :2].isfinite().all() and o[1].isfinite().all()
    for a, b in ((kc, vc), (vc, kc)):                   # groups of 20
        o = torch.empty(2, 40, D, dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_decode_fp8row(o, q.repeat_interleave(10, 1), a, b, bt, cl, 0.125)
        assert o[0, 20:].isnan().all() and o[0, :20].isfinite().all() and o[1].isfinite().all()


@pytest.mark.parametrize("H", [8, 40])
def test_decode_device_checks_and_repeats(H):
    out, (kc, vc, bt, cl, q) = check_decode([100, 33, 700], H, 2, 128, 16, "f16", seed=12)
    again = torch.empty_like(out)
    for _ in range(3):
        pkv.paged_attention_decode_fp8row(again, q, kc, vc, bt, cl, 128 ** -0.5)
        assert torch.equal(again, out)
    bad = bt.clone()
    bad[0, 1] = kc.shape[0]
    pkv.paged_attention_decode_fp8row(again, q, kc, vc, bad, cl, 128 ** -0.5)
    assert pkv.read_device_errors() == 1
    long = cl.clone()
    long[1] = bt.shape[1] * 16 + 1
    pkv.paged_attention_decode_fp8row(again, q, kc, vc, bt, long, 128 ** -0.5)
    assert pkv.read_device_errors() == 4 and (again[1] == 0).all() and torch.equal(again[0], out[0])


@pytest.mark.parametrize("dt,H", [("f16", 4), ("f32", 4), ("bf16", 80)])
def test_decode_wait_limit(dt, H):
    _, (kc, vc, bt, cl, q) = check_decode([600, 33], H, 4, 64, 16, dt, seed=13)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, 0.125)
    lost = torch.empty_like(q)
    pkv.set_wait_limit(0)
    try:
        pkv.paged_attention_decode_fp8row(lost, q, kc, vc, bt, cl, 0.125)
        assert pkv.read_device_errors() == 16
    finally:
        pkv.set_wait_limit(-1)
    pkv.paged_attention_decode_fp8row(lost, q, kc, vc, bt, cl, 0.125)
    assert pkv.read_device_errors() == 0 and torch.equal(lost, out)


# ---- chunk attention -------------------------------------------------------------
def check_prefill(lens, counts, H, Hkv, D, bs, dt, seed=0, scale=None, **kw):
    kc, vc, bt, cl, gc = paged_rows(lens, H, Hkv, D, bs, dt, seed, **kw)
    dtype = rm.DT[dt]
    start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    T = sum(counts)
    q = torch.randn(T, H, D, generator=gc, device="cuda").to(dtype)
    out = torch.full_like(q, math.nan)
    scale = D ** -0.5 if scale is None else scale
    pkv.paged_attention_prefill_fp8row(out, q, kc, vc, bt, cl, start, scale, max_query_len=max(counts))
    assert pkv.read_device_errors() == 0
    for s, (L, n) in enumerate(zip(lens, counts)):
        a = int(start[s])
        K, V = (rm.sequence(c, bs, D, bt, s, L) for c in (kc, vc))
        ref, logit, top = rm.attend(q[a:a + n], K, V, scale)
        rm.close(out[a:a + n], ref, rm.attention_bound(ref, logit, top, dtype, dtype, L))
    return out, (kc, vc, bt, cl, start, q)


@pytest.mark.parametrize("dt,G,D,bs", [("bf16", 1, 128, 16), ("f16", 1, 64, 16), ("f16", 4, 128, 32), ("bf16", 8, 64, 32),
                                       ("bf16", 3, 128, 32), ("f16", 7, 64, 32), ("bf16", 16, 128, 16), ("f16", 128, 64, 16),
                                       ("f16", 2, 128, 16), ("bf16", 100, 64, 16)])
def test_prefill_prompts_and_chunks(dt, G, D, bs):
    Hkv = 2 if G < 100 else 1
    check_prefill([1, 17, 128, 129, 300, 40, 700, 0], [1, 17, 128, 100, 1, 40, 257, 0], G * Hkv, Hkv, D, bs, dt, seed=G + D)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_long_context(dt):
    check_prefill([9000, 4097, 5], [130, 256, 5], 8, 2, 128, 16, dt, seed=20)


def test_prefill_many_items_per_cta():
    """More items than SMs: the streams run on across items of different lengths."""
    lens = [(37 * i) % 400 + 1 for i in range(40)]
    check_prefill(lens, lens, 16, 16, 64, 16, "f16", seed=21)


def test_prefill_rows_of_very_different_scales():
    """bf16 holds every row scale exactly, fp16 those its range holds."""
    def spread(lo, hi):
        return lambda x, g: x * torch.exp2(torch.randint(lo, hi + 1, x.shape[:2] + (1,), generator=g, device="cuda").float())
    check_prefill([300, 50], [200, 50], 4, 2, 128, 16, "bf16", seed=22, kscale=spread(-12, 2), vscale=spread(-40, 40))
    check_prefill([300, 50], [200, 50], 4, 2, 128, 16, "bf16", seed=23, scale=1e-6, kscale=spread(8, 12), vscale=spread(-3, 3))
    check_prefill([300, 50], [200, 50], 4, 2, 64, 32, "f16", seed=24, kscale=spread(-10, 2), vscale=spread(-4, 10))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_takes_elements_in_q_type(dt):
    """With one visible key the output is its V row in q's type: exact for every
    code and every scale byte the write can give."""
    bs, D = 16, 128
    n = 121 * 2                                        # exponents -60 .. 60, all 254 codes over two rows
    bt = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    vc = torch.zeros(pkv.fp8row_cache_shape(n, 1, bs, D), dtype=torch.uint8, device="cuda")
    kc = torch.zeros_like(vc)
    c, b = rm.codes_of(vc, bs, D)
    codes = torch.tensor([x for x in range(256) if x & 127 != 127] + [0, 0], device="cuda").to(torch.uint8).view(2, D)
    c[:, 0, 0] = codes.repeat(121, 1)
    b[:, 0, 0] = torch.arange(67, 188, device="cuda").repeat_interleave(2).to(torch.uint8)
    rm.codes_of(kc, bs, D)[1].fill_(127)
    q = torch.randn(n, 1, D, generator=gen_of(25), device="cuda").to(rm.DT[dt])
    out = torch.empty_like(q)
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    pkv.paged_attention_prefill_fp8row(out, q, kc, vc, bt, ones, start, 1.0, max_query_len=1)
    want = rm.value(c[:, 0, 0], b[:, 0, 0])
    same = want.float().to(rm.DT[dt]).view(n, 1, D)
    fine = same.isfinite()
    # (a row with an infinity of fp16: inf in its own elements; every finite row exact)
    assert torch.equal(out[fine], same[fine])
    assert (out[~fine] == same[~fine]).all()
    if dt == "bf16":
        assert fine.all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_nan_rows_and_codes(dt):
    """A NaN row of K (V) makes the queries that see its tile NaN in its head; a
    NaN code of a per-tensor V cache makes its dim NaN."""
    dtype, D, bs = rm.DT[dt], 64, 16
    kc, vc, bt, cl, gc = paged_rows([200, 40], 4, 2, D, bs, dt, 28)
    q = torch.randn(240, 4, D, generator=gc, device="cuda").to(dtype)
    start = torch.tensor([0, 200, 240], dtype=torch.int32, device="cuda")
    bad = torch.ones(1, 2, D, device="cuda")
    bad[0, 1, 3] = math.nan
    at = torch.tensor([130 % bs], device="cuda")
    for which in (0, 1):
        pair = [kc.clone(), vc.clone()]
        rm.put(pair[which], bs, D, bt[0, 130 // bs:130 // bs + 1].long(), at, bad)
        out = torch.empty_like(q)
        pkv.paged_attention_prefill_fp8row(out, q, *pair, bt, cl, start, 0.125, max_query_len=200)
        assert out[130:200, 2:].isnan().all() and out[:128].isfinite().all()
        assert out[:, :2].isfinite().all() and out[200:].isfinite().all()
    k8, v8 = (torch.full((bt.max() + 1, 2, bs, D), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2))   # 1.0
    v8[bt[0, 0].long(), 1, 5, 7] = 0xff
    pkv.paged_attention_prefill_fp8kv(out, q, k8, v8, bt, cl, start, 0.125, 1.0, 1.0, max_query_len=200)
    assert out[5:200, 2:, 7].isnan().all()
    out[:200, 2:, 7] = 1.0
    assert (out == 1.0).all()
    k8[bt[0, 0].long(), 0, 5, 7] = 0x7f
    pkv.paged_attention_prefill_fp8kv(out, q, k8, v8, bt, cl, start, 0.125, 1.0, 1.0, max_query_len=200)
    assert out[5:200, :2].isnan().all() and out[:5, :2].isfinite().all()


def test_prefill_checks_and_unwritten_rows():
    out, (kc, vc, bt, cl, start, q) = check_prefill([100, 60], [30, 60], 8, 2, 128, 16, "bf16", seed=26)
    bad = bt.clone()
    bad[0, 2] = kc.shape[0]
    o = torch.full_like(q, 7.0)
    pkv.paged_attention_prefill_fp8row(o, q, kc, vc, bad, cl, start, 128 ** -0.5, max_query_len=60)
    assert pkv.read_device_errors() == 1 and torch.equal(o[30:], out[30:])
    short = cl.clone()
    short[0] = 10                                       # more queries than tokens: skipped, flagged
    o.fill_(7.0)
    pkv.paged_attention_prefill_fp8row(o, q, kc, vc, bt, short, start, 128 ** -0.5, max_query_len=60)
    assert pkv.read_device_errors() == 4 and (o[:30] == 7).all() and torch.equal(o[30:], out[30:])


@pytest.mark.parametrize("polls", [0, 1])
def test_prefill_wait_limit(polls):
    out, (kc, vc, bt, cl, start, q) = check_prefill([900, 300], [900, 300], 8, 2, 64, 16, "f16", seed=27)
    o = torch.empty_like(q)
    pkv.set_wait_limit(polls)
    try:
        pkv.paged_attention_prefill_fp8row(o, q, kc, vc, bt, cl, start, 0.125, max_query_len=900)
        assert pkv.read_device_errors() == 16
    finally:
        pkv.set_wait_limit(-1)
    pkv.paged_attention_prefill_fp8row(o, q, kc, vc, bt, cl, start, 0.125, max_query_len=900)
    assert pkv.read_device_errors() == 0 and torch.equal(o, out)


@pytest.mark.parametrize("dt,G,D,bs,ks,vs", [("f16", 1, 64, 16, 0.02, 0.05), ("bf16", 8, 128, 16, 0.01, 3.0), ("bf16", 3, 64, 32, 0.02, 1e-6),
                                             ("f16", 4, 128, 32, 0.015, 0.01)])
def test_prefill_over_the_per_tensor_cache(dt, G, D, bs, ks, vs):
    """paged_attention_prefill_fp8kv over caches written by reshape_and_cache_fp8kv."""
    lens, counts, Hkv, dtype = [300, 17, 140, 1], [100, 17, 1, 1], 2, rm.DT[dt]
    g = torch.Generator()
    g.manual_seed(30)
    bt, NB = rm.pages(lens, bs, g)
    gc = gen_of(31)
    kc, vc = (torch.full((NB, Hkv, bs, D), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
    for s, L in enumerate(lens):
        t = torch.arange(L, device="cuda")
        slots = bt[s, t // bs].long() * bs + t % bs
        K, V = torch.randn(2, L, Hkv, D, generator=gc, device="cuda")
        pkv.reshape_and_cache_fp8kv(K, V * vs * 40, kc, vc, slots, ks, vs)
    start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    q = torch.randn(sum(counts), G * Hkv, D, generator=gc, device="cuda").to(dtype)
    out = torch.full_like(q, math.nan)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pkv.paged_attention_prefill_fp8kv(out, q, kc, vc, bt, cl, start, D ** -0.5, ks, vs, max_query_len=100)
    assert pkv.read_device_errors() == 0
    ks, vs = (float(torch.tensor(x, dtype=torch.float32)) for x in (ks, vs))
    for s, (L, n) in enumerate(zip(lens, counts)):
        t = torch.arange(L, device="cuda")
        K, V = (c.view(torch.float8_e4m3fn).double()[bt[s, t // bs].long(), :, t % bs] * x for c, x in ((kc, ks), (vc, vs)))
        a = int(start[s])
        ref, logit, top = rm.attend(q[a:a + n], K, V, D ** -0.5)
        tiny = 2.0 ** -25 if dt == "f16" else 0.0
        rm.close(out[a:a + n], ref, rm.attention_bound(ref, logit, top, dtype, dtype, L) + tiny)


# ---- as they are used together ------------------------------------------------
def test_serving_steps_with_the_block_manager():
    """Prompts in two chunks, a fork, copy-on-write, decode steps, a swap out and
    in, and the read-back: caches move as plain blocks, attention agrees with
    the 64-bit form over what the cache holds, keys are where the formula puts
    them."""
    H, Hkv, D, bs, NB, dtype = 8, 2, 64, 16, 40, torch.bfloat16
    gc = gen_of(40)
    kc, vc = dirty(NB, Hkv, bs, D, gc), dirty(NB, Hkv, bs, D, gc)
    f = pkv.rotary_frequencies(D)[0].cuda()
    bm = pkv.BlockManager(NB, bs, free_order=torch.randperm(NB).tolist())
    hist = {}                                     # sequence -> fp64 (rotated keys, values)
    scale = D ** -0.5

    def write(seq_slots, pos):
        T = pos.numel()
        q, k, v = packed(gc, T, H, Hkv, D, dtype)
        qo = torch.empty(T, H, D, dtype=dtype, device="cuda")
        pkv.rotary_reshape_and_cache_fp8row(qo, q, k, v, kc, vc, pos, seq_slots, f)
        return qo, rm.rotate(k, pos, f, False), v.double()

    def held(s, L):
        """The sequence's rows as the cache holds them, checked against its history."""
        table = torch.from_numpy(bm.block_table(s)).cuda()[None]
        K, V = (rm.sequence(c, bs, D, table, 0, L) for c in (kc, vc))
        for x, want in zip((K, V), hist[s]):
            top = want.abs().amax(-1, keepdim=True)
            rm.close(x, want, torch.maximum(want.abs() * 2.0 ** -4, top * 2.0 ** -18) + top * 2.0 ** -18)
        return K, V

    def check(out, q, s, L):
        K, V = held(s, L)
        ref, logit, top = rm.attend(q, K, V, scale)
        rm.close(out, ref, rm.attention_bound(ref, logit, top, dtype, torch.bfloat16, L))

    lens = {1: 50, 2: 21, 3: 100}
    for s, n in lens.items():
        bm.allocate(s, n)
    for part in (0, 1):                           # two chunks of every prompt
        ids, spans = list(lens), []
        for s, n in lens.items():
            spans.append((0, n // 2) if part == 0 else (n // 2, n))
        tables, _ = bm.fill_tables(ids, 8)
        bt = torch.from_numpy(tables).cuda()
        pos = torch.cat([torch.arange(a, b) for a, b in spans]).cuda()
        owner = torch.cat([torch.full((b - a,), i) for i, (a, b) in enumerate(spans)]).cuda().long()
        q, k, v = write(bt[owner, pos // bs].long() * bs + pos % bs, pos)
        counts = [b - a for a, b in spans]
        start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
        cl = torch.tensor([b for _, b in spans], dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        pkv.paged_attention_prefill_fp8row(out, q, kc, vc, bt, cl, start, scale, max_query_len=max(counts))
        for i, s in enumerate(ids):
            a, b = int(start[i]), int(start[i + 1])
            old = hist.get(s, (k[:0], v[:0]))
            hist[s] = torch.cat([old[0], k[a:b]]), torch.cat([old[1], v[a:b]])
            check(out[a:b], q[a:b], s, spans[i][1])
    bm.fork(1, 4)                                 # shares a partly filled block
    hist[4] = hist[1]
    ids = [1, 2, 3, 4]
    for _ in range(3):
        slots, cow = bm.append_slots(ids)
        if len(cow):
            pkv.copy_blocks([kc], [vc], torch.from_numpy(cow).cuda())
        tables, now = bm.fill_tables(ids, 8)
        bt, cl = torch.from_numpy(tables).cuda(), torch.from_numpy(now).cuda()
        q, k, v = write(torch.from_numpy(slots).cuda(), cl.long() - 1)
        out = torch.empty_like(q)
        pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, scale)
        for i, s in enumerate(ids):
            hist[s] = torch.cat([hist[s][0], k[i:i + 1]]), torch.cat([hist[s][1], v[i:i + 1]])
            check(out[i:i + 1], q[i:i + 1], s, int(now[i]))
    # sequence 3 to the host and back, into other blocks
    host = pkv.BlockManager(12, bs)
    hk, hv = (torch.zeros(pkv.fp8row_cache_shape(12, Hkv, bs, D), dtype=torch.uint8).pin_memory() for _ in range(2))
    before = [x.clone() for x in held(3, 103)]
    pkv.swap_blocks([kc, vc], [hk, hv], torch.from_numpy(bm.swap_out(host, 3)).cuda())
    torch.cuda.synchronize()
    bm.allocate(9, 30)
    pkv.swap_blocks([hk, hv], [kc, vc], torch.from_numpy(host.swap_out(bm, 3)).cuda())
    assert all(torch.equal(a, b) for a, b in zip(before, held(3, 103)))
    tables, now = bm.fill_tables([3, 4], 8)
    start = torch.tensor([0, now[0], now[0] + now[1]], dtype=torch.int32, device="cuda")
    ko, vo = torch.empty(2, int(start[-1]), Hkv, D, device="cuda")
    pkv.gather_cache_fp8row(ko, vo, kc, vc, torch.from_numpy(tables).cuda(), start)
    assert torch.equal(ko[:103].double(), before[0]) and torch.equal(vo[103:].double(), held(4, int(now[1]))[1])
    assert pkv.read_device_errors() == 0


def test_a_decode_step_captured_twice():
    """Two graphs of the whole step (write and decode) that share the binding's
    workspace, replayed in turn on new inputs."""
    lens, H, Hkv, D, bs = [600, 33, 250], 8, 2, 128, 16
    kc, vc, bt, cl, gc = paged_rows(lens, H, Hkv, D, bs, "f16", 41)
    f = pkv.rotary_frequencies(D)[0].cuda()
    bufs = []
    for i in range(2):
        q, k, v = packed(gc, 3, H, Hkv, D, torch.float16)
        bufs.append((q, k, v, torch.empty(3, H, D, dtype=torch.float16, device="cuda"),
                     torch.empty(3, H, D, dtype=torch.float16, device="cuda")))
    pos = cl.long() - 1
    slots = bt[torch.arange(3, device="cuda"), pos // bs].long() * bs + pos % bs

    def step(b):
        pkv.rotary_reshape_and_cache_fp8row(b[3], b[0], b[1], b[2], kc, vc, pos, slots, f)
        pkv.paged_attention_decode_fp8row(b[4], b[3], kc, vc, bt, cl, D ** -0.5)
    for b in bufs:
        step(b)
    torch.cuda.synchronize()
    graphs = []
    for b in bufs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(b)
    for turn in range(3):
        for b, gr in zip(bufs, graphs):
            b[0].normal_(generator=gc)
            b[1].normal_(generator=gc)
            gr.replay()
            got = b[4].clone()
            step(b)
            assert torch.equal(got, b[4])
            for s, L in enumerate(lens):
                K, V = (rm.sequence(c, bs, D, bt, s, L) for c in (kc, vc))
                ref, logit, top = rm.attend(b[3][s:s + 1], K, V, D ** -0.5)
                rm.close(got[s:s + 1], ref, rm.attention_bound(ref, logit, top, torch.float16, torch.float16, L))
    assert pkv.read_device_errors() == 0


def test_the_bindings_workspace_in_graphs_and_on_streams(monkeypatch):
    """Its first use inside a capture, its growth between a capture and the
    replays, and its first use on a stream that is not the current one."""
    monkeypatch.setattr(binding, "_workspaces", {})
    H, Hkv, D, bs = 8, 2, 128, 16
    lens = [700, 40, 1300]
    kc, vc, bt, cl, gc = paged_rows(lens, H, Hkv, D, bs, "f16", 43)
    q = torch.randn(3, H, D, generator=gc, device="cuda").half()
    outs = torch.zeros(4, 3, H, D, dtype=torch.float16, device="cuda")

    def step(out, **kw):
        return pkv.paged_attention_decode_fp8row(out, q, kc, vc, bt, cl, D ** -0.5, **kw)
    need = pkv.paged_attention_workspace_size(3, H, Hkv, D, bs, bt.shape[1] * bs, 1)
    step(outs[0], workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    want = outs[0].clone()

    def captured(out):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(out)
        return graph
    first = captured(outs[1])
    assert binding._workspaces == {}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(outs[2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(outs[2], want)
    second = captured(outs[3])
    old = binding._workspaces[q.device.index]
    assert binding.default_workspace(q.device, old.numel() + 1).numel() == 2 * old.numel()
    junk = torch.full((old.numel(),), 255, dtype=torch.uint8, device="cuda")    # what may lie in memory given back
    for _ in range(3):
        outs.zero_()
        for graph in (first, second):
            graph.replay()
        step(outs[2])
        assert all(torch.equal(o, want) for o in outs[1:])
    del junk
    assert pkv.read_device_errors() == 0
