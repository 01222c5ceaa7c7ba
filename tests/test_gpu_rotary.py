"""Rotary positions on the GPU against the 64-bit form: both layouts, parts of
the head, far positions, packed projections, in place, captured graphs; and
the fused cache write."""
import math

import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm

pytestmark = pytest.mark.gpu


def packed(gen, T, H, Hkv, D, dtype, extra=0):
    """q, k, v as views of one projection's output, tokens `extra` elements further apart."""
    both = torch.randn(T, (H + 2 * Hkv) * D + extra, generator=gen, device="cuda").to(dtype)
    return (both[:, :H * D].view(T, H, D) if not extra else both[:, :H * D].unflatten(1, (H, D)),
            both[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D)),
            both[:, (H + Hkv) * D:(H + 2 * Hkv) * D].unflatten(1, (Hkv, D)))


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check(y, x, pos, f, il, att=1.0):
    ref = rm.rotate(x, pos, f, il, att)
    rm.close(y, ref, rm.half_step(y.dtype) * ref.abs() + rm.rotate_slack(x, f, il, att)
             + torch.finfo(y.dtype).smallest_normal * rm.half_step(y.dtype) * 2)


CASES = [("f16", 1, 1, 1, 64, 64), ("f16", 3, 8, 2, 128, 128), ("bf16", 257, 32, 8, 128, 64), ("f32", 65, 5, 5, 64, 64),
         ("bf16", 700, 1, 1, 64, 32), ("f32", 9, 4, 1, 128, 20), ("f16", 33, 7, 7, 80, 32), ("bf16", 5, 3, 1, 128, 2),
         ("f16", 17, 2, 2, 256, 66), ("f32", 4, 2, 1, 512, 512), ("bf16", 2, 96, 8, 16, 14), ("f16", 4096, 2, 1, 64, 64),
         ("bf16", 300, 9, 3, 80, 40), ("f16", 21, 3, 1, 64, 24), ("bf16", 12, 2, 2, 128, 20), ("f32", 30, 3, 2, 64, 12)]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dt,T,H,Hkv,D,R", CASES)
def test_rotary_matches_the_formula(dt, T, H, Hkv, D, R, il):
    g = gen_of(T + D)
    q, k, _ = packed(g, T, H, Hkv, D, rm.DT[dt], extra=16)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g, device="cuda")
    f = pkv.rotary_frequencies(R)[0].cuda()
    qo, ko = torch.empty(T, H, D, dtype=q.dtype, device="cuda"), torch.empty(T, Hkv, D, dtype=q.dtype, device="cuda")
    pkv.rotary_embedding(qo, ko, q, k, pos, f, interleaved=il, attention_scale=1.25)
    check(qo, q, pos, f, il, 1.25)
    check(ko, k, pos, f, il, 1.25)
    # the part that is not rotated is copied, whatever it holds
    assert torch.equal(qo[..., R:], q[..., R:]) and torch.equal(ko[..., R:], k[..., R:])
    # in place, q alone: the same bits
    q2 = q.clone(memory_format=torch.preserve_format)
    pkv.rotary_embedding(q2, None, q2, None, pos, f, interleaved=il, attention_scale=1.25)
    assert torch.equal(q2, qo)
    # in place inside the packed projection: the neighbours stay
    rest = q.shape[1] * D
    whole = torch.randn(T, rest + 32, generator=g, device="cuda").to(q.dtype)
    keep = whole[:, rest:].clone()
    view = whole[:, :rest].unflatten(1, (H, D))
    want = torch.empty_like(qo)
    pkv.rotary_embedding(want, None, view.contiguous(), None, pos, f, interleaved=il)
    pkv.rotary_embedding(view, None, view, None, pos, f, interleaved=il)
    assert torch.equal(view, want) and torch.equal(whole[:, rest:], keep)


def test_rotary_far_positions_and_nonfinite_values():
    """fp64 angles: positions near 2^31 are as exact as near ones; infinities
    and NaN stay in their pairs, and beyond the rotated part they are copied."""
    f = pkv.rotary_frequencies(64, scaling="by_index", factor=16.0, original_context=4096)[0].cuda()
    pos = torch.tensor([0, 1, 1 << 24, (1 << 31) - 1, 10 ** 9 + 7], device="cuda")
    x = torch.randn(5, 2, 128, generator=gen_of(1), device="cuda")
    y = torch.empty_like(x)
    pkv.rotary_embedding(y, None, x, None, pos, f)
    check(y, x, pos, f, False)
    assert torch.equal(y[0], x[0])
    x[:, 0, 3], x[:, 1, 70], x[:, 1, 100] = math.inf, math.nan, -math.inf
    pkv.rotary_embedding(y, None, x, None, pos, f)
    bad = ~y.isfinite()
    assert bad[1:, 0, [3, 35]].all() and bad[:, 1, 70].all() and (y[:, 1, 100] == -math.inf).all()
    bad[:, 0, [3, 35]] = False
    bad[:, 1, [70, 100]] = False
    assert not bad.any()


def test_rotary_no_tokens_and_k_alone():
    f = torch.ones(32, device="cuda")
    e = torch.empty(0, 4, 64, device="cuda")
    pkv.rotary_embedding(e, e.clone(), e, e.clone(), torch.empty(0, dtype=torch.int64, device="cuda"), f)
    q = torch.empty(3, 0, 64, device="cuda")
    k = torch.randn(3, 2, 64, device="cuda")
    pos = torch.arange(3, device="cuda")
    ko = torch.empty_like(k)
    pkv.rotary_embedding(q, ko, q, k, pos, f)
    check(ko, k, pos, f, False)


def test_rotary_captured_and_on_another_stream():
    g = gen_of(3)
    q, k, _ = packed(g, 40, 8, 2, 128, torch.bfloat16)
    pos = torch.arange(40, device="cuda")
    f = pkv.rotary_frequencies(128)[0].cuda()
    qo, ko = torch.zeros(40, 8, 128, dtype=q.dtype, device="cuda"), torch.zeros(40, 2, 128, dtype=q.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.rotary_embedding(qo, ko, q, k, pos, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(qo, q, pos, f, False)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkv.rotary_embedding(qo, ko, q, k, pos, f)
    pos += 1000
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(qo, q, pos, f, False)
    check(ko, k, pos, f, False)


@pytest.mark.parametrize("dt,T,H,Hkv,D,R,bs,il", [("bf16", 37, 8, 2, 128, 128, 16, False), ("f16", 5, 4, 4, 64, 32, 32, True),
                                                  ("f32", 300, 3, 1, 64, 20, 16, False), ("bf16", 1, 0, 3, 128, 64, 32, False),
                                                  ("f32", 70, 2, 2, 128, 128, 16, True), ("bf16", 9, 2, 1, 64, 22, 16, False),
                                                  ("f16", 19, 2, 3, 64, 24, 16, False), ("bf16", 19, 2, 3, 128, 20, 32, False)])
def test_rotary_write_is_rotary_then_write(dt, T, H, Hkv, D, R, bs, il):
    """rotary_reshape_and_cache gives the bits of rotary_embedding followed by
    reshape_and_cache, and skips tokens without a slot."""
    g = gen_of(T)
    q, k, v = packed(g, T, H, Hkv, D, rm.DT[dt], extra=8)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda")
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g, device="cuda")[:T].contiguous()
    if T > 2:
        slots[1] = -1
    f = pkv.rotary_frequencies(R)[0].cuda()
    caches = [torch.randn(NB, Hkv, bs, D, generator=g, device="cuda").to(q.dtype) for _ in range(2)]
    want = [c.clone() for c in caches]
    qo, qw = torch.empty(T, H, D, dtype=q.dtype, device="cuda"), torch.empty(T, H, D, dtype=q.dtype, device="cuda")
    kw = torch.empty(T, Hkv, D, dtype=q.dtype, device="cuda")
    pkv.rotary_embedding(qw, kw, q, k, pos, f, interleaved=il)
    pkv.reshape_and_cache(kw, v, want[0], want[1], slots)
    pkv.rotary_reshape_and_cache(qo, q, k, v, caches[0], caches[1], pos, slots, f, interleaved=il)
    assert torch.equal(qo, qw) and torch.equal(caches[0], want[0]) and torch.equal(caches[1], want[1])
    assert pkv.read_device_errors() == 0
    # a slot past the pool is skipped and flagged, the others are written
    slots[0] = NB * bs
    pkv.rotary_reshape_and_cache(qo, q, k, v, caches[0], caches[1], pos, slots, f, interleaved=il)
    assert pkv.read_device_errors() == 2
    assert torch.equal(caches[0], want[0]) and torch.equal(caches[1], want[1])
