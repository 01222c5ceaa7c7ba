"""Rotary, 8-bit row cache and read-back calls on the host (CPU only): what
they refuse before any launch, the frequency table against closed forms, and
the 64-bit model that the GPU tests compare with against hand-made values."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_480_b200 as pkv
from paged_kv_cache_480_b200 import binding
from paged_kv_cache_480_b200 import build as pkv_build
import row_model as rm

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return binding.load_library()


def call(fn, names, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*[P(a[n]) if n in ("qo", "ko", "q", "k", "v", "kc", "vc", "pos", "sm", "f", "bt", "sl", "cl", "qsl", "out", "ws")
                else a[n] for n in names], None)


ROT = dict(qo=16, ko=16, q=16, k=16, pos=16, f=16, t=4, h=4, hkv=2, d=64, rot=64, il=0, att=1.0, sqo=256, sko=128,
           sq=256, sk=128, dtype=2)


def test_rotary_embedding_refusals(lib):
    def r(**kw):
        return call(lib.rotary_embedding, ROT, ROT, **kw)
    # (fake pointers: every call here fails its checks, or has nothing to do)
    assert r(t=0) == 0 and r(t=0, q=0) == 0
    assert r(h=0, hkv=0) == 0
    assert r(t=-1) == 1 and r(h=-1) == 1
    assert r(rot=0) == 1 and r(rot=-2) == 1 and r(rot=63) == 1 and r(rot=66) == 1
    assert r(d=0) == 2 and r(d=24) == 2 and r(d=528) == 2
    assert r(dtype=7) == 2
    assert r(att=math.nan) == 1 and r(att=math.inf) == 1
    assert r(pos=0) == 1 and r(f=0) == 1 and r(pos=4) == 1 and r(f=2) == 1
    for n in ("q", "k", "qo", "ko"):
        assert r(**{n: 0}) == 1 and r(**{n: 8}) == 1
    for n, row in (("sq", 256), ("sk", 128), ("sqo", 256), ("sko", 128)):
        assert r(**{n: row - 8}) == 1 and r(**{n: row + 4}) == 1


WRITE = dict(qo=16, q=16, k=16, v=16, kc=16, vc=16, pos=16, sm=16, f=16, t=4, h=4, hkv=2, d=64, rot=64, il=0, att=1.0,
             bs=16, nb=8, sqo=256, sq=256, sk=128, sv=128, dtype=2)


@pytest.mark.parametrize("name", ["rotary_reshape_and_cache", "rotary_reshape_and_cache_fp8row"])
def test_rotary_write_refusals(lib, name):
    def w(**kw):
        return call(getattr(lib, name), WRITE, WRITE, **kw)
    assert w(t=0) == 0
    assert w(hkv=0) == 1 and w(nb=0) == 1 and w(rot=0) == 1 and w(rot=80) == 1
    assert w(d=96, rot=64) == 2 and w(bs=8) == 2 and w(dtype=-1) == 2
    for n in ("q", "qo", "k", "v", "kc", "vc", "pos", "sm", "f"):
        assert w(**{n: 0}) == 1, n
    for n in ("q", "qo", "k", "v", "kc", "vc"):
        assert w(**{n: 8}) == 1, n
    assert w(sk=124) == 1 and w(sv=120) == 1 and w(sq=252) == 1


def test_quantising_write_refusals(lib):
    d = dict(k=16, v=16, kc=16, vc=16, sm=16, t=4, hkv=2, d=64, bs=16, nb=8, sk=128, sv=128, dtype=0)

    def w(**kw):
        return call(lib.reshape_and_cache_fp8row, d, d, **kw)
    assert w(t=0) == 0 and w(t=-1) == 1 and w(hkv=0) == 1 and w(nb=-1) == 1
    assert w(d=80) == 2 and w(bs=64) == 2 and w(dtype=3) == 2
    assert w(k=0) == 1 and w(sm=4) == 1 and w(sk=126) == 1 and w(sv=64) == 1


def test_gather_refusals(lib):
    d = dict(ko=16, vo=16, kc=16, vc=16, bt=16, sl=16, t=4, s=2, hkv=2, d=64, bs=16, nb=8, mb=4, dtype=2)

    def g(fn=lib.gather_cache, **kw):
        a = dict(d)
        a.update(kw)
        a["vo"] = P(a["vo"])
        names = list(d)
        if fn is lib.gather_cache_fp8kv:
            names = names[:6] + ["ks", "vs"] + names[6:]
            a.setdefault("ks", 1.0)
            a.setdefault("vs", 1.0)
        return call(fn, names, a)
    for fn in (lib.gather_cache, lib.gather_cache_fp8kv, lib.gather_cache_fp8row):
        assert g(fn, t=0) == 0
        assert g(fn, t=-1) == 1 and g(fn, s=0) == 1 and g(fn, hkv=0) == 1 and g(fn, nb=0) == 1 and g(fn, mb=0) == 1
        assert g(fn, d=32) == 2 and g(fn, bs=24) == 2 and g(fn, dtype=9) == 2
        for n in ("ko", "vo", "kc", "vc", "bt", "sl"):
            assert g(fn, **{n: 0}) == 1
        assert g(fn, ko=8) == 1 and g(fn, bt=2) == 1
    assert g(lib.gather_cache_fp8kv, ks=0.0) == 1 and g(lib.gather_cache_fp8kv, vs=math.nan) == 1


def test_row_attention_refusals(lib):
    d = dict(out=16, q=16, kc=16, vc=16, bt=16, cl=16, scale=0.1, hkv=4, bs=16, s=2, h=4, d=64, nb=8, mb=4, ctx=64,
             dtype=2, ps=0, ws=16, wsb=1 << 20)

    def a(**kw):
        return call(lib.paged_attention_decode_fp8row, d, d, **kw)
    assert a(out=0) == 1 and a(kc=8) == 1 and a(d=96) == 2 and a(bs=8) == 2 and a(h=6) == 2 and a(dtype=5) == 2
    assert a(ctx=100) == 1 and a(ps=40) == 1 and a(ws=0) == 6 and a(wsb=64) == 6 and a(scale=math.nan) == 1
    d = dict(out=16, q=16, kc=16, vc=16, bt=16, cl=16, qsl=16, scale=0.1, t=40, s=2, h=4, hkv=4, d=64, bs=16, nb=8,
             mb=4, mq=32, dtype=2)

    def p(**kw):
        return call(lib.paged_attention_prefill_fp8row, d, d, **kw)

    def p8(**kw):
        x = dict(d, ks=1.0, vs=1.0)
        x.update(kw)
        return call(lib.paged_attention_prefill_fp8kv, list(d)[:8] + ["ks", "vs"] + list(d)[8:], x)
    for f in (p, p8):
        assert f(t=0, mq=0) == 0
        assert f(out=0) == 1 and f(q=8) == 1 and f(qsl=0) == 1 and f(mq=41) == 1 and f(mq=0) == 1
        assert f(dtype=0) == 2 and f(d=96) == 2 and f(bs=8) == 2 and f(h=256, hkv=1) == 2
        assert f(scale=0.0) == 1 and f(scale=-1.0) == 1 and f(scale=math.nan) == 1
    assert p8(ks=0.0) == 1 and p8(vs=-1.0) == 1 and p8(ks=math.inf) == 1 and p8(scale=1e-30, ks=1e-30) == 1


# ---- the binding's own checks (CPU tensors never reach the library) ---------
def test_binding_refuses_cpu_tensors_and_mismatched_shapes():
    q = torch.zeros(2, 4, 64)
    f = torch.ones(32)
    pos = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkv.rotary_embedding(torch.empty_like(q), None, q, None, pos, f)          # not on a GPU
    with pytest.raises(ValueError):
        pkv.rotary_embedding(torch.empty_like(q), None, q, q, pos, f)             # k without k_out
    with pytest.raises(ValueError):
        pkv.rotary_embedding(torch.empty(2, 4, 32), None, q, None, pos, f)
    cache = torch.zeros(pkv.fp8row_cache_shape(4, 2, 16, 64), dtype=torch.uint8)
    assert cache.shape == (4, 2, 16 * 65)
    with pytest.raises(TypeError):
        pkv.reshape_and_cache_fp8row(q, q, cache.float(), cache.float(), pos)
    with pytest.raises(ValueError):
        pkv.reshape_and_cache_fp8row(q[:, :2], q[:, :2], cache[..., :-1], cache[..., :-1], pos)
    with pytest.raises(ValueError):
        pkv.gather_cache_fp8row(q[:, :2], q[:, :2], cache, cache, torch.zeros(1, 1, dtype=torch.int32),
                                torch.zeros(3, dtype=torch.int32))


# ---- frequencies ----------------------------------------------------------
def test_frequencies_plain_linear_and_base():
    f, att = pkv.rotary_frequencies(64)
    want = 10000.0 ** (-2.0 * np.arange(32) / 64)
    assert att == 1.0 and f.dtype == torch.float32 and np.array_equal(f.numpy(), want.astype(np.float32))
    g, _ = pkv.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert np.array_equal(g.numpy(), (want / 4).astype(np.float32))
    h, _ = pkv.rotary_frequencies(64, scaling="base", factor=4.0)
    assert h[0] == 1.0 and abs(h[-1] * 4 / f[-1] - 1) < 1e-6          # fastest kept, slowest divided by the factor
    one, _ = pkv.rotary_frequencies(2, scaling="base", factor=4.0)
    assert one.tolist() == [1.0]


def test_frequencies_by_parts():
    ctx, factor = 8192, 8.0
    f = 10000.0 ** (-2.0 * np.arange(64) / 128)
    turns = ctx * f / (2 * math.pi)
    g, att = pkv.rotary_frequencies(128, scaling="by_turns", factor=factor, original_context=ctx, fast_turns=4.0)
    g = g.double().numpy()
    assert att == 1.0
    assert np.allclose(g[turns > 4], f[turns > 4], rtol=1e-7) and np.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-7)
    mid = (turns >= 1) & (turns <= 4)
    keep = (turns[mid] - 1) / 3
    assert mid.any() and np.allclose(g[mid], f[mid] * (keep + (1 - keep) / 8), rtol=1e-6)
    g, att = pkv.rotary_frequencies(128, scaling="by_index", factor=factor, original_context=ctx)
    g = g.double().numpy()
    assert abs(att - (0.1 * math.log(8) + 1)) < 1e-6
    at = [128 * math.log(ctx / (2 * math.pi * t)) / (2 * math.log(10000.0)) for t in (32.0, 1.0)]
    low, high = math.floor(at[0]), math.ceil(at[1])
    ramp = np.clip((np.arange(64) - low) / (high - low), 0, 1)
    assert np.allclose(g, f * ((1 - ramp) + ramp / 8), rtol=1e-6)


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=5), dict(rotary_dim=-2), dict(rotary_dim=8, base=1.0),
                                dict(rotary_dim=8, base=math.nan), dict(rotary_dim=8, scaling="linear", factor=0.5),
                                dict(rotary_dim=8, scaling="base", factor=math.inf),
                                dict(rotary_dim=8, scaling="by_turns", factor=2.0),
                                dict(rotary_dim=8, scaling="by_index", factor=2.0, original_context=64, fast_turns=1.0,
                                     slow_turns=1.0)])
def test_frequency_refusals(kw):
    with pytest.raises(pkv.PagedKVError):
        pkv.rotary_frequencies(**kw)


def test_frequency_scaling_name():
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(8, scaling="twice")


# ---- the model -------------------------------------------------------------
def test_model_rows():
    D = 64
    x = torch.zeros(9, D, dtype=torch.float64)
    x[0, :3] = torch.tensor([448.0, -1.0, 0.4])
    x[1, 0] = 448.0 * (1 + 2.0 ** -20)                  # just above: the next exponent
    x[2, 0] = 3.0
    x[3, 0], x[3, 1] = math.inf, 1.0
    x[4, 0], x[4, 1] = math.nan, 1.0
    x[5, 0] = 1e-30
    x[6, 0] = -1e38
    x[7, :2] = torch.tensor([224.0, 17.0])              # e = -1: 34 lies between the codes 32 and 36, the even one is 32
    codes, b = rm.quantise(x)
    assert b.tolist() == [127, 128, 127 - 7, 187, 255, 67, 187, 126, 67]
    v = rm.value(codes, b)
    assert v[0, 0] == 448.0 and v[0, 1] == -1.0 and abs(float(v[0, 2]) - 0.4) <= 0.4 * 2.0 ** -4
    assert v[2, 0] == 3.0 and v[3, 0] == 448.0 * 2.0 ** 60 and v[3, 1] == 0.0
    assert v[4].isnan().all() and v[5, 0] == 0.0 and v[6, 0] == -448.0 * 2.0 ** 60
    assert v[7, 0] == 224.0 and v[7, 1] == 16.0 and (v[8] == 0).all()


def test_model_rotation_is_a_rotation():
    x = torch.randn(5, 3, 32, dtype=torch.float64)
    pos = torch.arange(5)
    f, _ = pkv.rotary_frequencies(32)
    for il in (False, True):
        y = rm.rotate(x, pos, f, il)
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1))
        assert torch.equal(y[0], x[0])
        # q . k depends on the distance of the positions alone
        a = (rm.rotate(x, pos, f, il) * rm.rotate(x.flip(0), pos + 3, f, il)).sum(-1)
        c = (rm.rotate(x, pos + 100, f, il) * rm.rotate(x.flip(0), pos + 103, f, il)).sum(-1)
        assert torch.allclose(a, c)
