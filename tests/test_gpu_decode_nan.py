"""Decode where NaN or infinite logits fill whole partitions of a context, for
every consumer and cache kind, against the 64-bit form."""
import math

import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from test_gpu_rotary import gen_of
from test_gpu_row_cache import check_decode

pytestmark = pytest.mark.gpu

LENS = [40, 193, 700, 3000, 1]
CONSUMERS = [("f32", 1, 64, 16), ("f32", 8, 128, 32), ("f16", 1, 128, 16), ("bf16", 2, 64, 32), ("bf16", 4, 128, 32),
             ("f16", 8, 64, 16), ("bf16", 16, 128, 16), ("bf16", 17, 128, 16), ("f16", 64, 64, 32)]


def a_nan_head(G, D, dt, seed):
    q = torch.randn(len(LENS), 2 * G, D, generator=gen_of(seed), device="cuda").to(rm.DT[dt])
    q[:, G // 2, 3] = math.nan                       # one head of the first KV head's group
    return q


@pytest.mark.parametrize("dt,G,D,bs", CONSUMERS)
def test_a_nan_in_q_over_row_caches(dt, G, D, bs):
    q = a_nan_head(G, D, dt, 50)
    out, _ = check_decode(LENS, 2 * G, 2, D, bs, dt, seed=50, q=q)
    assert out[:, G // 2].isnan().all()


@pytest.mark.parametrize("dt,G,D,bs", CONSUMERS)
@pytest.mark.parametrize("which", ["kscale", "vscale"])
def test_partitions_of_nan_rows(dt, G, D, bs, which):
    """Rows 192 and on of one head, among them whole partitions and (193 tokens)
    a partition of one; and rows 600 to 1400 of the longest."""
    def rows(x, g):
        x = x.clone()
        if x.shape[0] == 193:
            x[192:, 0] = math.nan
        if x.shape[0] == 3000:
            x[600:1400, 1, 5] = math.nan
        return x
    out, _ = check_decode(LENS, 2 * G, 2, D, bs, dt, seed=51, **{which: rows})
    assert out[1, :G].isnan().all() and out[3, G:].isnan().all() and out[1, G:].isfinite().all()
    assert out[3, :G].isfinite().all() and out[[0, 2, 4]].isfinite().all()


def same_type_pages(lens, Hkv, D, bs, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    bt, NB = rm.pages(lens, bs, g)
    gc = gen_of(seed)
    kc, vc = (torch.randn(NB, Hkv, bs, D, generator=gc, device="cuda").to(dtype) for _ in range(2))
    return kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), gc


def rows_of(cache, bt, s, L, bs):
    t = torch.arange(L, device="cuda")
    return cache[bt[s, t // bs].long(), :, t % bs].double()


def bound(ref, logit, top, dt, L):
    weights = None if dt == "f32" else rm.DT[dt]
    extra = 2.0 ** -25 if dt == "f16" else 0.0       # (outputs below 2^-14)
    return rm.attention_bound(ref, logit, top, rm.DT[dt], weights, L) + extra


@pytest.mark.parametrize("dt,G,D,bs", [("f32", 1, 128, 16), ("f16", 1, 64, 16), ("bf16", 4, 128, 32), ("f16", 8, 128, 16),
                                       ("bf16", 16, 128, 16), ("f16", 40, 64, 32)])
def test_a_nan_in_q_over_caches_of_the_same_type(dt, G, D, bs):
    kc, vc, bt, cl, gc = same_type_pages(LENS, 2, D, bs, rm.DT[dt], 52)
    q = a_nan_head(G, D, dt, 52)
    out = torch.empty_like(q)
    pkv.paged_attention_decode(out, q, kc, vc, bt, cl, D ** -0.5)
    for s, L in enumerate(LENS):
        ref, logit, top = rm.attend(q[s:s + 1], rows_of(kc, bt, s, L, bs), rows_of(vc, bt, s, L, bs), D ** -0.5)
        rm.close(out[s:s + 1], ref, bound(ref, logit, top, dt, L))
    assert out[:, G // 2].isnan().all() and pkv.read_device_errors() == 0


@pytest.mark.parametrize("dt,G", [("f32", 1), ("f16", 1), ("bf16", 8)])
def test_a_nan_in_q_over_per_tensor_caches(dt, G):
    D, bs = 128, 16
    kc, vc, bt, cl, gc = same_type_pages(LENS, 2, D, bs, torch.float32, 53)
    k8, v8 = (x.to(torch.float8_e4m3fn) for x in (kc, vc))
    q = a_nan_head(G, D, dt, 53)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_fp8kv(out, q, k8, v8, bt, cl, D ** -0.5, 1.0, 1.0)
    for s, L in enumerate(LENS):
        ref, logit, top = rm.attend(q[s:s + 1], *(rows_of(c.double(), bt, s, L, bs) for c in (k8, v8)), D ** -0.5)
        rm.close(out[s:s + 1], ref, rm.attention_bound(ref, logit, top, rm.DT[dt], None if dt == "f32" else torch.float16, L))
    assert pkv.read_device_errors() == 0


@pytest.mark.parametrize("dt,G,D,bs", [("f32", 1, 128, 16), ("f16", 2, 64, 16), ("bf16", 4, 128, 32), ("f16", 8, 128, 16)])
def test_keys_with_a_logit_of_minus_infinity(dt, G, D, bs):
    """They take no weight: whole partitions of them, and the first tokens of one."""
    lens = [900, 2000, 3]
    kc, vc, bt, cl, gc = same_type_pages(lens, 2, D, bs, rm.DT[dt], 54)
    q = torch.randn(3, 2 * G, D, generator=gc, device="cuda").to(rm.DT[dt])
    q[..., 0] = 1.0
    gone = {0: range(0, 40), 1: list(range(20)) + list(range(500, 1700)), 2: range(1)}
    for s, ts in gone.items():
        t = torch.tensor(list(ts), device="cuda")
        rows = torch.zeros(len(t), 2, D, device="cuda", dtype=rm.DT[dt])
        rows[..., 0] = -math.inf
        kc[bt[s, t // bs].long(), :, t % bs] = rows
    out = torch.empty_like(q)
    pkv.paged_attention_decode(out, q, kc, vc, bt, cl, D ** -0.5)
    for s, L in enumerate(lens):
        keep = [t for t in range(L) if t not in set(gone[s])]
        ref, logit, top = rm.attend(q[s:s + 1], rows_of(kc, bt, s, L, bs)[keep], rows_of(vc, bt, s, L, bs)[keep], D ** -0.5)
        rm.close(out[s:s + 1], ref, bound(ref, logit, top, dt, L))
