"""Decode with a softmax scale of zero and of either sign: groups that the
tensor-core kernel takes for a positive one, and smaller ones."""
import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from test_gpu_decode_nan import bound, rows_of, same_type_pages
from test_gpu_row_cache import check_decode

pytestmark = pytest.mark.gpu

LENS = [1, 70, 128, 300, 1000]


@pytest.mark.parametrize("scale", [0.0, -0.125, 0.125])
@pytest.mark.parametrize("dt,G,D,bs", [("f16", 20, 64, 16), ("bf16", 20, 128, 32), ("f16", 130, 64, 32), ("bf16", 8, 128, 16),
                                       ("f16", 1, 64, 16), ("f32", 2, 64, 16)])
def test_over_row_caches(dt, G, D, bs, scale):
    check_decode(LENS, 2 * G, 2, D, bs, dt, seed=60, scale=scale)


@pytest.mark.parametrize("scale", [0.0, -0.125, 0.125])
@pytest.mark.parametrize("dt,G,D,bs", [("f16", 20, 64, 16), ("bf16", 16, 128, 32), ("bf16", 130, 64, 32), ("f16", 8, 128, 16)])
def test_over_caches_of_the_same_type(dt, G, D, bs, scale):
    kc, vc, bt, cl, gc = same_type_pages(LENS, 2, D, bs, rm.DT[dt], 61)
    q = torch.randn(len(LENS), 2 * G, D, generator=gc, device="cuda").to(rm.DT[dt])
    out = torch.empty_like(q)
    pkv.paged_attention_decode(out, q, kc, vc, bt, cl, scale)
    for s, L in enumerate(LENS):
        ref, logit, top = rm.attend(q[s:s + 1], rows_of(kc, bt, s, L, bs), rows_of(vc, bt, s, L, bs), scale)
        rm.close(out[s:s + 1], ref, bound(ref, logit, top, dt, L))
    assert pkv.read_device_errors() == 0
