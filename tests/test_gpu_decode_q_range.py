"""Decode over E4M3 caches with bf16 q of any size: heads far below and beyond
fp16's range, beside one another in a group."""
import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from test_gpu_decode_nan import rows_of, same_type_pages
from test_gpu_rotary import gen_of
from test_gpu_row_cache import check_decode

pytestmark = pytest.mark.gpu

LENS = [1, 17, 33, 300, 1000]


@pytest.mark.parametrize("G,D,bs", [(1, 64, 16), (2, 128, 16), (4, 128, 32), (7, 64, 32), (16, 128, 16), (20, 64, 16)])
@pytest.mark.parametrize("size", [1e-30, 1e-8, 1e-6, 1e5, 1e15])
def test_over_row_caches(G, D, bs, size):
    q = (torch.randn(len(LENS), 2 * G, D, generator=gen_of(80), device="cuda") * size).bfloat16()
    # (K of the other size; past the format's 2^60 the softmax scale takes the rest)
    k = min(max(1.0 / size, 1e-16), 1e16)
    check_decode(LENS, 2 * G, 2, D, bs, "bf16", seed=80, q=q, scale=D ** -0.5 / (size * k), kscale=lambda x, g: x * k)


@pytest.mark.parametrize("G", [2, 8])
def test_heads_of_different_sizes_in_a_group(G):
    q = torch.randn(len(LENS), 2 * G, 128, generator=gen_of(81), device="cuda")
    q *= torch.tensor([1e-8, 1.0, 1e-6, 1e5, 1e-3, 0.0, 300.0, 1e-5], device="cuda")[:G].repeat(2)[None, :, None]
    q[:, :, ::3] *= 1e-3                                   # and elements of different sizes in a head
    check_decode(LENS, 2 * G, 2, 128, 16, "bf16", seed=81, q=q.bfloat16(), scale=1e-2)


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("size", [1e-8, 1e-6, 1e5])
def test_over_per_tensor_caches(G, size):
    D, bs = 64, 16
    kc, vc, bt, cl, gc = same_type_pages(LENS, 2, D, bs, torch.float32, 82)
    k8, v8 = (x.to(torch.float8_e4m3fn) for x in (kc, vc))
    q = (torch.randn(len(LENS), 2 * G, D, generator=gc, device="cuda") * size).bfloat16()
    out = torch.empty_like(q)
    ks = float(torch.tensor(1.0 / size, dtype=torch.float32))
    pkv.paged_attention_decode_fp8kv(out, q, k8, v8, bt, cl, D ** -0.5, ks, 1.0)
    for s, L in enumerate(LENS):
        K, V = rows_of(k8.double() * ks, bt, s, L, bs), rows_of(v8.double(), bt, s, L, bs)
        ref, logit, top = rm.attend(q[s:s + 1], K, V, D ** -0.5)
        rm.close(out[s:s + 1], ref, rm.attention_bound(ref, logit, top, torch.bfloat16, torch.float16, L))
    assert pkv.read_device_errors() == 0
