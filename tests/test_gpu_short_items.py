"""The 16-bit caches on the tensor cores with many short contexts, most of which end
inside a block: several items (chunk attention) and units (decode) of one or two
key tiles follow each other on an SM."""
import random

import pytest
import torch

import paged_kv_cache_480_b200 as pkv
import row_model as rm
from test_gpu_decode_nan import bound, rows_of, same_type_pages

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,D,G,hi", [("f16", 64, 1, 600), ("bf16", 64, 1, 300), ("bf16", 64, 4, 200), ("f16", 128, 1, 400),
                                       ("bf16", 64, 16, 40)])
def test_prompts(dt, D, G, hi):
    rnd, Hkv, bs = random.Random(hi), 16, 16
    lens = [rnd.choice([rnd.randint(1, hi), rnd.randint(1, hi), 16 * rnd.randint(1, max(1, hi // 16))]) for _ in range(40)]
    kc, vc, bt, cl, gc = same_type_pages(lens, Hkv, D, bs, rm.DT[dt], 97)
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    q = torch.randn(sum(lens), G * Hkv, D, generator=gc, device="cuda").to(rm.DT[dt])
    out = torch.empty_like(q)
    pkv.paged_attention_prefill(out, q, kc, vc, bt, cl, start, D ** -0.5, max_query_len=max(lens))
    assert pkv.read_device_errors() == 0
    for s, L in enumerate(lens):
        a = int(start[s])
        ref, logit, top = rm.attend(q[a:a + L], rows_of(kc, bt, s, L, bs), rows_of(vc, bt, s, L, bs), D ** -0.5)
        rm.close(out[a:a + L], ref, bound(ref, logit, top, dt, L))
    again = torch.empty_like(q)
    for _ in range(30):
        again.zero_()
        pkv.paged_attention_prefill(again, q, kc, vc, bt, cl, start, D ** -0.5, max_query_len=max(lens))
        assert torch.equal(again, out)
    assert pkv.read_device_errors() == 0


@pytest.mark.parametrize("dt,D,G,hi", [("f16", 64, 16, 120), ("bf16", 64, 20, 300), ("bf16", 128, 16, 120), ("f16", 64, 130, 200)])
def test_decode(dt, D, G, hi):
    rnd, bs, S = random.Random(hi), 16, 900
    lens = [rnd.choice([rnd.randint(1, hi), rnd.randint(1, hi), 16 * rnd.randint(1, hi // 16)]) for _ in range(S)]
    kc, vc, bt, cl, gc = same_type_pages(lens, 1, D, bs, rm.DT[dt], 98)
    q = torch.randn(S, G, D, generator=gc, device="cuda").to(rm.DT[dt])
    out = torch.empty_like(q)
    pkv.paged_attention_decode(out, q, kc, vc, bt, cl, D ** -0.5)
    assert pkv.read_device_errors() == 0
    for s in range(0, S, 13):
        ref, logit, top = rm.attend(q[s:s + 1], rows_of(kc, bt, s, lens[s], bs), rows_of(vc, bt, s, lens[s], bs), D ** -0.5)
        rm.close(out[s:s + 1], ref, bound(ref, logit, top, dt, lens[s]))
    again = torch.empty_like(q)
    for _ in range(30):
        again.zero_()
        pkv.paged_attention_decode(again, q, kc, vc, bt, cl, D ** -0.5)
        assert torch.equal(again, out)
    assert pkv.read_device_errors() == 0
