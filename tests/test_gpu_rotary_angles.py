"""How exact the angles of the rotary kernels are."""
import pytest
import torch

import paged_kv_cache_480_b200 as pkv
from test_gpu_rotary import gen_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [4096, 1 << 20])
def test_cosines_and_sines_are_rounded_about_once(far):
    """The rotation of (1, 0) in fp32 is (cos, sin).  Rounding a value of [0, 1]
    spread as cosines are costs 1.5e-8 rms; two such roundings, 2.1e-8.  An
    angle that is narrowed to fp32 first costs 3.3e-8."""
    T, D = 20000, 128
    g = gen_of(90)
    pos = torch.randint(0, far, (T,), generator=g, device="cuda")
    f = pkv.rotary_frequencies(D)[0].cuda()
    x = torch.zeros(T, 1, D, device="cuda")
    x[..., :D // 2] = 1.0
    out = torch.empty_like(x)
    pkv.rotary_embedding(out, None, x, None, pos, f)
    a = pos.double()[:, None, None] * f.double()
    for got, want in ((out[..., :D // 2], a.cos()), (out[..., D // 2:], a.sin())):
        err = got.double() - want
        assert float(err.square().mean().sqrt()) < 2.5e-8
        assert float(err.abs().max()) < 2.0 ** -23          # a step of sincospi at most and half of one
