"""The roundings of an accumulated embedding gradient, bit for bit (one token per row, so that
there is no sum whose order counts)."""
import pytest
import torch

import lm_head_linear_tmem_b200 as flce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [45.25, 0.3, 1.0])
@pytest.mark.parametrize("H", [5, 12, 64, 1000])
@pytest.mark.parametrize("din", [torch.float32, torch.bfloat16])
def test_roundings_of_accumulation(H, din, scale):
    V, N = 300, 200
    g = torch.Generator(device="cuda").manual_seed(H)
    ids = torch.randperm(V, device="cuda", generator=g)[:N]
    d = torch.randn(N, H, device="cuda", generator=g).to(din)
    old = torch.randn(V, H, device="cuda", generator=g)
    s = torch.tensor(scale, dtype=torch.float32, device="cuda")
    got = flce.embedding_backward(d, ids, V, scale=scale, d_weight=old.clone(), accumulate=True)
    want = old.clone()
    want[ids] = old[ids] + d.float() * s  # two fp32 roundings
    assert torch.equal(got, want)
    low = old.to(torch.bfloat16)
    got = flce.embedding_backward(d, ids, V, scale=scale, d_weight=low.clone(), accumulate=True)
    want = low.clone()
    # products of 24 by 24 bits are exact in fp64, and so is their sum with a bf16 of like size
    # to 2^-53: rounded to fp32, then to bf16
    want[ids] = (low[ids].double() + d.double() * s.double()).float().to(torch.bfloat16)
    assert torch.equal(got, want)
    # written, not added: one rounding of the product to fp32
    got = flce.embedding_backward(d, ids, V, scale=scale)
    assert torch.equal(got[ids], d.float() * s)
