"""Batches without tokens through the differentiable calls, with a trained and with a frozen
head."""
import pytest
import torch

import lm_head_linear_tmem_b200 as flce

pytestmark = pytest.mark.gpu


def _loss(h, w, y):
    return flce.fused_linear_cross_entropy(h, w, y)[0]


def _score(h, w, y):
    f = flce.fused_linear_logprobs(h, w, y, top_k=2)
    return f.logprobs.sum() + f.entropy.sum()


@pytest.mark.parametrize("call", [_loss, _score])
@pytest.mark.parametrize("train", ["hidden", "weight", "both"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_tokens(dtype, train, call):
    h = torch.empty(2, 0, 64, device="cuda", dtype=dtype, requires_grad=train != "weight")
    w = torch.randn(300, 64, device="cuda").to(dtype).requires_grad_(train != "hidden")
    y = torch.empty(2, 0, device="cuda", dtype=torch.int64)
    out = call(h, w, y)
    assert float(out.detach()) == 0.0
    out.backward()
    if train != "weight":
        assert h.grad.shape == (2, 0, 64) and h.grad.dtype == dtype
    if train != "hidden":
        assert w.grad.dtype == dtype and torch.all(w.grad == 0)


def test_no_tokens_through_the_embedding():
    w = torch.randn(300, 64, device="cuda", requires_grad=True)
    out = flce.fused_embedding(w, torch.empty(3, 0, device="cuda", dtype=torch.int64))
    assert out.shape == (3, 0, 64)
    out.sum().backward()
    assert torch.all(w.grad == 0)
