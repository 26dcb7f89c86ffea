"""Row orders at the sizes where one way of ordering takes over from another."""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native
from tests import _gpu as G

pytestmark = pytest.mark.gpu
IGN = -100
SIZES = [127, 128, 129, 255, 256, 257, 1023, 1024, 1025, 2047, 2048, 2049, 16384, 16385]


@pytest.mark.parametrize("V", [40, 70000])
@pytest.mark.parametrize("N", SIZES)
def test_embedding_gradient(N, V):
    g = torch.Generator(device="cuda").manual_seed(N)
    ids = torch.randint(0, V, (N,), device="cuda", generator=g)
    ids[::3] = IGN
    ids[N // 2] = V - 1
    d = torch.randint(-4, 5, (N, 8), device="cuda", generator=g).float()  # exact sums
    want = torch.zeros(V, 8, device="cuda").index_add_(0, ids.clamp(min=0), d * (ids != IGN)[:, None])
    assert torch.equal(flce.embedding_backward(d, ids, V, check_status=True), want)


@pytest.mark.parametrize("N", SIZES)
def test_rows_of_the_loss_and_of_scoring(N):
    """With and without the rows left out of the products: the forward's tiles see other rows,
    each row's logits are the same sums."""
    H, V = 16, 300
    g = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn(N, H, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randn(V, H, device="cuda", generator=g).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), device="cuda", generator=g)
    y[torch.randperm(N, device="cuda", generator=g)[:N // 3]] = IGN
    f = flce.forward(h, w, y, check_status=True)
    s = flce.logprobs_forward(h, w, y, top_k=2, check_status=True)
    assert int(f.num_tokens) == int((y != IGN).sum())
    with _native.options(fwd_compact=0):
        f0, s0 = flce.forward(h, w, y), flce.logprobs_forward(h, w, y, top_k=2)
    assert torch.equal(f.lse, f0.lse) and torch.equal(s.top_ids, s0.top_ids)
    for a, b in zip(s[:3], s0[:3]):
        assert float((a - b).abs().max()) <= 2.0 ** -18  # (runs of tiles are cut otherwise)
    dh, dw = flce.backward(h, w, y, f.lse, check_status=True)
    z = torch.softmax(h.double() @ w.double().t(), -1)
    z[torch.arange(N, device="cuda"), y.clamp(min=0)] -= 1.0
    z *= (y != IGN)[:, None]
    # dZ in bf16: 2^-8 of an entry at most
    assert G.rel_l2(dh.cpu().numpy(), (z @ w.double()).cpu().numpy()) <= 2.0 ** -8
    assert G.rel_l2(dw.cpu().numpy(), (z.t() @ h.double()).cpu().numpy()) <= 2.0 ** -8
    assert np.all(dh[y == IGN].cpu().numpy() == 0.0)
