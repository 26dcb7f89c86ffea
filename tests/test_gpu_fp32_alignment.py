"""fp32 hidden and weight that start on any element (slices of larger tensors)."""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from oracle import logprobs_ref as ref
from tests import _gpu as G
from tests.test_gpu_logprobs import IGN, check_forward, problem

pytestmark = pytest.mark.gpu


def shifted(t, by):
    """The same values, `by` elements past an aligned address."""
    flat = torch.zeros(t.numel() + by, device="cuda")
    out = flat[by:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == 4 * by % 16 and out.is_contiguous()
    return out


@pytest.mark.parametrize("by_h,by_w", [(1, 0), (0, 2), (3, 1)])
@pytest.mark.parametrize("N,H", [(5, 64), (9, 65), (40, 64), (70, 67)])
def test_shifted_inputs(N, H, by_h, by_w):
    host, (h0, w0, y) = problem(N, H, 700, seed=80 + N, n_ign=N // 5, w_std=0.1, dtype="fp32")
    h, w = shifted(h0, by_h), shifted(w0, by_w)
    got = flce.logprobs_forward(h, w, y, temperature=0.9, top_k=5, check_status=True)
    check_forward(got, host, 0.0, 0.9, 5)
    g = np.random.default_rng(81)
    a, b = (g.standard_normal(N).astype(np.float32) for _ in range(2))
    grads = flce.logprobs_backward(h, w, y, got.saved, torch.from_numpy(a).cuda(),
                                   torch.from_numpy(b).cuda(), temperature=0.9,
                                   check_status=True)
    # fp32 throughout, as test_backward_fp32
    for x, r in zip(grads, ref.backward(*host, a, b, IGN, 0.0, 0.9)):
        assert G.rel_l2(x.cpu().numpy(), r) <= 2e-5
    # the loss reads element by element wherever the rows start
    f, f0 = flce.forward(h, w, y, check_status=True), flce.forward(h0, w0, y)
    for x, z in zip(f, f0):
        assert torch.equal(x, z)
    for x, z in zip(flce.backward(h, w, y, f.lse, check_status=True),
                    flce.backward(h0, w0, y, f0.lse)):
        assert torch.equal(x, z)


def test_rows_of_a_larger_tensor():
    """hidden[1:], with an odd hidden size."""
    host, (h0, w, y) = problem(20, 33, 300, seed=82, dtype="fp32")
    big = torch.zeros(21, 33, device="cuda")
    big[1:] = h0
    got = flce.logprobs_forward(big[1:], w, y, top_k=3, check_status=True)
    check_forward(got, host, top_k=3)
