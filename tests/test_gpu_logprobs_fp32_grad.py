"""fp32 gradients of the scoring operator: odd sizes, accumulation, bf16 results.  fp32
throughout: each p is off by its fp32 logits' rounding (H products: some 1e-6 here) and the
sums by 2^-24 of what they add, 2e-5 relative in all; a bf16 result rounds once more, by 2^-8 of
each entry at most, and accumulating adds one rounding of the sum."""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from oracle import logprobs_ref as ref
from tests import _gpu as G
from tests.test_gpu_logprobs import IGN, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap,T", [(0.0, 1.0), (4.0, 0.7)])
@pytest.mark.parametrize("N,H,V", [(1, 8, 5), (2, 13, 300), (18, 67, 1025), (70, 202, 513),
                                   (300, 33, 1100)])
def test_sizes_accumulation_and_bf16_results(N, H, V, softcap, T):
    host, dev = problem(N, H, V, seed=90 + N, n_ign=N // 5, w_std=0.1, dtype="fp32")
    g = np.random.default_rng(91)
    a, b = (g.standard_normal(N).astype(np.float32) for _ in range(2))
    up = [torch.from_numpy(t).cuda() for t in (a, b)]
    kw = dict(softcap=softcap, temperature=T)
    f = flce.logprobs_forward(*dev, **kw)
    want = ref.backward(*host, a, b, IGN, softcap, T)
    got = flce.logprobs_backward(*dev, f.saved, *up, check_status=True, **kw)
    for x, r in zip(got, want):
        assert G.rel_l2(x.cpu().numpy(), r) <= 2e-5
    assert np.all(got[0].cpu().numpy()[host[2] == IGN] == 0.0)
    again = flce.logprobs_backward(*dev, f.saved, *up, **kw)
    base = [torch.randn_like(x) for x in got]
    acc = flce.logprobs_backward(*dev, f.saved, *up, d_hidden=base[0].clone(),
                                 d_weight=base[1].clone(), accumulate_d_hidden=True,
                                 accumulate_d_weight=True, **kw)
    low = flce.logprobs_backward(*dev, f.saved, *up, grad_dtype=torch.bfloat16, **kw)
    for x, y, z, s, o in zip(got, again, base, acc, low):
        assert torch.equal(x, y)
        assert torch.equal(s, z + x)
        assert torch.equal(o, x.to(torch.bfloat16))
    only, none = flce.logprobs_backward(*dev, f.saved, *up, compute_d_weight=False, **kw)
    assert none is None and torch.equal(only, got[0])
