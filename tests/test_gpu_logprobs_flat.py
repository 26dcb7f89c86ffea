"""Scoring fp32 rows whose probability is spread over the whole vocabulary at logits of 100: the
sum is what the listed logits leave, and nothing but rounding to nearest is in it.

Tolerance of a log probability of size log V: its own rounding 2^-24 log V, 2^-21 for the
exponentials and the sums, and the mean over V logits of their rounding errors: H additions
a logit, of partial sums that grow to 100, each off by a half step at most (a deviation of
2^-24 / sqrt 3 of the partial sum, whose root mean square is 100 / sqrt 3), signs as good as random:
sqrt(H) 2^-24 100 / 3 a logit, over sqrt(V); four of those.
"""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("top_k", [0, 1, 4])
@pytest.mark.parametrize("N,H", [(8, 1000), (8, 1001), (64, 1000)])
def test_flat_fp32_rows(N, H, top_k, sign):
    V = 32000
    g = torch.Generator(device="cuda").manual_seed(60 + N)
    h = 0.5 + torch.rand(N, H, device="cuda", generator=g)
    w = sign * (0.1 + 0.03 * torch.randn(V, H, device="cuda", generator=g) / np.sqrt(H))
    y = torch.randint(0, V, (N,), device="cuda", generator=g)
    f = flce.logprobs_forward(h, w, y, top_k=top_k)
    z = h.double() @ w.double().t()
    logp = torch.log_softmax(z, -1)
    want = logp.gather(1, y[:, None])[:, 0]
    log_v = float(want.abs().max())
    tol = 2.0 ** -24 * log_v + 2.0 ** -21 + 4 * np.sqrt(H / V) * 2.0 ** -24 * float(z.abs().max()) / 3
    err = (f.logprobs.double() - want).abs().max()
    assert float(err) <= tol, (float(err), tol)
    ent = -(logp.exp() * logp).sum(-1)
    assert float((f.entropy.double() - ent).abs().max()) <= 2 * tol
