"""fp32 scoring where the kernel of few rows hands over to the one of more."""
import pytest

import lm_head_linear_tmem_b200 as flce
from tests.test_gpu_logprobs import check_forward, problem


@pytest.mark.gpu
@pytest.mark.parametrize("N", [16, 17, 24, 25])
@pytest.mark.parametrize("H", [511, 512, 1001, 3536, 3537, 4000])
def test_rows_at_the_border(N, H):
    host, dev = problem(N, H, 150, seed=N + H, n_ign=N // 5, w_std=0.1, dtype="fp32")
    got = flce.logprobs_forward(*dev, temperature=0.8, top_k=4, check_status=True)
    check_forward(got, host, 0.0, 0.8, 4)
