"""The scoring operator without a GPU: the oracle's gradients against differences,
and the argument checks of the C ABI and of the PyTorch binding."""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native, build
from oracle import logprobs_ref as ref

FAKE = 0x10000  # a 256-aligned, never-dereferenced address for argument-check tests
ARG, SHAPE, WS = 1, 2, 7


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


@pytest.mark.parametrize("softcap,temperature", [(0.0, 1.0), (0.0, 0.6), (2.0, 1.0), (3.0, 1.7)])
def test_oracle_gradient_agrees_with_differences(softcap, temperature):
    g = np.random.default_rng(3)
    N, H, V = 4, 5, 9
    h, w = g.standard_normal((N, H)), 0.7 * g.standard_normal((V, H))
    y = np.array([2, -100, 8, 0])
    a, b = g.standard_normal(N), g.standard_normal(N)

    def value(h, w):
        f = ref.forward(h, w, y, softcap=softcap, temperature=temperature)
        return (a * f["logprobs"] + b * f["entropy"]).sum()

    dh, dw = ref.backward(h, w, y, a, b, softcap=softcap, temperature=temperature)
    eps = 1e-5
    # central differences: eps^2 of curvature (third derivatives below 1e2 here) and
    # 2^-53 / eps of rounding of values of about 10, so 1e-8 + 1e-10
    for x, dx in ((h, dh), (w, dw)):
        for i in np.ndindex(*x.shape):
            up, down = x.copy(), x.copy()
            up[i] += eps
            down[i] -= eps
            args = ((up, w), (down, w)) if x is h else ((h, up), (h, down))
            assert abs((value(*args[0]) - value(*args[1])) / (2 * eps) - dx[i]) < 2e-8


def test_oracle_against_torch_on_plain_rows():
    g = np.random.default_rng(4)
    h, w = g.standard_normal((6, 7)), g.standard_normal((11, 7))
    y = np.array([0, 10, 3, -100, 5, 11])
    f = ref.forward(h, w, y, top_k=4)
    lp = torch.log_softmax(torch.from_numpy(h @ w.T), -1)
    live = [0, 1, 2, 4]
    assert np.allclose(f["logprobs"][live], lp[live, y[live]].numpy(), atol=1e-14)
    assert np.all(f["logprobs"][[3, 5]] == 0) and np.all(f["top_ids"][[3, 5]] == -1)
    assert np.array_equal(f["top_ids"][live], lp.topk(4).indices.numpy()[live])
    assert np.allclose(f["entropy"][live], torch.distributions.Categorical(
        logits=lp).entropy().numpy()[live], atol=1e-14)


def test_workspace_bytes(lib):
    ws = lib.flce_logprobs_workspace_bytes
    assert ws(-1, 64, 512, 0, 0) == 0
    assert ws(4, 4, 512, 0, 0) == 0
    assert ws(4, 68, 512, 0, 0) == 0 and ws(4, 68, 512, 1, 0) > 0
    assert ws(4, 64, 0, 0, 0) == 0
    assert ws(4, 64, 512, 2, 0) == 0
    assert ws(4, 64, 512, 0, -1) == 0
    assert ws(4, 64, 512, 0, 33) == 0
    assert ws(4, 64, 8, 0, 9) == 0 and ws(4, 64, 8, 0, 8) > 0
    assert ws(1 << 20, 64, 1 << 30, 0, 0) == 0   # tile indices past 2^26
    assert ws(131071, 64, 512, 1, 0) == 0        # fp32: rows past the grid's second dimension
    for n, top_k in ((1, 0), (1, 32), (129, 0), (5000, 8)):
        assert ws(n, 64, 512, 0, top_k) % 256 == 0
    assert ws(5000, 64, 512, 0, 8) > ws(5000, 64, 512, 0, 0)
    assert ws(0, 64, 512, 0, 4) > 0
    # longer runs of tiles bound the lists: at most 16 tiles of 256 columns (softcap), so 512 / 16
    # runs and about 10 short ones, two lists of 96 entries each for 16384 rows: 1.06e9 bytes,
    # and the rows' hidden states, 1.3e8
    assert ws(16384, 4096, 131072, 0, 32) < 5 << 28
    assert ws(4096, 4096, 131072, 0, 8) < 700 << 20


def _fwd(lib, N=64, H=64, V=512, softcap=0.0, temperature=1.0, top_k=4, dtype=0, hidden=FAKE,
         weight=FAKE, tokens=FAKE, logprobs=FAKE, entropy=FAKE, lse=FAKE, saved=FAKE, top=FAKE, ids=FAKE,
         ws=FAKE, ws_size=None):
    if ws_size is None:
        ws_size = lib.flce_logprobs_workspace_bytes(N, H, V, dtype, top_k) or 1 << 30
    return lib.flce_logprobs_forward(hidden, weight, tokens, N, H, V, -100, softcap, temperature,
                                     top_k, dtype, logprobs, entropy, lse, saved, top, ids, ws,
                                     ws_size,
                                     None)


def test_forward_refusals(lib):
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-31, 1e31):
        assert _fwd(lib, temperature=bad) == ARG
    for bad in (-1.0, float("nan"), float("inf")):
        assert _fwd(lib, softcap=bad) == ARG
    for bad in (-1, 33):
        assert _fwd(lib, top_k=bad) == ARG
    assert _fwd(lib, V=3, top_k=4) == ARG
    assert _fwd(lib, dtype=2) == ARG
    assert _fwd(lib, H=68) == SHAPE
    assert _fwd(lib, N=-1) == SHAPE
    assert _fwd(lib, V=0, top_k=0) == SHAPE
    assert _fwd(lib, H=12296, dtype=1) == SHAPE
    for name in ("hidden", "weight", "entropy", "lse", "saved", "top", "ids", "ws"):
        assert _fwd(lib, **{name: None}) == ARG, name
    # tokens and their log probabilities go together
    assert _fwd(lib, tokens=None) == ARG
    assert _fwd(lib, logprobs=None) == ARG
    assert _fwd(lib, weight=FAKE + 8) == ARG
    assert _fwd(lib, tokens=FAKE + 4) == ARG
    assert _fwd(lib, ids=FAKE + 4) == ARG
    assert _fwd(lib, ws=FAKE + 128) == ARG
    assert _fwd(lib, ws_size=256) == WS


def _bwd(lib, N=64, H=64, V=512, temperature=1.0, d_hidden=FAKE, d_weight=FAKE, flags=0,
         saved=FAKE, tokens=FAKE, ws_size=None):
    if ws_size is None:
        ws_size = lib.flce_workspace_bytes_ex(N, H, V, 0, 0)
    return lib.flce_logprobs_backward(FAKE, FAKE, tokens, saved, N, H, V, -100, 0.0, temperature,
                                      0, FAKE, FAKE, d_hidden, d_weight, flags, FAKE, ws_size,
                                      None)


def test_backward_refusals(lib):
    assert _bwd(lib, temperature=0.0) == ARG
    assert _bwd(lib, temperature=float("nan")) == ARG
    assert _bwd(lib, d_hidden=None, d_weight=None) == ARG
    assert _bwd(lib, flags=16) == ARG
    assert _bwd(lib, saved=None) == ARG
    assert _bwd(lib, tokens=None) == ARG
    assert _bwd(lib, H=60) == SHAPE
    assert _bwd(lib, flags=8) == WS            # a bf16 dWeight needs the larger workspace
    assert _bwd(lib, ws_size=256) == WS


def test_binding_refuses_host_tensors():
    h, w, y = torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        flce.logprobs_forward(h, w, y)
    with pytest.raises(ValueError):
        flce.logprobs_forward(h, w)
    with pytest.raises(ValueError):
        flce.logprobs_backward(h, w, y, torch.zeros(2, 2), torch.zeros(2))
    with pytest.raises(ValueError):
        flce.fused_linear_logprobs(h.requires_grad_(), w, y)


def test_refusals_of_the_forms_with_three_saved_rows(lib):
    """They refuse what the others do."""
    class Ex:
        flce_logprobs_workspace_bytes = lib.flce_logprobs_workspace_bytes
        flce_workspace_bytes_ex = lib.flce_workspace_bytes_ex
        flce_logprobs_forward = lib.flce_logprobs_forward_ex
        flce_logprobs_backward = lib.flce_logprobs_backward_ex

    test_forward_refusals(Ex)
    test_backward_refusals(Ex)


def test_lists_of_many_rows_share_memory(lib):
    """Lists take 1 GiB at most; statistics, counts and (bf16) a chunk's hidden rows beside them."""
    ws = lib.flce_logprobs_workspace_bytes
    assert ws(131070, 4096, 131072, 1, 32) < 3 << 29
    assert ws(65536, 1000, 131072, 1, 20) < 3 << 29
    assert ws(131072, 4096, 262144, 0, 32) < 3 << 29
    assert ws(1 << 20, 512, 131072, 0, 8) < 3 << 30   # (1 GiB of hidden rows in one chunk)
    assert ws(131070, 4096, 131072, 1, 32) % 256 == 0


def test_alignment_refusals_by_type(lib):
    """bf16 rows go through TMA; fp32 ones may start on any element."""
    for off in (2, 4, 8):
        assert _fwd(lib, weight=FAKE + off) == ARG and _fwd(lib, hidden=FAKE + off) == ARG
    for off in (1, 2, 6):
        assert _fwd(lib, weight=FAKE + off, dtype=1) == ARG
        assert _fwd(lib, hidden=FAKE + off, dtype=1) == ARG
    # (past the alignment, the next check answers)
    assert _fwd(lib, hidden=FAKE + 4, dtype=1, ws_size=256) == WS
