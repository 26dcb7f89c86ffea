"""The embedding's argument checks (C ABI and PyTorch binding), without a GPU."""
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native, build

FAKE = 0x10000  # a 256-aligned, never-dereferenced address
ARG, SHAPE, WS = 1, 2, 7


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


def _fwd(lib, N=5, H=64, V=100, scale=1.0, dtype=0, weight=FAKE, ids=FAKE, out=FAKE, status=None):
    return lib.flce_embedding_forward(weight, ids, N, H, V, -100, scale, dtype, out, status, None)


def test_forward_refusals(lib):
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert _fwd(lib, scale=bad) == ARG
    assert _fwd(lib, dtype=2) == ARG
    for name in ("weight", "ids", "out"):
        assert _fwd(lib, **{name: None}) == ARG
    assert _fwd(lib, ids=FAKE + 4) == ARG
    assert _fwd(lib, weight=FAKE + 1) == ARG
    assert _fwd(lib, out=FAKE + 2, dtype=1) == ARG
    assert _fwd(lib, status=FAKE + 2) == ARG
    for size in (dict(N=-1), dict(V=0), dict(H=0), dict(H=(1 << 20) + 1), dict(N=1 << 31)):
        assert _fwd(lib, **size) == SHAPE


def test_workspace_bytes(lib):
    ws = lib.flce_embedding_workspace_bytes
    assert ws(-1, 64, 100) == 0 and ws(5, 0, 100) == 0 and ws(5, 64, 0) == 0
    assert ws(0, 64, 100) > 0
    for n in (1, 16384, 16385):
        assert ws(n, 64, 100) % 256 == 0
    # past one block's sort: the label sort's arrays
    assert ws(16385, 64, 100) - ws(16384, 64, 100) >= 5 * 4 * 16385


def _bwd(lib, N=5, H=64, V=100, scale=1.0, dtype=0, padding=-1, d_out=FAKE, ids=FAKE, dw=FAKE,
         flags=0, ws=FAKE, size=None):
    if size is None:
        size = lib.flce_embedding_workspace_bytes(N, H, V) or 1 << 30
    return lib.flce_embedding_backward(d_out, ids, N, H, V, -100, padding, scale, dtype, dw, flags,
                                       ws, size, None)


def test_backward_refusals(lib):
    assert _bwd(lib, scale=float("nan")) == ARG
    assert _bwd(lib, dtype=5) == ARG
    for flags in (1, 4, 16, -1):  # only the dWeight flags exist here
        assert _bwd(lib, flags=flags) == ARG
    assert _bwd(lib, padding=100) == ARG
    for name in ("d_out", "ids", "dw", "ws"):
        assert _bwd(lib, **{name: None}) == ARG
    assert _bwd(lib, ws=FAKE + 16) == ARG
    assert _bwd(lib, dw=FAKE + 2) == ARG
    assert _bwd(lib, size=256) == WS
    assert _bwd(lib, N=-1) == SHAPE and _bwd(lib, V=0) == SHAPE and _bwd(lib, H=0) == SHAPE


def test_binding_refuses_host_tensors():
    w, y = torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        flce.embedding_forward(w, y)
    with pytest.raises(ValueError):
        flce.embedding_backward(torch.zeros(2, 8), y, 4)
    with pytest.raises(ValueError):
        flce.fused_embedding(w.requires_grad_(), y)
    with pytest.raises(ValueError):
        flce.fused_embedding(w, y, padding_idx=4)
