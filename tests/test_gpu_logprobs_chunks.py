"""Scoring calls whose lists would take more than 1 GiB work on chunks of rows: outputs, statuses
and gradients as of one piece.  Tolerances as in test_gpu_logprobs.py."""
import numpy as np
import pytest
import torch

import flce_inputs as fi
import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native
from oracle import logprobs_ref as ref
from tests.test_gpu_logprobs import IGN, on_gpu, tolerances

pytestmark = pytest.mark.gpu

SIZES = {"bf16": 12001, "fp32": 8003}
H, V, K = 8, 131072, 32


def rows_of(dtype, seed):
    N = SIZES[dtype]
    g = np.random.default_rng(seed)
    h = g.standard_normal((N, H)).astype(np.float32)
    w = g.standard_normal((V, H)).astype(np.float32)
    if dtype == "bf16":
        h, w = fi.bf16_to_f32(fi.bf16_round(h)), fi.bf16_to_f32(fi.bf16_round(w))
    y = g.integers(0, V, N)
    y[g.permutation(N)[:N // 5]] = IGN
    y[[0, 4095, 4096, 6143, 6144, N - 1]] = 17  # around the ends of chunks
    return on_gpu(h, w, y, dtype)


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_in_chunks(dtype, softcap):
    host, dev = rows_of(dtype, 70)
    h, w, y = host
    N = len(y)
    got = flce.logprobs_forward(*dev, softcap=softcap, top_k=K, check_status=True)
    one = flce.logprobs_forward(*dev, softcap=softcap, check_status=True)  # short lists: one piece
    g = np.random.default_rng(71)
    at = np.concatenate([[0, 4095, 4096, 6143, 6144, N - 1], g.integers(0, N, 26)])
    f = ref.forward(h[at], w, y[at], IGN, softcap, 1.0, K)
    t_lse, t_ent = tolerances(h[at], w, softcap, 1.0, f)
    assert np.array_equal(got.top_ids.cpu().numpy()[at], f["top_ids"])
    assert np.abs(got.logprobs.cpu().numpy()[at] - f["logprobs"]).max() <= t_lse
    assert np.abs(got.lse.cpu().numpy()[at] - f["lse"]).max() <= t_lse
    assert np.abs(got.entropy.cpu().numpy()[at] - f["entropy"]).max() <= t_ent
    assert np.abs(got.top_logprobs.cpu().numpy()[at] - f["top_logprobs"]).max() <= t_lse
    # every row, against the call in one piece (each within its bound of the truth)
    A = float((np.abs(h).astype(np.float64).max(0) * np.abs(w).astype(np.float64).max(0)).sum())
    dx = (H / 16 + 4) * 2.0 ** -23 * A + 2.0 ** -21 * softcap
    for name in ("logprobs", "lse", "entropy"):
        a, b = getattr(got, name).double(), getattr(one, name).double()
        e = float(one.entropy.max()) if name == "entropy" else 0.0
        tol = 2 * (2 * (e + 1) * dx + 2.0 ** -20 * (1 + e + float(b.abs().max())))
        assert float((a - b).abs().max()) <= tol
    dead = torch.from_numpy(y == IGN).cuda()
    assert torch.all(got.lse[dead] == 0) and torch.all(got.top_ids[dead] == -1)
    # (the matrix products round alike, whatever the chunk)
    if dtype == "bf16":
        assert torch.equal(got.saved[0], one.saved[0])
    again = flce.logprobs_forward(*dev, softcap=softcap, top_k=K)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [5, -3])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_bad_token_of_any_chunk_is_reported(dtype, bad):
    _, (h, w, y) = rows_of(dtype, 72)
    y[bad] = V
    ws = torch.empty(flce.logprobs_workspace_bytes(len(y), H, V, h.dtype, K), dtype=torch.uint8,
                     device="cuda")
    got = flce.logprobs_forward(h, w, y, top_k=K, workspace=ws)
    assert _native.STATUS_NAMES[flce.status(ws)] == "FLCE_ERR_LABEL_RANGE"
    assert float(got.lse[bad]) == 0.0 and torch.all(got.top_ids[bad] == -1)
    y[bad] = 3
    got = flce.logprobs_forward(h, w, y, top_k=K, workspace=ws)
    assert flce.status(ws) == 0 and float(got.lse[bad]) != 0.0


def test_chunks_without_tokens_and_captured():
    _, (h, w, y) = rows_of("bf16", 73)
    ws = torch.empty(flce.logprobs_workspace_bytes(len(y), H, V, h.dtype, K), dtype=torch.uint8,
                     device="cuda")
    want = flce.logprobs_forward(h, w, top_k=K)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        got = flce.logprobs_forward(h, w, top_k=K, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert got.logprobs is None
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a, b)
