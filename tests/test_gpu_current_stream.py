"""The handle of the current stream, by torch's raw call and, without that one, by its public call."""
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import flce as binding

pytestmark = pytest.mark.gpu


def test_the_handle_is_the_current_stream_s():
    dev = torch.device("cuda", 0)
    for stream in (torch.cuda.default_stream(dev), torch.cuda.Stream(dev), torch.cuda.Stream(dev)):
        with torch.cuda.stream(stream):
            assert binding._stream(dev) == torch.cuda.current_stream(dev).cuda_stream
            assert binding._stream(dev) == stream.cuda_stream


def test_without_the_raw_call(monkeypatch):
    w = torch.randn(50, 64, device="cuda")
    ids = torch.randint(0, 50, (9,), device="cuda")
    monkeypatch.setattr(binding, "_raw_stream", None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert binding._stream(w.device) == side.cuda_stream
        out = flce.embedding_forward(w, ids)
        f = flce.logprobs_forward(w[:9].contiguous(), w, ids, check_status=True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, w[ids])
    assert torch.equal(f.lse, flce.logprobs_forward(w[:9].contiguous(), w, ids).lse)
