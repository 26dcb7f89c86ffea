"""GPU parity of the tied embedding: lookup and gradient.

The lookup rounds one product once, so it equals torch's (w.float() * scale).to(dtype)
bit for bit.  The gradient adds c fp32 numbers in some fixed order (each addition off by
at most 2^-24 of the sum of magnitudes), scales and rounds once:
  |error| <= (c + 1) 2^-24 scale sum|d| + half a step of the result (2^-24 fp32, 2^-8 bf16;
  and of the old value's fp32 sum when accumulating).
"""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native

pytestmark = pytest.mark.gpu
IGN = -100
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def tokens(N, V, kind, seed):
    g = np.random.default_rng(seed)
    if kind == "uniform":
        y = g.integers(0, V, N)
    elif kind == "zipf":
        y = np.minimum(g.zipf(1.3, N) - 1, V - 1)
    elif kind == "one":
        y = np.full(N, V // 2)
    else:  # few ids in long runs, and the ends of the vocabulary
        y = g.choice([0, 1, V // 3, V - 1], N)
    return torch.from_numpy(y.astype(np.int64)).cuda()


def check_grad(got, d_out, ids, V, scale, ignore=IGN, padding=None, old=None):
    g, y = d_out.double().cpu().reshape(-1, d_out.shape[-1]), ids.cpu().reshape(-1)
    live = (y != ignore) & (y >= 0) & (y < V)
    if padding is not None:
        live &= y != padding
    ref = torch.zeros(V, g.shape[1], dtype=torch.float64)
    mag, cnt = torch.zeros_like(ref), torch.zeros(V, 1, dtype=torch.float64)
    ref.index_add_(0, y[live], g[live], alpha=scale)
    mag.index_add_(0, y[live], g[live].abs(), alpha=abs(scale))
    cnt.index_add_(0, y[live], torch.ones(int(live.sum()), 1, dtype=torch.float64))
    if old is not None:
        ref += old.double().cpu()
        mag += old.double().cpu().abs()
    bound = (cnt + 2) * 2.0 ** -24 * mag + HALF[got.dtype] * ref.abs() + 1e-45
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    untouched = cnt[:, 0] == 0
    base = torch.zeros_like(got.cpu()) if old is None else old.cpu()
    assert torch.equal(got.cpu()[untouched], base[untouched])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 45.25, -0.3])
@pytest.mark.parametrize("N,H,V", [(1, 1, 1), (1, 64, 7), (7, 5, 100), (130, 12, 33),
                                   (257, 1000, 1000), (33, 4096, 50), (5, 4100, 9)])
def test_lookup(N, H, V, scale, dtype):
    g = torch.Generator(device="cuda").manual_seed(N + H)
    w = torch.randn(V, H, device="cuda", generator=g).to(dtype)
    ids = torch.randint(0, V, (N,), device="cuda", generator=g)
    ids[N // 2] = IGN if N > 2 else ids[N // 2]
    got = flce.embedding_forward(w, ids, scale=scale, check_status=True)
    want = (w[ids.clamp(min=0)].float() * scale).to(dtype)
    want[ids == IGN] = 0
    assert got.dtype == dtype and torch.equal(got, want)


def test_lookup_shapes_strides_and_integer_types():
    w = torch.randn(50, 64, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, 50, (3, 5), device="cuda")
    want = w[ids]
    assert torch.equal(flce.embedding_forward(w, ids), want)
    assert torch.equal(flce.embedding_forward(w, ids.int()), want)
    assert torch.equal(flce.embedding_forward(w, ids.t()), w[ids.t()])
    wide = torch.zeros(50, 128, device="cuda", dtype=torch.bfloat16)
    wide[:, ::2] = w
    assert torch.equal(flce.embedding_forward(wide[:, ::2], ids), want)
    flat = torch.zeros(50 * 64 + 1, device="cuda", dtype=torch.bfloat16)
    off = flat[1:].view(50, 64)  # two bytes past a 16-byte boundary
    off.copy_(w)
    assert torch.equal(flce.embedding_forward(off, ids), want)
    assert flce.embedding_forward(w, ids[:0]).shape == (0, 5, 64)
    assert torch.equal(flce.embedding_forward(w, ids[0, 0]), w[ids[0, 0]])


def test_lookup_keeps_nan_and_infinity_and_writes_zero_for_ignored():
    w = torch.tensor([[float("nan")] * 8, [float("inf")] * 8, [1.0] * 8], device="cuda")
    got = flce.embedding_forward(w, torch.tensor([0, 1, 7, 2], device="cuda"), ignore_index=7)
    assert torch.isnan(got[0]).all() and torch.isinf(got[1]).all()
    assert torch.all(got[2] == 0) and torch.all(got[3] == 1)


@pytest.mark.parametrize("bad", [50, -1, 1 << 40])
def test_id_outside_the_vocabulary(bad):
    w = torch.randn(50, 64, device="cuda")
    ids = torch.tensor([3, bad, 4], device="cuda")
    got = flce.embedding_forward(w, ids)
    assert torch.equal(got[[0, 2]], w[[3, 4]]) and torch.all(got[1] == 0)
    with pytest.raises(flce.FlceError) as e:
        flce.embedding_forward(w, ids, check_status=True)
    assert e.value.status == 3
    d = torch.randn(3, 64, device="cuda")
    ws = torch.empty(flce.embedding_workspace_bytes(3, 64, 50), dtype=torch.uint8, device="cuda")
    dw = flce.embedding_backward(d, ids, 50, workspace=ws)
    assert flce.status(ws) == 3
    check_grad(dw, d, ids, 50, 1.0)


@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "runs"])
@pytest.mark.parametrize("din,dout", [(torch.bfloat16, torch.bfloat16),
                                      (torch.bfloat16, torch.float32),
                                      (torch.float32, torch.float32),
                                      (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("N,H,V", [(1, 1, 1), (2, 8, 2), (31, 5, 100), (33, 12, 65), (64, 64, 3),
                                   (1000, 136, 500), (1025, 1100, 40)])
def test_gradient(N, H, V, din, dout, kind):
    ids = tokens(N, V, kind, seed=N)
    ids[N // 3] = IGN if N > 4 else ids[N // 3]
    d = torch.randn(N, H, device="cuda").to(din)
    # `runs` names id 1 in a vocabulary of one: reported, and left out
    known = bool(((ids == IGN) | (ids < V)).all())
    got = flce.embedding_backward(d, ids, V, scale=1.5, grad_dtype=dout, check_status=known)
    assert got.dtype == dout
    check_grad(got, d, ids, V, 1.5)
    old = torch.randn(V, H, device="cuda").to(dout)
    acc = flce.embedding_backward(d, ids, V, scale=1.5, d_weight=old.clone(), accumulate=True,
                                  check_status=known)
    check_grad(acc, d, ids, V, 1.5, old=old)


@pytest.mark.parametrize("N", [16383, 16384, 16385, 40000])
@pytest.mark.parametrize("V", [255, 256, 131072])
def test_gradient_at_the_sort_s_limits(N, V):
    ids = tokens(N, V, "zipf", seed=V)
    ids[::7] = IGN
    d = torch.randn(N, 16, device="cuda")
    got = flce.embedding_backward(d, ids, V, check_status=True)
    check_grad(got, d, ids, V, 1.0)
    for _ in range(3):
        assert torch.equal(got, flce.embedding_backward(d, ids, V))
    old = torch.randn(V, 16, device="cuda")
    acc = flce.embedding_backward(d, ids, V, d_weight=old.clone(), accumulate=True)
    check_grad(acc, d, ids, V, 1.0, old=old)


def test_ids_of_a_very_large_vocabulary():
    V = 40_000_000  # four sort digits; one column keeps the gradient small
    ids = torch.tensor([V - 1, 0, V - 1, 1 << 24, (1 << 24) + 1], device="cuda")
    d = torch.randn(5, 1, device="cuda")
    got = flce.embedding_backward(d, ids, V)
    want = torch.zeros(V, 1, device="cuda", dtype=torch.float64).index_add_(0, ids, d.double())
    assert (got - want).abs().max() <= 2.0 ** -22 * 8
    assert int((got != 0).sum()) == 4


def test_rows_past_32_bit_offsets():
    V, H = 270_000, 8192  # 2.2e9 elements: offsets past 2^31
    w = torch.zeros(V, H, device="cuda", dtype=torch.bfloat16)
    w[V - 1] = 3.0
    w[0] = 1.0
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda")
    got = flce.embedding_forward(w, ids, scale=2.0)
    assert torch.all(got[0] == 6) and torch.all(got[1] == 2) and torch.all(got[2] == 6)
    dw = flce.embedding_backward(got, ids, V, d_weight=w, accumulate=True)
    assert torch.all(dw[V - 1] == 15) and torch.all(dw[0] == 3) and torch.all(dw[V - 2] == 0)


def test_padding_idx_is_looked_up_but_gets_no_gradient():
    ids = tokens(300, 20, "uniform", seed=1)
    d = torch.randn(300, 64, device="cuda")
    check_grad(flce.embedding_backward(d, ids, 20, padding_idx=3), d, ids, 20, 1.0, padding=3)
    ids[:200] = 3  # a run of padding across segments
    got = flce.embedding_backward(d, ids, 20, padding_idx=3)
    check_grad(got, d, ids, 20, 1.0, padding=3)
    assert torch.all(got[3] == 0)
    w = torch.randn(20, 64, device="cuda", requires_grad=True)
    out = flce.fused_embedding(w, ids, padding_idx=3)
    assert torch.equal(out.detach(), w.detach()[ids])
    out.backward(d)
    assert torch.equal(w.grad, got)


def test_all_ignored_and_no_tokens():
    ids = torch.full((70,), IGN, device="cuda")
    d = torch.randn(70, 24, device="cuda")
    for i, g in ((ids, d), (ids[:0], d[:0])):
        out = torch.full((40, 24), 7.0, device="cuda")
        assert torch.all(flce.embedding_backward(g, i, 40, d_weight=out) == 0)
        out = torch.full((40, 24), 7.0, device="cuda")
        flce.embedding_backward(g, i, 40, d_weight=out, accumulate=True)
        assert torch.all(out == 7)


def test_autograd_against_torch_with_broadcast_gradient():
    ids = torch.randint(0, 60, (4, 9), device="cuda")
    w = torch.randn(60, 32, device="cuda", requires_grad=True)
    w2 = w.detach().clone().requires_grad_()
    flce.fused_embedding(w, ids, scale=3.0).sum().backward()  # an expanded gradient
    (torch.nn.functional.embedding(ids, w2) * 3.0).sum().backward()
    assert torch.equal(w.grad, w2.grad)  # small whole numbers times 3
    b = torch.randn(60, 32, device="cuda").to(torch.bfloat16).requires_grad_()
    flce.fused_embedding(b, ids).float().sum().backward()
    assert b.grad.dtype == torch.bfloat16


def test_result_may_be_changed_in_place():
    w = torch.randn(60, 32, device="cuda", requires_grad=True)
    x = flce.fused_embedding(w, torch.randint(0, 60, (4, 9), device="cuda"))
    x += 1.0
    x.mul_(2.0)
    x.sum().backward()
    assert float(w.grad.sum()) == 2.0 * 4 * 9 * 32


@pytest.mark.parametrize("N", [700, 20000])
def test_captured_and_replayed(N):
    V, H = 300, 40
    ids, d = tokens(N, V, "zipf", 5), torch.randn(N, H, device="cuda")
    w = torch.randn(V, H, device="cuda")
    ws = torch.empty(flce.embedding_workspace_bytes(N, H, V), dtype=torch.uint8, device="cuda")
    dw = torch.empty(V, H, device="cuda")

    def step():
        flce.embedding_backward(d, ids, V, d_weight=dw, workspace=ws)
        return flce.embedding_forward(w, ids)

    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (6, 7):
        ids.copy_(tokens(N, V, "runs" if seed == 6 else "uniform", seed))
        d.copy_(torch.randn(N, H, device="cuda"))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w[ids])
        check_grad(dw, d, ids, V, 1.0)


def test_two_streams_at_once():
    jobs = []
    for i, N in enumerate((900, 18000)):
        jobs.append((tokens(N, 500, "zipf", i), torch.randn(N, 64, device="cuda")))
    torch.cuda.synchronize()
    got = [None, None]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = flce.embedding_backward(jobs[i][1], jobs[i][0], 500)
    torch.cuda.synchronize()
    for g, (ids, d) in zip(got, jobs):
        check_grad(g, d, ids, 500, 1.0)


def test_refusals_on_the_device():
    w = torch.randn(9, 8, device="cuda")
    y = torch.zeros(3, dtype=torch.int64, device="cuda")
    d = torch.randn(3, 8, device="cuda")
    with pytest.raises(TypeError):
        flce.embedding_forward(w.half(), y)
    with pytest.raises(TypeError):
        flce.embedding_forward(w, y.float())
    with pytest.raises(ValueError):
        flce.embedding_forward(w[0], y)
    with pytest.raises(ValueError):
        flce.embedding_forward(w, y.cpu())
    with pytest.raises(flce.FlceError):
        flce.embedding_forward(w, y, scale=float("inf"))
    with pytest.raises(ValueError):
        flce.embedding_backward(d[:2], y, 9)
    with pytest.raises(ValueError):
        flce.embedding_backward(d, y, 9, accumulate=True)
    with pytest.raises(ValueError):
        flce.embedding_backward(d, y, 9, d_weight=torch.zeros(8, 8, device="cuda"))
    with pytest.raises(ValueError):
        flce.embedding_backward(d, y, 9, padding_idx=9)
    with pytest.raises(ValueError):
        flce.embedding_backward(d, y, 0)
    with pytest.raises(TypeError):
        flce.embedding_backward(d, y, 9, grad_dtype=torch.float16)
    with pytest.raises(flce.FlceError):
        flce.embedding_backward(d, y, 9, workspace=torch.empty(256, dtype=torch.uint8,
                                                               device="cuda"))


# ---------------------------------------------------------------- together
def test_tied_training_step():
    """Embedding, a tanh, the LM head's log probabilities with the same weight, and
    the cross-entropy: the three gradients land in one fp32 buffer."""
    N, H, V = 260, 64, 700
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (0.2 * torch.randn(V, H, device="cuda", generator=g)).to(torch.bfloat16)
    ids = torch.randint(0, V, (N,), device="cuda", generator=g)
    nxt = torch.roll(ids, -1)
    nxt[-1] = IGN
    a = torch.randn(N, device="cuda", generator=g)

    x = flce.embedding_forward(w, ids, scale=8.0)
    h = torch.tanh(x.float()).to(torch.bfloat16)
    f = flce.logprobs_forward(h, w, nxt, top_k=3)
    loss = flce.forward(h, w, nxt)
    dh1, dw = flce.logprobs_backward(h, w, nxt, f.saved, a)
    dh2, dw = flce.backward(h, w, nxt, loss.lse, grad_scale=0.5, d_weight=dw,
                            accumulate_d_weight=True)
    dx = (dh1 + dh2) * (1 - h.float().square())
    dw = flce.embedding_backward(dx, ids, V, scale=8.0, d_weight=dw, accumulate=True)

    w64 = w.double().requires_grad_()
    x64 = w64[ids] * 8.0
    # the values of this run: x and h as they were rounded, derivatives of the formulas
    h64 = h.double().detach().requires_grad_()
    lp = torch.log_softmax(h64 @ w64.t(), -1)
    live = nxt != IGN
    tok = lp[torch.arange(N), nxt.clamp(min=0)]
    (tok[live] * a[live].double()).sum().add(-0.5 * tok[live].sum()).backward()
    d64 = h64.grad * (1 - h.double().square())
    (x64 * d64).sum().backward()
    assert abs(float(loss.loss) + float(tok[live].detach().sum())) <= 1e-5 * abs(float(loss.loss))
    rel = float((dw.double() - w64.grad).norm() / w64.grad.norm())
    # dZ in bf16 (half a step is 2^-8, but its label entries in fp32) in both heads
    assert rel <= 2.0 ** -8, rel
