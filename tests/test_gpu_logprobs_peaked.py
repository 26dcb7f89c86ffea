"""Gradients of the scoring operator on peaked rows: one token has nearly all the probability,
so that 1 - p, which the gradient is made of, is a small difference, divided by the
temperature.  Also the C ABI's forms with two saved rows.

Tolerances, for every entry of dHidden.  dZ of the row's own token is a (1 - p) / T + ...,
with p = 2^lp2 of a small lp2: off by a step of numbers just below 1 and the exponential's
error (2^-22 together; the test takes 2^-21), and by what dx = dz / T (dz = (H / 16 + 4) 2^-23 A,
see test_gpu_logprobs.py; fp32: 2^-24 A) makes of 1 - p: (e^(2 dx) - 1) (1 - p).  Other
entries are off by (e^(2 dx) - 1 + r) of themselves, r the half step of bf16 2^-8 (fp32: 2^-20 for
the exponential and the products), and the products' sums by 2^-20 of the sum of magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import flce_inputs as fi
import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native
from oracle import logprobs_ref as ref
from tests import _gpu as G
from tests.test_gpu_logprobs import IGN, gradient_tolerance, on_gpu, problem

pytestmark = pytest.mark.gpu


def peaked(N, H, V, top, seed, dtype):
    """Rows whose token's logit stands about `top` above the others' (of size 1 or so)."""
    g = np.random.default_rng(seed)
    w = (0.5 / np.sqrt(H) * g.standard_normal((V, H))).astype(np.float32)
    if dtype == "bf16":
        w = fi.bf16_to_f32(fi.bf16_round(w))
    y = g.integers(0, V, N)
    lift = (top / (w[y].astype(np.float64) ** 2).sum(1))[:, None]
    h = (g.standard_normal((N, H)) + lift * w[y]).astype(np.float32)
    if dtype == "bf16":
        h = fi.bf16_to_f32(fi.bf16_round(h))
    y[1] = IGN
    return on_gpu(h, w, y, dtype)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("T", [1.0, 0.1, 0.01, 1e-4])
@pytest.mark.parametrize("dtype,N,H,V,top", [
    ("bf16", 24, 1024, 1500, 14.0), ("bf16", 300, 256, 900, 20.0), ("fp32", 9, 200, 700, 14.0),
    ("fp32", 40, 201, 700, 20.0)])
def test_gradients_of_peaked_rows(dtype, N, H, V, top, T, softcap):
    host, dev = peaked(N, H, V, top, 50, dtype)
    h, w, y = host
    g = np.random.default_rng(51)
    a, b = (g.standard_normal(N).astype(np.float32) for _ in range(2))
    f = flce.logprobs_forward(*dev, softcap=softcap, temperature=T)
    dh, _ = flce.logprobs_backward(*dev, f.saved, torch.from_numpy(a).cuda(),
                                   torch.from_numpy(b).cuda(), softcap=softcap, temperature=T,
                                   check_status=True)
    d = ref.dz(h, w, y, a, b, IGN, softcap, T)
    A = float((np.abs(h).astype(np.float64) @ np.abs(w).astype(np.float64).T).max())
    dz = ((H / 16 + 4) * 2.0 ** -23 if dtype == "bf16" else 2.0 ** -24) * A + 2.0 ** -21 * softcap
    grow = np.expm1(min(2 * dz / T, 500.0))
    e = np.abs(d) * (grow + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -20))
    live = y != IGN
    own = (np.arange(N)[live], y[live])
    # (1 - p and p log p + E of the token's own entry, both put together in |d|)
    e[own] = np.abs(d[own]) * (grow + 2.0 ** -20) + 2.0 ** -21 * ((np.abs(a) + np.abs(b)) / T)[live]
    bound = e @ np.abs(w).astype(np.float64) + 2.0 ** -20 * (np.abs(d) @ np.abs(w))
    err = np.abs(dh.cpu().numpy() - d @ w.astype(np.float64))
    assert np.all(err <= bound + 1e-30), float((err / (bound + 1e-30)).max())
    if T <= 0.01:  # nothing is left of the gradient but rounding, a / T of the token's row
        assert np.abs(d).max() <= 2.0 ** -24 * np.abs(a).max() / T
        assert np.all(err[live] <= 2.0 ** -20 * (np.abs(a) + np.abs(b))[live, None] / T
                      * np.abs(w).max())


@pytest.mark.parametrize("T", [1.0, 0.1])
@pytest.mark.parametrize("dtype,N,H,V", [("bf16", 300, 136, 2000), ("fp32", 33, 41, 700)])
def test_rows_of_dz_sum_to_zero(dtype, N, H, V, T):
    """A weight column of ones makes dHidden's entry the row's sum of dZ, which is 0."""
    host, _ = problem(N, H, V, seed=52, n_ign=N // 6, w_std=0.1, dtype=dtype)
    h, w, y = host
    w[:, 0], h[:, 0] = 1.0, 0.0
    host, dev = on_gpu(h, w, y, dtype)
    g = np.random.default_rng(53)
    a, b = (g.standard_normal(N).astype(np.float32) for _ in range(2))
    f = flce.logprobs_forward(*dev, temperature=T)
    dh, _ = flce.logprobs_backward(*dev, f.saved, torch.from_numpy(a).cuda(),
                                   torch.from_numpy(b).cuda(), temperature=T)
    d = np.abs(ref.dz(h, w, y, a, b, IGN, 0.0, T))
    d[np.arange(N)[y != IGN], y[y != IGN]] = 0.0  # put right in fp32
    # bf16: half steps of all other entries, with signs as good as random (a deviation of 2^-8 /
    # sqrt 3 of each at most, four of those); 2^-20 for fp32 sums and exponentials
    rounding = 4 * 2.0 ** -8 / np.sqrt(3.0) * np.sqrt((d ** 2).sum(1)) if dtype == "bf16" else 0.0
    scale = (np.abs(a) + np.abs(b) * (1 + f.entropy.cpu().numpy())) / T
    assert np.all(np.abs(dh[:, 0].cpu().numpy()) <= rounding + 2.0 ** -18 * scale)


@pytest.mark.parametrize("T", [0.1, 0.02])
def test_flat_rows_at_low_temperatures(T):
    host, dev = problem(300, 136, 2000, seed=54, n_ign=40, w_std=0.02)
    g = np.random.default_rng(55)
    a, b = (g.standard_normal(300).astype(np.float32) for _ in range(2))
    f = flce.logprobs_forward(*dev, temperature=T)
    grads = flce.logprobs_backward(*dev, f.saved, torch.from_numpy(a).cuda(),
                                   torch.from_numpy(b).cuda(), temperature=T, check_status=True)
    A = float((np.abs(host[0]).astype(np.float64) @ np.abs(host[1]).astype(np.float64).T).max())
    dx = (136 / 16 + 4) * 2.0 ** -23 * A / T
    tol = gradient_tolerance(host[0], host[1], ref.dz(*host, a, b, IGN, 0.0, T), host[2])
    for x, r, t in zip(grads, ref.backward(*host, a, b, IGN, 0.0, T), tol):
        assert G.rel_l2(x.cpu().numpy(), r) <= t + 4 * dx


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("softcap", [0.0, 4.0])
def test_c_abi_with_two_saved_rows(dtype, softcap):
    """flce_logprobs_forward / _backward: lse and entropy in 2 N floats, none behind them."""
    N, H, V, T = 150, 64, 700, 1.3
    host, (h, w, y) = problem(N, H, V, seed=56, n_ign=20, dtype=dtype)
    lib, dt = flce.load(), _native.BF16 if dtype == "bf16" else _native.FP32
    stream = torch.cuda.current_stream().cuda_stream
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    out = torch.full((3, N), 7.0, device="cuda")
    saved = torch.full((3, N), 7.0, device="cuda")
    ws = torch.empty(flce.logprobs_workspace_bytes(N, H, V, h.dtype, 0), dtype=torch.uint8,
                     device="cuda")
    st = lib.flce_logprobs_forward(ptr(h), ptr(w), ptr(y), N, H, V, IGN, softcap, T, 0, dt,
                                   ptr(out[0]), ptr(out[1]), ptr(out[2]), ptr(saved), None, None,
                                   ptr(ws), ws.numel(), stream)
    assert st == 0 and flce.status(ws) == 0
    f = flce.logprobs_forward(h, w, y, softcap=softcap, temperature=T)
    for x, z in zip(out, (f.logprobs, f.entropy, f.lse)):
        assert torch.equal(x, z)
    assert torch.all(saved[2] == 7.0)
    assert torch.equal(saved[1], f.saved[2])
    m, l2 = f.saved[0].double(), f.saved[1].double()
    want = torch.where(y != IGN, m / T + l2 * np.log(2.0), 0.0)
    assert torch.all((saved[0] - want).abs() <= 2.0 ** -23 * (1 + want.abs()))
    a = torch.randn(N, device="cuda")
    dh, dw = torch.empty(N, H, device="cuda"), torch.empty(V, H, device="cuda")
    wsb = flce.alloc_workspace(N, H, V, h.dtype, "cuda")
    st = lib.flce_logprobs_backward(ptr(h), ptr(w), ptr(y), ptr(saved), N, H, V, IGN, softcap, T,
                                    dt, ptr(a), ptr(a), ptr(dh), ptr(dw), 0, ptr(wsb),
                                    wsb.numel(), stream)
    assert st == 0 and flce.status(wsb) == 0
    # an lse of at most 32 in one float: 2^-19 of p; bf16: some entries then round the other way
    ex = flce.logprobs_backward(h, w, y, f.saved, a, a, softcap=softcap, temperature=T)
    for x, z in zip((dh, dw), ex):
        assert G.rel_l2(x.cpu().numpy(), z.double().cpu().numpy()) <= (
            2.0 ** -11 if dtype == "bf16" else 2.0 ** -17)
