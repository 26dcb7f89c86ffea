"""The scoring operator over the whole range of temperatures that it takes, against the
float64 oracle: logits of one sign, softcaps, masked columns and rows.

Tolerances.  An fp32 logit is off by dz = (H / 16 + 4) 2^-23 A (A = max sum_k |h_k w_k|;
see test_gpu_logprobs.py), which the division by T makes dz / T: the general bound, of use
down to T of about 1e-2.  Below, the listed logits decide, and those come from fp64: off
by d64 = 2 H 2^-53 A / T (two orders of summation), where the entries that are not listed
hold no probability (asserted).  The results are float32 (2^-24 relative) of sums in fp32
(2^-20 covers the noise of what the listed terms leave of a sum of 1 to 2, at most doubled).
"""
import numpy as np
import pytest
import torch

import lm_head_linear_tmem_b200 as flce
from oracle import logprobs_ref as ref
from tests.test_gpu_logprobs import IGN, check_forward, on_gpu, problem

pytestmark = pytest.mark.gpu


def one_sided(N, H, V, seed, dtype, sign):
    """`problem` with all logits negative (-1) or positive (1); 0: of both signs."""
    host, dev = problem(N, H, V, seed=seed, n_ign=N // 8, dtype=dtype)
    if sign == 0:
        return host, dev
    h, w, y = host
    return on_gpu(np.abs(h), sign * np.abs(w), y, dtype)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("sign", [-1, 0, 1])
@pytest.mark.parametrize("dtype,N", [("bf16", 40), ("bf16", 300), ("fp32", 9), ("fp32", 70)])
@pytest.mark.parametrize("T", [1e-30, 1e-9, 1e-7, 1e-5])
def test_low_temperatures(T, dtype, N, sign, softcap):
    H, V, k = 72, 1100, 6
    host, dev = one_sided(N, H, V, 40, dtype, sign)
    h, w, y = host
    z, x = ref.logits(h, w, softcap, T)
    first = z.argmax(1)
    y = np.where(y == IGN, y, first)
    y[::3] = np.where(y[::3] == IGN, IGN, host[2][::3])  # some rows' tokens are not the best
    got = flce.logprobs_forward(dev[0], dev[1], torch.from_numpy(y).cuda(), softcap=softcap,
                                temperature=T, top_k=k, check_status=True)
    f = ref.forward(h, w, y, IGN, softcap, T, k)
    live = y != IGN
    with np.errstate(over="ignore"):
        # what the row's listed (k + 4 best) logits leave
        beyond = np.sort(x, 1)[:, -(k + 5)] - x.max(1)
        assert np.exp(beyond[live]).max() * V < 2.0 ** -24
    A = float((np.abs(h).astype(np.float64) @ np.abs(w).astype(np.float64).T).max())
    d64 = 2 * H * 2.0 ** -53 * A / T

    def close(a, b, more=0.0):
        a, b = a.astype(np.float64), b.astype(np.float32).astype(np.float64)  # (past fp32: inf)
        inf = np.isinf(b)
        assert np.array_equal(a[inf], b[inf])
        err = np.abs(a[~inf] - b[~inf])
        tol = d64 + 2.0 ** -23 * np.abs(b[~inf]) + 2.0 ** -20 + more
        assert np.all(err <= tol), float((err - tol).max())

    close(got.lse.cpu().numpy(), f["lse"])
    close(got.logprobs.cpu().numpy(), f["logprobs"])
    assert np.array_equal(got.top_ids.cpu().numpy(), f["top_ids"])
    close(got.top_logprobs.cpu().numpy(), f["top_logprobs"])
    # d(entropy) <= 2 (E + 1) max dx of the few entries that hold the probability
    e = float(f["entropy"].max())
    close(got.entropy.cpu().numpy(), f["entropy"], 2 * (e + 1) * (d64 + 2.0 ** -20))
    # and nothing is left to chance where one entry holds it all, however large d64
    z2 = np.sort(z, 1)
    sure = live & ((z2[:, -1] - z2[:, -2]) > 60 * T + 1e-12 * A) if softcap == 0 else live & False
    best = sure & (y == first)
    assert softcap or best.any()
    assert np.abs(got.logprobs.cpu().numpy()[best]).max(initial=0.0) <= 2.0 ** -20
    assert np.abs(got.entropy.cpu().numpy()[sure]).max(initial=0.0) <= 2.0 ** -20
    assert np.all(got.logprobs.cpu().numpy() <= 2.0 ** -20)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("dtype,N", [("bf16", 40), ("bf16", 300), ("fp32", 9), ("fp32", 70)])
@pytest.mark.parametrize("T", [1e-2, 0.1, 30.0, 1e30])
def test_other_temperatures(T, dtype, N, sign, softcap):
    host, dev = one_sided(N, 72, 1100, 41, dtype, sign)
    for k in (0, 6):
        got = flce.logprobs_forward(*dev, softcap=softcap, temperature=T, top_k=k,
                                    check_status=True)
        # (at high temperatures the order of the logits is that of z, not of fp32 quotients)
        check_forward(got, host, softcap, T, k)


@pytest.mark.parametrize("T", [1e-30, 1.5, 1e9, 1e30])
@pytest.mark.parametrize("low", [-1.1e30, -3.3895313892515355e38])
@pytest.mark.parametrize("dtype,N", [("bf16", 6), ("bf16", 200), ("fp32", 6), ("fp32", 70)])
def test_masks_at_any_temperature(dtype, N, low, T):
    """Masked columns are probabilities of 0, a row of nothing else has lse -inf, whatever
    the temperature."""
    g = np.random.default_rng(42)
    h = np.zeros((N, 8), np.float32)
    h[:, 1:] = g.integers(1, 3, (N, 7))
    h[:, 0] = 1.0
    w = np.zeros((600, 8), np.float32)
    w[:, 1:] = g.integers(-2, 3, (600, 7))
    off = np.ones(600, bool)
    off[[5, 77, 300, 599]] = False
    w[off, 0] = low
    h[2, 1:] = 0.0
    y = np.full(N, 77)
    # row 2: every column masked, by an entry of its own that the others multiply by 0
    w = np.concatenate([w, np.where(off, 0.0, low)[:, None].astype(np.float32),
                        np.zeros((600, 7), np.float32)], 1)
    h = np.concatenate([h, np.zeros((N, 8), np.float32)], 1)
    h[2, 8] = 1.0
    host, dev = on_gpu(h, w, y, dtype)
    got = flce.logprobs_forward(*dev, top_k=6, temperature=T, check_status=True)
    others = [i for i in range(N) if i != 2]
    f = ref.forward(h[others], w, y[others], IGN, 0.0, T, 6)
    for name in ("logprobs", "entropy", "lse", "top_logprobs"):
        a = getattr(got, name).cpu().numpy()[others].astype(np.float64)
        b = f[name].astype(np.float32).astype(np.float64)
        inf = np.isinf(b)
        assert np.array_equal(a[inf], b[inf])
        # whole-number logits, exact: x in fp64, the results in fp32
        assert np.all(np.abs(a[~inf] - b[~inf]) <= 2.0 ** -20 * (1 + np.abs(b[~inf])))
    ids = got.top_ids.cpu().numpy()
    assert np.array_equal(ids[others], f["top_ids"]) and np.all(ids[others, 4:] == -1)
    assert torch.isneginf(got.lse[2]) and torch.all(got.top_ids[2] == -1)
    assert torch.isnan(got.logprobs[2]) and torch.isnan(got.entropy[2])


@pytest.mark.parametrize("T", [1e-3, 1.5, 1e21])
@pytest.mark.parametrize("dtype,N", [("bf16", 6), ("bf16", 200), ("fp32", 6), ("fp32", 70)])
def test_logits_just_above_the_masks_count(dtype, N, T):
    """-9.9e29 and -6e29 are logits (and far from one another); masks begin at -1e30."""
    V = 300
    h = np.zeros((N, 8), np.float32)
    h[:, 0] = 1.0
    w = np.zeros((V, 8), np.float32)
    w[:, 0] = -9.9e29 if T < 1e21 else -1.1e30
    w[[5, 99], 0] = -6e29
    host, dev = on_gpu(h, w, np.full(N, 99), dtype)
    got = flce.logprobs_forward(*dev, top_k=3, temperature=T, check_status=True)
    assert torch.all(got.top_ids[:, 0] == 5) and torch.all(got.top_ids[:, 1] == 99)
    assert torch.all(got.top_ids[:, 2] == (0 if T < 1e21 else -1))
    for t in (got.logprobs, got.top_logprobs[:, 0]):
        assert float((t + np.log(2.0)).abs().max()) <= 2.0 ** -20
    assert float((got.entropy - np.log(2.0)).abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("softcap", [17.0, 30.0, 50.0])
@pytest.mark.parametrize("T", [1e-30, 1e-9, 1e-6])
@pytest.mark.parametrize("dtype,N", [("bf16", 5), ("bf16", 200), ("fp32", 5), ("fp32", 40)])
def test_softcapped_logits_one_float_apart(dtype, N, T, softcap):
    """Consecutive floats, whose rounded tanh need not keep their order: the largest term is
    still the largest.  The listed logits are fp64's, so the best token's is known."""
    V = 1000
    h = np.zeros((N, 8), np.float32)
    h[:, :3] = 1.0
    k = np.random.default_rng(43).permutation(V)
    w = np.zeros((V, 8), np.float32)
    w[:, 0] = 16.0
    w[:, 1] = (k // 32) * 2.0 ** -14  # 16 + k 2^-19: five bits each, exact in bf16
    w[:, 2] = (k % 32) * 2.0 ** -19
    best = int(k.argmax())
    host, dev = on_gpu(h, w, np.full(N, best), dtype)
    a = torch.ones(N, device="cuda")
    f = flce.logprobs_forward(*dev, softcap=softcap, temperature=T, top_k=2, check_status=True)
    assert torch.all(f.top_ids[:, 0] == best)
    r = ref.forward(h[:1], w, host[2][:1], IGN, softcap, T, 2)
    for t in f[:4]:
        assert torch.isfinite(t).all()
    # (the unlisted ones are at fp32's mercy at 1e-6, where a step of L is 1 to 2 nats: within V of them)
    assert torch.all(f.logprobs <= 2.0 ** -20) and torch.all(f.logprobs >= -np.log(2.0 * V))
    assert torch.all(f.entropy >= -2.0 ** -20) and torch.all(f.entropy <= np.log(2.0 * V))
    if T <= 1e-9:  # the best one has it all
        assert float((f.lse.double() - float(r["lse"][0])).abs().max()) <= 2.0 ** -22 * abs(r["lse"][0])
    dh, dw = flce.logprobs_backward(*dev, f.saved, a, a, softcap=softcap, temperature=T,
                                    check_status=True)
    # |dZ| sums to at most 2 (|a| + |b| log V) / T a row, whichever token has the probability
    bound = 2.0 * (1 + np.log(V)) / T
    assert float(dh.abs().max()) <= 1.01 * bound * 16.01
    assert float(dw.abs().max()) <= 1.01 * bound * N


@pytest.mark.parametrize("T", [1e-30, 1e-12, 1e-9])
@pytest.mark.parametrize("N", [5, 40])
def test_fp32_gradients_of_near_ties_at_low_temperatures(N, T):
    """Many tokens within fp32's rounding of the best: which of them has the probability is
    open, but it is at most 1."""
    H, V = 257, 200
    g = np.random.default_rng(44)
    h = g.standard_normal((N, H)).astype(np.float32)
    w = np.tile(0.3 * g.standard_normal(H), (V, 1))
    w = (w * (1 + 1e-7 * g.standard_normal((V, 1)))).astype(np.float32)
    host, dev = on_gpu(h, w, g.integers(0, V, N), "fp32")
    a = torch.ones(N, device="cuda")
    f = flce.logprobs_forward(*dev, temperature=T, check_status=True)
    for t in f[:3]:
        assert torch.isfinite(t).all()
    assert torch.all(f.logprobs <= 2.0 ** -20)
    dh, dw = flce.logprobs_backward(*dev, f.saved, a, a, temperature=T, check_status=True)
    # each of V probabilities at most 1
    bound = 1.01 * V * (2.0 + 2 * np.log(V)) / T
    assert float(dh.abs().max()) <= bound * np.abs(w).max()
    assert float(dw.abs().max()) <= bound * N * np.abs(h).max()


@pytest.mark.parametrize("top_k", [0, 1])
@pytest.mark.parametrize("dtype,N,V", [("fp32", 5, 5), ("fp32", 40, 9), ("bf16", 60, 9),
                                       ("bf16", 300, 9)])
def test_near_ties_with_the_token_behind_the_kept_ones(dtype, N, V, top_k):
    """V tokens alike to fp32 rounding, fewer kept than that: whichever the token is, its term is
    counted once.  Logits of size 10 or so that differ by some 1e-6 at most (bf16: the last
    products of H = 2000, tensor-core rounding), so every probability is 1 / V to 1e-4."""
    H = 257 if dtype == "fp32" else 2000
    g = np.random.default_rng(45)
    h = g.standard_normal((N, H)).astype(np.float32)
    w = np.tile(0.3 / np.sqrt(H / 257) * g.standard_normal(H), (V, 1))
    if dtype == "fp32":
        w *= 1 + 1e-7 * g.standard_normal((V, 1))
    else:
        w[:, -3:] = 1e-7 * g.standard_normal((V, 3))
    host, dev = on_gpu(h, w.astype(np.float32), g.integers(0, V, N), dtype)
    for y in range(V):
        f = flce.logprobs_forward(dev[0], dev[1], torch.full((N,), y, device="cuda"), top_k=top_k)
        assert float((f.logprobs + np.log(V)).abs().max()) <= 1e-4
        assert float((f.entropy - np.log(V)).abs().max()) <= 1e-4
