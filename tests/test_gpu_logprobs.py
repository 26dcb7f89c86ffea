"""GPU parity of the scoring operator (log probabilities, entropy, alternatives and
their gradients) against its float64 oracle.

Tolerances.  The tensor cores add H bf16 products (exact in fp32) in fp32; with
A = sum_k |h_k w_k| each of about H / 16 additions is off by at most one fp32
step 2^-23 A, so |dz| <= (H / 16 + 4) 2^-23 A_max.  The softmax then adds 2^-20
relative (exp2 to 2^-22, sums of 4 partial chains) and the softcap's tanh 2^-21 of
the cap.  lse moves by at most max|dx|; entropy by sum p |log p + E| |dx| <=
2 (E + 1) max|dx|; the token's logit is evaluated in fp64.  The results are
float32: half a step, 2^-24 relative.
Gradients: dZ is rounded to bf16 (at most 2^-8 relative, its label entries are put
right in fp32), so dHidden moves by sum_v e_v W_v with |e_v| <= 2^-8 |dZ_v| and signs
as good as random: the tolerance is three times the root of the summed squares
at the half-step bound's uniform deviation 2^-8 / sqrt(3), and 1e-4 for the fp32 rest.
"""
import numpy as np
import pytest
import torch

import flce_inputs as fi
import lm_head_linear_tmem_b200 as flce
from lm_head_linear_tmem_b200 import _native
from oracle import logprobs_ref as ref
from tests import _gpu as G

pytestmark = pytest.mark.gpu
IGN = fi.IGNORE_INDEX


def problem(N, H, V, seed, n_ign=0, w_std=0.3, dtype="bf16"):
    """(hidden, weight, tokens) as float64-exact numpy arrays and as device tensors."""
    g = np.random.default_rng(seed)
    h = g.standard_normal((N, H)).astype(np.float32)
    w = (w_std * g.standard_normal((V, H))).astype(np.float32)
    if dtype == "bf16":
        h, w = fi.bf16_to_f32(fi.bf16_round(h)), fi.bf16_to_f32(fi.bf16_round(w))
    y = g.integers(0, V, N)
    y[g.permutation(N)[:n_ign]] = IGN
    return on_gpu(h, w, y, dtype)


def on_gpu(h, w, y, dtype="bf16"):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return (h, w, y), (torch.from_numpy(h).cuda().to(dt), torch.from_numpy(w).cuda().to(dt),
                       None if y is None else torch.from_numpy(y).cuda())


def tolerances(h, w, softcap, temperature, f):
    """(lse and log probability, entropy) bounds of the module docstring."""
    H = h.shape[1]
    A = float((np.abs(h).astype(np.float64) @ np.abs(w).astype(np.float64).T).max())
    dx = ((H / 16 + 4) * 2.0 ** -23 * A + 2.0 ** -21 * softcap) / temperature
    big = float(np.abs(f["lse"]).max() + np.abs(f["logprobs"]).max())
    e = float(np.abs(f["entropy"]).max())
    return dx + 2.0 ** -20 * (1 + big), 2 * (e + 1) * dx + 2.0 ** -20 * (1 + e + big)


def check_forward(got, host, softcap=0.0, temperature=1.0, top_k=0):
    h, w, y = host
    f = ref.forward(h, w, y, IGN, softcap, temperature, top_k)
    t_lse, t_ent = tolerances(h, w, softcap, temperature, f)
    if y is None:
        assert got.logprobs is None
    else:
        assert np.abs(got.logprobs.cpu().numpy().ravel() - f["logprobs"]).max() <= t_lse
        dead = (y == IGN) | (y < 0) | (y >= w.shape[0])
        for t in (got.logprobs, got.entropy, got.lse):
            assert np.all(t.cpu().numpy().ravel()[dead] == 0.0)
    assert np.abs(got.lse.cpu().numpy().ravel() - f["lse"]).max() <= t_lse
    assert np.abs(got.entropy.cpu().numpy().ravel() - f["entropy"]).max() <= t_ent
    if top_k:
        assert np.array_equal(got.top_ids.cpu().numpy().reshape(-1, top_k), f["top_ids"])
        a, b = got.top_logprobs.cpu().numpy().reshape(-1, top_k), f["top_logprobs"]
        inf = np.isinf(b)
        assert np.array_equal(a[inf], b[inf])
        assert np.abs(a[~inf] - b[~inf]).max(initial=0.0) <= t_lse
    else:
        assert got.top_ids is None and got.top_logprobs is None
    return f


@pytest.mark.parametrize("softcap,temperature", [(0.0, 1.0), (4.0, 1.0), (0.0, 0.7), (3.0, 1.4)])
@pytest.mark.parametrize("N,H,V,top_k", [
    (1, 8, 1, 1), (1, 64, 32, 5), (3, 200, 1000, 8), (127, 72, 257, 0), (128, 64, 256, 32),
    (129, 136, 511, 20), (300, 200, 1000, 4), (513, 72, 2049, 6)])
def test_bf16_sizes(N, H, V, top_k, softcap, temperature):
    host, dev = problem(N, H, V, seed=N + V, n_ign=N // 5)
    got = flce.logprobs_forward(*dev, softcap=softcap, temperature=temperature, top_k=top_k,
                                check_status=True)
    check_forward(got, host, softcap, temperature, top_k)


@pytest.mark.parametrize("softcap,temperature", [(0.0, 1.0), (3.0, 0.8)])
@pytest.mark.parametrize("N,H,V,top_k", [
    (1, 8, 1, 1), (1, 33, 32, 5), (9, 201, 1000, 8), (17, 72, 257, 0), (2, 5400, 300, 32),
    (3, 12288, 40, 3)])
def test_fp32_sizes(N, H, V, top_k, softcap, temperature):
    host, dev = problem(N, H, V, seed=N + V, n_ign=N // 5, w_std=0.1, dtype="fp32")
    got = flce.logprobs_forward(*dev, softcap=softcap, temperature=temperature, top_k=top_k,
                                check_status=True)
    check_forward(got, host, softcap, temperature, top_k)


@pytest.mark.parametrize("softcap,temperature", [(0.0, 1.0), (3.0, 0.8)])
@pytest.mark.parametrize("N,H,V,top_k", [
    (18, 64, 64, 2), (63, 65, 63, 32), (64, 128, 129, 0), (65, 8, 130, 5), (130, 1001, 300, 7),
    (33, 12288, 70, 3), (17, 12, 1, 1), (600, 8, 32007, 6), (577, 67, 33000, 0)])
def test_fp32_sizes_of_many_rows(N, H, V, top_k, softcap, temperature):
    host, dev = problem(N, H, V, seed=N + V, n_ign=N // 5, w_std=0.1, dtype="fp32")
    got = flce.logprobs_forward(*dev, softcap=softcap, temperature=temperature, top_k=top_k,
                                check_status=True)
    check_forward(got, host, softcap, temperature, top_k)
    again = flce.logprobs_forward(*dev, softcap=softcap, temperature=temperature, top_k=top_k)
    assert torch.equal(got.lse, again.lse) and torch.equal(got.entropy, again.entropy)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_tokens_every_row_is_scored(dtype):
    host, dev = problem(150, 64, 700, seed=1, n_ign=40, dtype=dtype)
    got = flce.logprobs_forward(dev[0], dev[1], top_k=3, check_status=True)
    check_forward(got, (host[0], host[1], None), top_k=3)


def test_no_rows_and_all_rows_ignored():
    host, dev = problem(200, 64, 300, seed=2, n_ign=200)
    got = flce.logprobs_forward(*dev, top_k=4, check_status=True)
    for t in (got.logprobs, got.entropy, got.lse, got.top_logprobs):
        assert torch.all(t == 0)
    assert torch.all(got.top_ids == -1)
    dh, dw = flce.logprobs_backward(*dev, got.saved, torch.ones(200, device="cuda"),
                                    torch.ones(200, device="cuda"), check_status=True)
    assert torch.all(dh == 0) and torch.all(dw == 0)
    none = flce.logprobs_forward(dev[0][:0], dev[1], dev[2][:0], top_k=2)
    assert none.logprobs.shape == (0,) and none.top_ids.shape == (0, 2)


@pytest.mark.parametrize("N", [5, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_token_outside_the_vocabulary_is_reported_and_its_row_left_out(N, dtype):
    host, dev = problem(N, 64, 300, seed=3, n_ign=1, dtype=dtype)
    host[2][2], host[2][4] = 300, -7
    dev = (dev[0], dev[1], torch.from_numpy(host[2]).cuda())
    ws = torch.empty(flce.logprobs_workspace_bytes(N, 64, 300, dev[0].dtype, 3),
                     dtype=torch.uint8, device="cuda")
    got = flce.logprobs_forward(*dev, top_k=3, workspace=ws)
    assert _native.STATUS_NAMES[flce.status(ws)] == "FLCE_ERR_LABEL_RANGE"
    check_forward(got, host, top_k=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [3, 260])
def test_ties_go_to_the_lowest_id(N, dtype):
    """Small integers: every logit is exact, many are equal (a zero row makes all
    of them equal)."""
    g = np.random.default_rng(5)
    h = g.integers(-1, 2, (N, 16)).astype(np.float32)
    h[0] = 0.0
    w = g.integers(-1, 2, (1500, 16)).astype(np.float32)
    w[700:900] = w[100:300]
    host, dev = on_gpu(h, w, g.integers(0, 1500, N), dtype)
    got = flce.logprobs_forward(*dev, top_k=32, check_status=True)
    f = check_forward(got, host, top_k=32)
    assert np.array_equal(f["top_ids"][0], np.arange(32))


@pytest.mark.parametrize("order", ["rising", "falling", "late"])
@pytest.mark.parametrize("N", [40, 600])
def test_alternatives_in_unfavourable_orders(N, order):
    """Rising logits make every column a candidate when it is seen; `late` has all
    the best ids in the last partial tile."""
    V = 9000
    g = np.random.default_rng(6)
    h = np.abs(g.integers(1, 3, (N, 8))).astype(np.float32)
    w = np.zeros((V, 8), np.float32)
    steps = np.arange(V)
    if order == "falling":
        steps = steps[::-1]
    if order == "late":
        steps = np.where(steps > V - 11, steps, 0)
    w[:, 0], w[:, 1] = steps // 128, (steps % 128) / 128  # exact in bf16 up to 8 bits each
    host, dev = on_gpu(h, w, g.integers(0, V, N))
    got = flce.logprobs_forward(*dev, top_k=20, check_status=True)
    check_forward(got, host, top_k=20)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [6, 200])
@pytest.mark.parametrize("low", [-np.inf, -3.3895313892515355e38])
def test_columns_switched_off_by_their_weight(N, low, dtype):
    """A logit of -inf, or of the type's lowest value, is a probability of zero:
    nothing of it reaches the entropy, and it is never an alternative."""
    g = np.random.default_rng(7)
    h = np.zeros((N, 8), np.float32)
    h[:, 0] = 1.0
    h[:, 1:] = g.integers(-2, 3, (N, 7))
    w = np.zeros((600, 8), np.float32)
    w[:, 1:] = g.integers(-2, 3, (600, 7))
    off = np.ones(600, bool)
    off[[5, 77, 300, 599]] = False
    w[off, 0] = low
    w[off, 1:] = 0.0
    y = np.full(N, 77)
    host, dev = on_gpu(h, w, y, dtype)
    got = flce.logprobs_forward(*dev, top_k=6, check_status=True)
    f = ref.forward(h, w, y, IGN, top_k=6)
    assert np.abs(got.logprobs.cpu().numpy() - f["logprobs"]).max() < 1e-5
    assert np.abs(got.entropy.cpu().numpy() - f["entropy"]).max() < 1e-5
    ids = got.top_ids.cpu().numpy()
    assert np.array_equal(ids[:, :4], f["top_ids"][:, :4])
    assert np.all(ids[:, 4:] == -1) and np.all(np.isneginf(got.top_logprobs.cpu()[:, 4:].numpy()))
    # a token that is masked has probability 0
    off_tok = torch.full((N,), 6, device="cuda")
    assert torch.isneginf(flce.logprobs_forward(dev[0], dev[1], off_tok).logprobs).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [6, 200])
@pytest.mark.parametrize("low", [-np.inf, -3.3895313892515355e38])
def test_rows_whose_mask_leaves_nothing(N, low, dtype):
    """Row 2 sees only masked columns: no alternatives, nothing to take a logarithm
    of; the other rows are as without it."""
    g = np.random.default_rng(27)
    h = np.zeros((N, 8), np.float32)
    h[:, 1:] = g.integers(1, 3, (N, 7))
    w = np.zeros((300, 8), np.float32)
    w[:, 1:] = g.integers(-2, 3, (300, 7))
    host, dev = on_gpu(h, w, np.full(N, 5), dtype)
    clean = flce.logprobs_forward(*dev, top_k=4)
    wide = dev[1].clone()
    wide[:, 0] = low
    hid = dev[0].clone()
    # finite weights (or zero hidden entries against -inf would be NaN)
    if np.isinf(low):
        hid = hid[2:3].clone()
        hid[:, 0] = 1.0
        got = flce.logprobs_forward(hid, wide, dev[2][2:3], top_k=4, check_status=True)
        row = 0
    else:
        hid[2, 0] = 1.0
        got = flce.logprobs_forward(hid, wide, dev[2], top_k=4, check_status=True)
        row = 2
        keep = [i for i in range(N) if i != 2]
        for a, b in zip(clean[:5], got[:5]):
            assert torch.equal(a[keep], b[keep])
    assert torch.all(got.top_ids[row] == -1) and torch.isneginf(got.top_logprobs[row]).all()
    assert torch.isneginf(got.lse[row])
    assert torch.isnan(got.logprobs[row]) and torch.isnan(got.entropy[row])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [6, 200])
def test_nan_and_infinite_rows_stay_by_themselves(N, dtype):
    host, dev = problem(N, 64, 300, seed=8, dtype=dtype)
    clean = flce.logprobs_forward(*dev, top_k=5)
    h = dev[0].clone()
    h[1] = float("nan")
    h[3, 7] = float("inf")
    got = flce.logprobs_forward(h, dev[1], dev[2], top_k=5, check_status=True)
    for t in (got.logprobs, got.entropy, got.lse):
        assert torch.isnan(t[[1, 3]]).all()
    assert torch.all(got.top_ids[1] == -1)
    assert torch.all((got.top_ids >= -1) & (got.top_ids < 300))
    keep = [i for i in range(N) if i not in (1, 3)]
    for a, b in zip(clean[:5], got[:5]):
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(clean.saved[:, keep], got.saved[:, keep])


def test_every_schedule_gives_the_same_answers():
    host, dev = problem(700, 72, 5000, seed=9, n_ign=100)
    for opt in ({}, {"cta_group": 1}, {"fwd_tile_n": 256}, {"fwd_compact": 0}, {"fwd_dynamic": 0},
                {"fwd_group_m": 1}, {"cta_group": 1, "fwd_dynamic": 0, "fwd_compact": 0}):
        with _native.options(**opt):
            got = flce.logprobs_forward(*dev, top_k=7, check_status=True)
        check_forward(got, host, top_k=7)


def test_repeated_calls_are_bit_identical():
    _, dev = problem(400, 136, 30000, seed=10, n_ign=30)
    first = flce.logprobs_forward(*dev, top_k=20)
    for _ in range(20):
        for a, b in zip(first, flce.logprobs_forward(*dev, top_k=20)):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- gradients
def gradient_tolerance(h, w, dz, tokens):
    """Relative L2 bounds of dHidden and dWeight (module docstring)."""
    e = np.abs(dz) * 2.0 ** -8 / np.sqrt(3.0)
    live = (tokens != IGN)
    e[np.arange(len(tokens))[live], tokens[live]] = 0.0
    dh, dw = dz @ w.astype(np.float64), dz.T @ h.astype(np.float64)
    var_h = (e ** 2) @ (w.astype(np.float64) ** 2)
    var_w = (e ** 2).T @ (h.astype(np.float64) ** 2)
    return (3 * np.sqrt(var_h.sum()) / np.linalg.norm(dh) + 1e-4,
            3 * np.sqrt(var_w.sum()) / np.linalg.norm(dw) + 1e-4)


@pytest.mark.parametrize("softcap,temperature", [(0.0, 1.0), (4.0, 1.3)])
@pytest.mark.parametrize("which", ["logprobs", "entropy", "both"])
@pytest.mark.parametrize("N,H,V", [(1, 8, 16), (7, 64, 100), (300, 200, 1000), (513, 72, 2049)])
def test_backward_bf16(N, H, V, which, softcap, temperature):
    host, dev = problem(N, H, V, seed=N + H, n_ign=N // 4)
    g = np.random.default_rng(11)
    a = g.standard_normal(N).astype(np.float32) if which != "entropy" else None
    b = g.standard_normal(N).astype(np.float32) if which != "logprobs" else None
    f = flce.logprobs_forward(*dev, softcap=softcap, temperature=temperature)
    up = [None if t is None else torch.from_numpy(t).cuda() for t in (a, b)]
    with G.chunks(256, 512):
        dh, dw = flce.logprobs_backward(*dev, f.saved, *up, softcap=softcap,
                                        temperature=temperature, check_status=True)
    rh, rw = ref.backward(*host, a, b, IGN, softcap, temperature)
    t_h, t_w = gradient_tolerance(host[0], host[1],
                                  ref.dz(*host, a, b, IGN, softcap, temperature), host[2])
    assert G.rel_l2(dh.cpu().numpy(), rh) <= t_h
    assert G.rel_l2(dw.cpu().numpy(), rw) <= t_w
    assert np.all(dh.cpu().numpy()[host[2] == IGN] == 0.0)


@pytest.mark.parametrize("softcap,temperature", [(0.0, 1.0), (4.0, 1.3)])
def test_backward_fp32(softcap, temperature):
    N, H, V = 33, 40, 700
    host, dev = problem(N, H, V, seed=12, n_ign=6, dtype="fp32")
    g = np.random.default_rng(13)
    a, b = (g.standard_normal(N).astype(np.float32) for _ in range(2))
    f = flce.logprobs_forward(*dev, softcap=softcap, temperature=temperature)
    dh, dw = flce.logprobs_backward(*dev, f.saved, torch.from_numpy(a).cuda(),
                                    torch.from_numpy(b).cuda(), softcap=softcap,
                                    temperature=temperature, check_status=True)
    rh, rw = ref.backward(*host, a, b, IGN, softcap, temperature)
    # fp32 throughout: p is off by (40 products + exp) about 1e-5 relative at most
    assert G.rel_l2(dh.cpu().numpy(), rh) <= 2e-5
    assert G.rel_l2(dw.cpu().numpy(), rw) <= 2e-5


def test_with_unit_gradients_it_is_the_loss():
    """-sum logprobs is the 'sum' loss: same value, same gradients."""
    host, dev = problem(300, 136, 900, seed=14, n_ign=50, w_std=0.1)
    loss = flce.forward(*dev)
    f = flce.logprobs_forward(*dev)
    assert abs(float(-f.logprobs.double().sum()) - float(loss.loss)) <= 1e-5 * float(loss.loss)
    rows = host[2] != IGN
    assert np.abs(f.lse.cpu().numpy() - loss.lse.cpu().numpy())[rows].max() <= 1e-5
    dh0, dw0 = flce.backward(*dev, loss.lse)
    dh1, dw1 = flce.logprobs_backward(*dev, f.saved, torch.full((300,), -1.0,
                                                                         device="cuda"))
    assert G.rel_l2(dh1.cpu().numpy(), dh0.double().cpu().numpy()) <= 2e-3
    assert G.rel_l2(dw1.cpu().numpy(), dw0.double().cpu().numpy()) <= 2e-3


def test_accumulation_and_skipped_gradients():
    host, dev = problem(260, 64, 600, seed=15, n_ign=30)
    a = torch.randn(260, device="cuda")
    f = flce.logprobs_forward(*dev)
    dh, dw = flce.logprobs_backward(*dev, f.saved, a)
    base = torch.randn_like(dw)
    only, buf = flce.logprobs_backward(*dev, f.saved, a, compute_d_hidden=False,
                                       d_weight=base.clone(), accumulate_d_weight=True)
    assert only is None
    # one fp32 rounding of a sum of two numbers of at most about 8, and of its parts' order
    assert (buf - (base + dw)).abs().max() <= 1e-5
    bf, none = flce.logprobs_backward(*dev, f.saved, a, compute_d_weight=False,
                                      grad_dtype=torch.bfloat16)
    assert none is None and (bf.float() - dh).abs().max() <= 2.0 ** -8 * dh.abs().max() + 1e-6


def test_autograd_shapes_and_broadcast_gradients():
    host, dev = problem(2 * 70, 64, 500, seed=16, n_ign=20)
    h = dev[0].view(2, 70, 64).requires_grad_()
    w = dev[1].requires_grad_()
    y = dev[2].view(2, 70)
    f = flce.fused_linear_logprobs(h, w, y, temperature=0.9, top_k=2)
    assert f.logprobs.shape == (2, 70) and f.top_ids.shape == (2, 70, 2)
    assert not f.top_logprobs.requires_grad and not f.lse.requires_grad
    (f.logprobs.sum() - 0.1 * f.entropy.mean()).backward()  # expanded upstream gradients
    a, b = np.ones(140), np.full(140, -0.1 / 140)
    rh, rw = ref.backward(*host, a, b, IGN, 0.0, 0.9)
    assert h.grad.shape == h.shape and h.grad.dtype == torch.bfloat16
    # bf16 results: 2^-8 on top of the bound of the fp32 ones
    t_h, t_w = gradient_tolerance(host[0], host[1], ref.dz(*host, a, b, IGN, 0.0, 0.9), host[2])
    assert G.rel_l2(h.grad.float().cpu().numpy().reshape(140, 64), rh) <= t_h + 2.0 ** -8
    assert G.rel_l2(w.grad.float().cpu().numpy(), rw) <= t_w + 2.0 ** -8


def test_results_may_be_changed_in_place():
    _, dev = problem(2 * 30, 64, 500, seed=28)
    h = dev[0].view(2, 30, 64).requires_grad_()
    f = flce.fused_linear_logprobs(h, dev[1], dev[2].view(2, 30), top_k=2)
    want, = torch.autograd.grad((3.0 * f.logprobs).sum(), h, retain_graph=True)
    f.logprobs.mul_(3.0)
    f.lse.zero_()
    f.top_logprobs.zero_()
    got, = torch.autograd.grad(f.logprobs.sum(), h)
    assert torch.equal(got, want)


@pytest.mark.parametrize("opt", [{"bwd_compact": 0}, {"cta_group": 1}, {"bwd_fuse": 0},
                                 {"dz_buffers": 2}, {"mn3d": 0}, {"grad_tile_n": 256},
                                 {"dz_tile_n": 256}, {"bwd_compact": 0, "cta_group": 1}])
@pytest.mark.parametrize("softcap", [0.0, 4.0])
def test_every_backward_schedule(opt, softcap):
    host, dev = problem(600, 136, 3000, seed=29, n_ign=100)
    g = np.random.default_rng(30)
    a, b = (g.standard_normal(600).astype(np.float32) for _ in range(2))
    up = [torch.from_numpy(t).cuda() for t in (a, b)]
    rh, rw = ref.backward(*host, a, b, IGN, softcap, 0.8)
    d = ref.dz(*host, a, b, IGN, softcap, 0.8)
    # without the compaction there is no fp32 label correction: label entries round too
    y = np.full(600, IGN) if "bwd_compact" in opt else host[2]
    t_h, t_w = gradient_tolerance(host[0], host[1], d, y)
    f = flce.logprobs_forward(*dev, softcap=softcap, temperature=0.8)
    with _native.options(chunk_tokens=256, chunk_vocab=1024, **opt):
        dh, dw = flce.logprobs_backward(*dev, f.saved, *up, softcap=softcap, temperature=0.8,
                                        check_status=True)
    assert G.rel_l2(dh.cpu().numpy(), rh) <= t_h
    assert G.rel_l2(dw.cpu().numpy(), rw) <= t_w


def test_entropy_alone_needs_no_tokens():
    host, dev = problem(150, 64, 300, seed=17)
    h = dev[0].requires_grad_()
    f = flce.fused_linear_logprobs(h, dev[1])
    f.entropy.sum().backward()
    rh, _ = ref.backward(host[0], host[1], None, None, np.ones(150))
    dz = ref.dz(host[0], host[1], None, None, np.ones(150))
    t_h, _ = gradient_tolerance(host[0], host[1], dz, np.full(150, IGN))
    assert G.rel_l2(h.grad.float().cpu().numpy(), rh) <= t_h + 2.0 ** -8


def test_lse_and_alternatives_carry_no_gradient():
    _, dev = problem(5, 64, 300, seed=18)
    f = flce.fused_linear_logprobs(dev[0].requires_grad_(), dev[1], dev[2], top_k=2)
    with pytest.raises(RuntimeError):
        f.lse.sum().backward()


# ---------------------------------------------------------------- streams, graphs, layouts
@pytest.mark.parametrize("N", [9, 300])
def test_captured_and_replayed(N):
    host, dev = problem(N, 64, 900, seed=19, n_ign=N // 3)
    ws = torch.empty(flce.logprobs_workspace_bytes(N, 64, 900, torch.bfloat16, 6),
                     dtype=torch.uint8, device="cuda")
    wsb = flce.alloc_workspace(N, 64, 900, torch.bfloat16, "cuda")
    a = torch.randn(N, device="cuda")

    def step():
        f = flce.logprobs_forward(*dev, top_k=6, workspace=ws)
        return f, flce.logprobs_backward(*dev, f.saved, a, a, workspace=wsb)

    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            f, grads = step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (20, 21):  # new inputs in place, two replays back to back
        new, new_dev = problem(N, 64, 900, seed=seed, n_ign=N // 4)
        for old, t in zip(dev, new_dev):
            old.copy_(t)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        check_forward(f, new, top_k=6)
        eager = flce.logprobs_forward(*new_dev, top_k=6)
        for x, z in zip(f, eager):
            assert torch.equal(x, z)
        for x, z in zip(grads, flce.logprobs_backward(*new_dev, eager.saved, a, a)):
            assert torch.equal(x, z)


def test_two_streams_at_once():
    cases = [problem(N, 136, 3000, seed=22 + N, n_ign=3) for N in (10, 300)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(5):
        for i, (s, (_, dev)) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[i] = flce.logprobs_forward(*dev, top_k=9)
    torch.cuda.synchronize()
    for g, (host, _) in zip(got, cases):
        check_forward(g, host, top_k=9)


def test_strided_inputs_and_int32_tokens():
    host, dev = problem(2 * 30, 64, 300, seed=24, n_ign=5)
    h = torch.zeros(30, 2, 64, device="cuda", dtype=torch.bfloat16)
    h.copy_(dev[0].view(2, 30, 64).transpose(0, 1))
    w = torch.zeros(300, 128, device="cuda", dtype=torch.bfloat16)
    w[:, ::2] = dev[1]
    got = flce.logprobs_forward(h.transpose(0, 1), w[:, ::2], dev[2].view(2, 30).int(), top_k=3)
    assert got.top_ids.shape == (2, 30, 3)
    check_forward(got, host, top_k=3)


def test_refusals_on_the_device():
    _, (h, w, y) = problem(5, 64, 300, seed=25)
    for bad in (-1, 33):
        with pytest.raises(ValueError):
            flce.logprobs_forward(h, w, y, top_k=bad)
    with pytest.raises(ValueError):
        flce.logprobs_forward(h, w[:4].contiguous(), y, top_k=5)
    with pytest.raises(flce.FlceError):
        flce.logprobs_forward(h, w, y, temperature=0.0)
    with pytest.raises(TypeError):
        flce.logprobs_forward(h.half(), w.half(), y)
    with pytest.raises(ValueError):
        flce.logprobs_forward(h, w, y[:3])
    with pytest.raises(ValueError):
        flce.logprobs_forward(h, w, y, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(flce.FlceError):
        flce.logprobs_forward(h, w, y, workspace=torch.empty(512, dtype=torch.uint8,
                                                             device="cuda"))
    f = flce.logprobs_forward(h, w, y)
    with pytest.raises(ValueError):
        flce.logprobs_backward(h, w, None, f.saved, f.lse)
    with pytest.raises(ValueError):
        flce.logprobs_backward(h, w, y, f.saved, torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        flce.logprobs_backward(h, w, y, f.lse, f.lse)


@pytest.mark.parametrize("N,H,V", [(1, 64, 5000), (40, 128, 3000), (300, 72, 9000),
                                   (257, 264, 2100)])
def test_backward_of_few_tokens_cuts_the_vocabulary(N, H, V):
    """Few token rows: dHidden's sum over the vocabulary runs in several ranges that
    are added in order, over one and over several chunks."""
    host, dev = problem(N, H, V, seed=N + V, n_ign=N // 5)
    a = np.random.default_rng(26).standard_normal(N).astype(np.float32)
    f = flce.logprobs_forward(*dev)
    up = torch.from_numpy(a).cuda()
    rh, rw = ref.backward(*host, a, None, IGN)
    t_h, t_w = gradient_tolerance(host[0], host[1], ref.dz(*host, a, None, IGN), host[2])
    for tokens, vocab in ((16384, 16384), (256, 1280)):
        with G.chunks(tokens, vocab):
            first = flce.logprobs_backward(*dev, f.saved, up, check_status=True)
            again = flce.logprobs_backward(*dev, f.saved, up)
            base = torch.randn_like(first[0])
            acc, _ = flce.logprobs_backward(*dev, f.saved, up, d_hidden=base.clone(),
                                            accumulate_d_hidden=True, compute_d_weight=False)
        for x, y, r, t in zip(first, again, (rh, rw), (t_h, t_w)):
            assert torch.equal(x, y)
            assert G.rel_l2(x.cpu().numpy(), r) <= t
        # two fp32 roundings of sums of at most about 8
        assert (acc - (base + first[0])).abs().max() <= 1e-5


@pytest.mark.parametrize("N,H,V", [(17000, 16, 300), (5000, 8, 3000), (16385, 8, 40)])
def test_many_rows(N, H, V):
    """More rows than one block orders, more row tiles than a raster group."""
    host, dev = problem(N, H, V, seed=N, n_ign=N // 3)
    got = flce.logprobs_forward(*dev, top_k=3, check_status=True)
    check_forward(got, host, top_k=3)
    a = np.random.default_rng(31).standard_normal(N).astype(np.float32)
    grads = flce.logprobs_backward(*dev, got.saved, torch.from_numpy(a).cuda(), check_status=True)
    tol = gradient_tolerance(host[0], host[1], ref.dz(*host, a, None, IGN), host[2])
    for g, r, t in zip(grads, ref.backward(*host, a, None, IGN), tol):
        assert G.rel_l2(g.cpu().numpy(), r) <= t


@pytest.mark.parametrize("order", ["random", "rising"])
def test_long_runs_of_a_large_vocabulary(order):
    """Lists of 36 for 4096 rows take the longer runs; a sample of rows is checked."""
    N, H, V = 4096, 8, 131072
    g = np.random.default_rng(32)
    h = fi.bf16_to_f32(fi.bf16_round(g.standard_normal((N, H)).astype(np.float32)))
    w = fi.bf16_to_f32(fi.bf16_round(g.standard_normal((V, H)).astype(np.float32)))
    if order == "rising":  # every block of columns brings better ones (bf16 has 8 bits each)
        h = np.abs(h)
        w[:] = 0.0
        w[:, 0] = np.arange(V) // 512
        w[:, 1] = (np.arange(V) % 512) // 2 / 256
        h[:, 0] = 1.0
    y = g.integers(0, V, N)
    host, dev = on_gpu(h, w, y)
    got = flce.logprobs_forward(*dev, top_k=32, check_status=True)
    rows = np.concatenate([[0, 127, 128, 255, 256, N - 1], g.integers(0, N, 26)])
    f = ref.forward(h[rows], w, y[rows], IGN, 0.0, 1.0, 32)
    t_lse, t_ent = tolerances(h[rows], w, 0.0, 1.0, f)
    assert np.array_equal(got.top_ids.cpu().numpy()[rows], f["top_ids"])
    assert np.abs(got.logprobs.cpu().numpy()[rows] - f["logprobs"]).max() <= t_lse
    assert np.abs(got.top_logprobs.cpu().numpy()[rows] - f["top_logprobs"]).max() <= t_lse
    assert np.abs(got.entropy.cpu().numpy()[rows] - f["entropy"]).max() <= t_ent


@pytest.mark.parametrize("top_k,several", [(0, 1), (1, 4), (8, 4), (20, 16)])
def test_dominant_tokens_at_fp64_accuracy(top_k, several):
    """Rows whose probability sits in a few tokens with logits of 12 to 20, where H = 4096
    truncated partial sums cost 1e-4: as many as are kept (2 without alternatives,
    else top_k + 4) are taken from fp64, so that lse and log probabilities are fp32
    numbers of size up to 20 (half a step 1e-6) from sums in fp32 (2^-22 of log 2 and
    2^-22 relative, twice): 3e-6, and 2e-6 more for the rest of the probability (a tenth at
    most, off by its truncation of at most 2e-5)."""
    N, H, V = 64, 4096, 4000
    g = torch.Generator(device="cuda").manual_seed(33 + top_k)
    w = (0.02 * torch.randn(V, H, device="cuda", generator=g)).to(torch.bfloat16)
    t = torch.stack([torch.randperm(V, device="cuda", generator=g)[:several] for _ in range(N)])
    h = torch.randn(N, H, device="cuda", generator=g)
    for j in range(several):
        h += 16.0 / (4e-4 * H) * w[t[:, j]].float()
    h = h.to(torch.bfloat16)
    f = flce.logprobs_forward(h, w, t[:, 0].contiguous(), top_k=top_k)
    z = h.double() @ w.double().t()
    lse = torch.logsumexp(z, -1)
    lp = z.gather(1, t[:, :1])[:, 0] - lse
    p = torch.log_softmax(z, -1)
    ent = -(p.exp() * p).sum(-1)
    assert float((f.lse - lse).abs().max()) <= 5e-6
    assert float((f.logprobs - lp).abs().max()) <= 5e-6
    assert float((f.entropy - ent).abs().max()) <= 5e-6 * (1 + float(ent.max()))
