"""Cases that measure the LM head's scoring operators and the tied embedding.

Two operators, each in its forms for serving and for training:

  logprobs   log probabilities of given tokens under softmax(softcap(hidden . weight^T) / T),
             the entropy of each row's distribution and its top alternatives; with "grad", the
             gradients of hidden and weight for upstream gradients of the log probabilities and
             the entropies
  embedding  rows of the [vocab, hidden] weight that an LM head shares with its embedding, times a
             scale; with "grad", the weight's gradient, written whole or added into a buffer that
             already holds the LM head's part

`run` computes them in elementary torch operations, or with `own` set through this repository's
package; `exact` computes the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100
W_STD = 0.02


def listed():
    return [
        # one sequence decoding: the next token's alternatives for a sampler or a client
        dict(name="score 1 token", op="logprobs", grad=False, dtype="bf16", N=1, H=2048, V=32000,
             top_k=5, ignored=0.0, softcap=0.0, temperature=1.0),
        # a decode step of a serving batch, alternatives reported at a sampling temperature
        dict(name="score 32 tokens", op="logprobs", grad=False, dtype="bf16", N=32, H=4096,
             V=131072, top_k=20, ignored=0.0, softcap=0.0, temperature=0.7),
        # a ragged prompt scored by a softcapped model with a large vocabulary
        dict(name="score 777 softcap", op="logprobs", grad=False, dtype="bf16", N=777, H=3584,
             V=256000, top_k=8, ignored=0.1, softcap=30.0, temperature=1.0),
        # a prompt's tokens with alternatives, the padded part left out
        dict(name="score 4096", op="logprobs", grad=False, dtype="bf16", N=4096, H=4096, V=131072,
             top_k=8, ignored=0.2, softcap=0.0, temperature=1.0),
        # old log probabilities of a rollout batch (no alternatives)
        dict(name="score 8192 plain", op="logprobs", grad=False, dtype="bf16", N=8192, H=2048,
             V=32000, top_k=0, ignored=0.3, softcap=0.0, temperature=1.0),
        # fp32 weights and activations, the size of a check against a float32 model
        dict(name="score 60 fp32", op="logprobs", grad=False, dtype="fp32", N=60, H=1000, V=8009,
             top_k=3, ignored=0.1, softcap=0.0, temperature=1.0),
        # a policy-gradient step on a small odd-sized model: log probabilities, entropy bonus
        dict(name="policy step 500", op="logprobs", grad=True, dtype="bf16", N=500, H=1000,
             V=10007, top_k=0, ignored=0.2, softcap=0.0, temperature=1.0),
        # the same on a full micro-batch of a rollout
        dict(name="policy step 4096", op="logprobs", grad=True, dtype="bf16", N=4096, H=4096,
             V=131072, top_k=0, ignored=0.3, softcap=0.0, temperature=1.0),
        # one decode step's lookup
        dict(name="lookup 8", op="embedding", grad=False, dtype="bf16", N=8, H=4096, V=131072,
             accumulate=False, scale=64.0),
        # a training batch's lookup ([2, 8192] tokens)
        dict(name="lookup 16384", op="embedding", grad=False, dtype="bf16", N=16384, H=4096,
             V=131072, accumulate=False, scale=1.0),
        # its gradient, the whole bf16 weight gradient written
        dict(name="lookup grad 16384", op="embedding", grad=True, dtype="bf16", N=16384, H=4096,
             V=131072, accumulate=False, scale=1.0),
        # tied weights: a micro-batch's lookup gradient added into the LM head's fp32 gradient
        dict(name="lookup grad tied", op="embedding", grad=True, dtype="bf16", N=4093, H=2048,
             V=32000, accumulate=True, scale=45.25),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["score", "score", "few", "fp32", "policy", "lookup", "lookup grad"])
    V = _log_int(rng, 500, 131072)
    H = 8 * _log_int(rng, 8, 512)
    if kind in ("lookup", "lookup grad"):
        grad = kind == "lookup grad"
        return dict(op="embedding", grad=grad, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    N=_log_int(rng, 1, 16384), H=H // 2 if H > 2048 else H, V=V,
                    accumulate=grad and rng.random() < 0.5,
                    scale=rng.choice([1.0, round(math.sqrt(H), 3)]))
    if kind == "fp32":
        N, H, V = _log_int(rng, 1, 60), min(H, 1000) + rng.randint(0, 24), min(V, 8000)
    elif kind == "few":
        N = _log_int(rng, 1, 128)
    elif kind == "policy":
        N = _log_int(rng, 16, 4096)
    else:
        N = _log_int(rng, 64, 4096)
    return dict(op="logprobs", grad=kind == "policy", dtype="fp32" if kind == "fp32" else "bf16",
                N=N, H=H, V=V, top_k=0 if kind == "policy" else rng.choice([0, 1, 4, 5, 8, 20]),
                ignored=0.0 if N < 8 else round(rng.uniform(0.0, 0.5), 2),
                softcap=rng.choice([0.0, 0.0, 30.0]),
                temperature=rng.choice([1.0, 1.0, 0.6, 1.3]))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _zipf(n, V, gen):
    """Token ids with Zipf(1.1) frequencies (id 0 the most frequent), as text has them."""
    cdf = torch.arange(1, V + 1, device="cuda", dtype=torch.float64).pow(-1.1).cumsum(0)
    u = torch.rand(n, device="cuda", dtype=torch.float64, generator=gen) * cdf[-1]
    return torch.searchsorted(cdf, u, right=True).clamp_(max=V - 1)


def _ignored(case):
    return int(case["N"] * case["ignored"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, H, V, dt = case["N"], case["H"], case["V"], _dtype(case)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float32) * std

    if case["op"] == "embedding":
        st = dict(case=case, ids=_zipf(N, V, gen))
        if case["grad"]:
            st["d_out"] = normal(N, H, std=1e-2).to(dt)
            if case["accumulate"]:
                # what the LM head's backward left there
                st["d_weight"] = normal(V, H, std=1e-2)
        else:
            st["weight"] = normal(V, H, std=W_STD).to(dt)
        return st
    weight = normal(V, H, std=W_STD).to(dt)
    tokens = _zipf(N, V, gen)
    # a trained model prefers the token that comes: its logit stands 0 to 14 above the others'
    lift = torch.rand(N, 1, device="cuda", generator=gen) * (14.0 / (W_STD * W_STD * H))
    hidden = (normal(N, H) + lift * weight[tokens].float()).to(dt)
    if _ignored(case):
        tokens[torch.randperm(N, device="cuda", generator=gen)[:_ignored(case)]] = IGNORE
    st = dict(case=case, hidden=hidden, weight=weight, tokens=tokens)
    if case["grad"]:
        hidden.requires_grad_()
        weight.requires_grad_()
        st["d_logprobs"] = normal(N)  # advantages
        st["d_entropy"] = torch.full((N,), -0.01, device="cuda")  # an entropy bonus
    return st


# ---------------------------------------------------------------- plain forms
def _plain_logprobs(st):
    c = st["case"]
    cap, temp, k, V = c["softcap"], c["temperature"], c["top_k"], c["V"]
    hidden, weight, tokens = st["hidden"].detach(), st["weight"].detach(), st["tokens"]
    live = tokens != IGNORE
    h, w = hidden.float(), weight.float()
    z = h @ w.t()
    x = (cap * torch.tanh(z / cap) if cap else z) / temp
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1)
    log_s = torch.log(s)
    lse = m[:, 0] + log_s
    entropy = log_s - (e * (x - m)).sum(1) / s
    y = tokens.clamp(min=0)
    out = {"logprobs": torch.where(live, x.gather(1, y[:, None])[:, 0] - lse, 0.0),
           "entropy": torch.where(live, entropy, 0.0)}
    if k:
        # logits next to one another are told apart in 64 bits; ties go to the lowest index
        cand = torch.sort(z.topk(min(k + 8, V), dim=1).indices, dim=1).values
        zc = (weight[cand].double() @ hidden.double()[:, :, None])[:, :, 0]
        zc, order = torch.sort(zc, dim=1, descending=True, stable=True)
        zc, ids = zc[:, :k], cand.gather(1, order[:, :k])
        xc = (cap * torch.tanh(zc / cap) if cap else zc) / temp
        out["top_logprobs"] = torch.where(live[:, None], (xc - lse[:, None].double()).float(), 0.0)
        out["top_ids"] = torch.where(live[:, None], ids, -1)
    if c["grad"]:
        p = e / s[:, None]
        a = torch.where(live, st["d_logprobs"], 0.0)
        b = torch.where(live, st["d_entropy"], 0.0)
        dx = -p * (a[:, None] + b[:, None] * (x - lse[:, None] + entropy[:, None]))
        dx.scatter_add_(1, y[:, None], a[:, None])
        dz = dx / temp
        if cap:
            dz = dz * (1.0 - (x * temp / cap).square())
        out["d_hidden"] = (dz @ w).to(hidden.dtype)
        out["d_weight"] = (dz.t() @ h).to(weight.dtype)
    return out


def _plain_embedding(st):
    c = st["case"]
    if not c["grad"]:
        w = st["weight"]
        return {"out": (w[st["ids"]].float() * c["scale"]).to(w.dtype)}
    g = st["d_out"].float() * c["scale"]
    total = torch.zeros(c["V"], c["H"], device=g.device).index_add_(0, st["ids"], g)
    if c["accumulate"]:
        return {"d_weight": st["d_weight"] + total}
    return {"d_weight": total.to(st["d_out"].dtype)}


# ---------------------------------------------------------------- this repository's calls
def _own_logprobs(st):
    import lm_head_linear_tmem_b200 as flce
    c = st["case"]
    if not c["grad"]:
        f = flce.logprobs_forward(st["hidden"], st["weight"], st["tokens"], ignore_index=IGNORE,
                                  softcap=c["softcap"], temperature=c["temperature"],
                                  top_k=c["top_k"])
        out = {"logprobs": f.logprobs, "entropy": f.entropy}
        if c["top_k"]:
            out |= {"top_logprobs": f.top_logprobs, "top_ids": f.top_ids}
        return out
    f = flce.fused_linear_logprobs(st["hidden"], st["weight"], st["tokens"], ignore_index=IGNORE,
                                   softcap=c["softcap"], temperature=c["temperature"])
    dh, dw = torch.autograd.grad((f.logprobs, f.entropy), (st["hidden"], st["weight"]),
                                 (st["d_logprobs"], st["d_entropy"]))
    return {"logprobs": f.logprobs.detach(), "entropy": f.entropy.detach(), "d_hidden": dh,
            "d_weight": dw}


def _own_embedding(st):
    import lm_head_linear_tmem_b200 as flce
    c = st["case"]
    if not c["grad"]:
        return {"out": flce.embedding_forward(st["weight"], st["ids"], scale=c["scale"])}
    if c["accumulate"]:
        # the buffer goes on growing over a step's micro-batches; the same sum every pass here
        d = st["d_weight"].clone()
        return {"d_weight": flce.embedding_backward(st["d_out"], st["ids"], c["V"],
                                                    scale=c["scale"], d_weight=d,
                                                    accumulate=True)}
    return {"d_weight": flce.embedding_backward(st["d_out"], st["ids"], c["V"], scale=c["scale"],
                                                grad_dtype=st["d_out"].dtype)}


def run(state):
    if state["case"]["op"] == "logprobs":
        return _own_logprobs(state) if own else _plain_logprobs(state)
    return _own_embedding(state) if own else _plain_embedding(state)


# ---------------------------------------------------------------- floors
def _distinct(N, V):
    """Expected number of distinct ids among N Zipf(1.1) draws."""
    p = np.arange(1, V + 1, dtype=np.float64) ** -1.1
    p /= p.sum()
    return float(-np.expm1(N * np.log1p(-p)).sum())


def work(case):
    N, H, V = case["N"], case["H"], case["V"]
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "embedding":
        rows = _distinct(N, V)
        if not case["grad"]:
            return {"bytes": 8 * N + b * H * (rows + N), "flops": N * H}
        if case["accumulate"]:
            # the pass's own copy of the buffer, then the rows that the tokens touch
            written = 2 * 4 * V * H + 2 * 4 * rows * H
        else:
            written = b * V * H
        return {"bytes": 8 * N + b * N * H + written, "flops": 2 * N * H}
    n = N - _ignored(case)
    read = b * (N + V) * H + 8 * N
    out = (8 + 12 * case["top_k"]) * N
    if not case["grad"]:
        return {"bytes": read + out, "flops": 2 * n * H * V}
    return {"bytes": 2 * b * (N + V) * H + 16 * N + out, "flops": 8 * n * H * V}


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_embedding(c, st):
    if not c["grad"]:
        return {"out": torch.index_select(st["weight"].double(), 0, st["ids"]).mul_(c["scale"])}
    total = st["d_weight"].double() if c["accumulate"] else torch.zeros(
        c["V"], c["H"], dtype=torch.float64, device="cuda")
    # every id's rows, added in the order of the tokens
    return {"d_weight": total.index_add_(0, st["ids"], st["d_out"].double(), alpha=c["scale"])}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "embedding":
        return _exact_embedding(case, st)
    N, V, k, cap, temp = case["N"], case["V"], case["top_k"], case["softcap"], case["temperature"]
    w = st["weight"].detach().double()
    hid = st["hidden"].detach()
    out = {key: [] for key in ("logprobs", "entropy", "top_logprobs", "top_ids", "d_hidden")}
    d_weight = torch.zeros_like(w) if case["grad"] else None
    rows = max(1, (1 << 27) // V)
    for a in range(0, N, rows):
        part = slice(a, a + rows)
        h, y = hid[part].double(), st["tokens"][part]
        z = torch.matmul(h, w.t())
        q = z.clone() if cap == 0 else torch.tanh(z / cap) * cap
        logp = torch.log_softmax(q / temp, dim=-1)
        prob = logp.exp()
        keep = (y != IGNORE).double()
        at = torch.where(y == IGNORE, 0, y)
        i = torch.arange(len(y), device="cuda")
        ent = -(prob * logp).sum(-1)
        out["logprobs"].append(logp[i, at] * keep)
        out["entropy"].append(ent * keep)
        if k:
            # the k largest logits, one after another; the first of equals
            rest, ids = z.clone(), []
            for _ in range(k):
                j = rest.argmax(-1)
                ids.append(j)
                rest[i, j] = -math.inf
            ids = torch.stack(ids, -1)
            out["top_logprobs"].append(logp.gather(-1, ids) * keep[:, None])
            out["top_ids"].append(torch.where(y[:, None] == IGNORE, -1, ids))
        if case["grad"]:
            ga, gb = st["d_logprobs"][part].double() * keep, st["d_entropy"][part].double() * keep
            # d logprob_y / d x_v = [v = y] - p_v;  d entropy / d x_v = -p_v (log p_v + entropy)
            g = prob * (logp + ent[:, None]) * -gb[:, None] - prob * ga[:, None]
            g[i, at] += ga
            g /= temp
            if cap:
                g *= 1.0 - (q / cap) ** 2
            out["d_hidden"].append(torch.matmul(g, w))
            d_weight += torch.matmul(g.t(), h)
    got = {key: torch.cat(v) for key, v in out.items() if v}
    if d_weight is not None:
        got["d_weight"] = d_weight
    return got
