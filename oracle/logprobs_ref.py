"""Float64 oracle of the scoring operator (test infrastructure only): log
probabilities of given tokens, entropy, top alternatives and their gradients,
written from the definitions.  x = softcap(hidden . weight^T) / temperature.
"""
from __future__ import annotations

import numpy as np


def logits(hidden, weight, softcap=0.0, temperature=1.0):
    """(z, x): the raw logits and those that the softmax sees, float64 [N, V]; raw
    logits at or below -1e30 (masks) count as -inf."""
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.asarray(hidden, np.float64) @ np.asarray(weight, np.float64).T
        z = np.where(z <= -1e30, -np.inf, z)
        x = softcap * np.tanh(z / softcap) if softcap > 0 else z
        return z, x / temperature


def _live(tokens, N, V, ignore_index):
    if tokens is None:
        return np.ones(N, bool), np.zeros(N, np.int64)
    y = np.asarray(tokens)
    live = (y != ignore_index) & (y >= 0) & (y < V)
    return live, np.where(live, y, 0)


def forward(hidden, weight, tokens=None, ignore_index=-100, softcap=0.0, temperature=1.0,
            top_k=0):
    """dict(logprobs, entropy, lse, top_logprobs, top_ids); rows that take no part
    hold 0 and ids -1."""
    z, x = logits(hidden, weight, softcap, temperature)
    N, V = x.shape
    live, y = _live(tokens, N, V, ignore_index)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(1, keepdims=True)
        log_s = np.log(np.exp(x - m).sum(1, keepdims=True))
        lse = (m + log_s)[:, 0]
        logp = (x - m) - log_s  # (x - lse would lose log_s where x / T is large)
        p = np.exp(logp)
        ent = -np.where(p > 0, p * logp, np.where(np.isnan(p), np.nan, 0.0)).sum(1)
    # ties: the lowest id, so a stable sort of the ids by descending logit
    order = np.argsort(-np.where(np.isnan(z), -np.inf, z), axis=1, kind="stable")[:, :top_k]
    zt = np.take_along_axis(z, order, 1)
    ids = np.where(zt > -np.inf, order, -1)
    top = np.where(ids >= 0, np.take_along_axis(logp, order, 1), -np.inf)
    keep = live[:, None]
    return dict(logprobs=np.where(live, logp[np.arange(N), y], 0.0),
                entropy=np.where(live, ent, 0.0), lse=np.where(live, lse, 0.0),
                top_logprobs=np.where(keep, top, 0.0), top_ids=np.where(keep, ids, -1))


def dz(hidden, weight, tokens, d_logprobs=None, d_entropy=None, ignore_index=-100, softcap=0.0,
       temperature=1.0):
    """Gradient of sum(d_logprobs * logprobs + d_entropy * entropy) by the raw logits, [N, V]."""
    z, x = logits(hidden, weight, softcap, temperature)
    N, V = x.shape
    live, y = _live(tokens, N, V, ignore_index)
    a = np.zeros(N) if d_logprobs is None else np.where(live, d_logprobs, 0.0)
    b = np.zeros(N) if d_entropy is None else np.where(live, d_entropy, 0.0)
    m = x.max(1, keepdims=True)
    logp = (x - m) - np.log(np.exp(x - m).sum(1, keepdims=True))
    p = np.exp(logp)
    plogp = np.where(p > 0, p * logp, 0.0)
    ent = -plogp.sum(1, keepdims=True)
    d = -p * a[:, None] - b[:, None] * (plogp + p * ent)
    d[np.arange(N), y] += a
    d = d / temperature
    if softcap > 0:
        d = d * (1.0 - np.tanh(z / softcap) ** 2)
    return np.where(live[:, None], d, 0.0)


def backward(hidden, weight, tokens, d_logprobs=None, d_entropy=None, ignore_index=-100,
             softcap=0.0, temperature=1.0):
    """(d_hidden, d_weight) in float64."""
    g = dz(hidden, weight, tokens, d_logprobs, d_entropy, ignore_index, softcap, temperature)
    return g @ np.asarray(weight, np.float64), g.T @ np.asarray(hidden, np.float64)
