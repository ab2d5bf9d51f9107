"""Plain CPU oracle of log probabilities over a vocabulary and of the divergence
from a teacher's words with its gradient (test infrastructure). float64 NumPy; it
shares no code with the GPU library.

Source: the digest's section 方法步骤详情, stage 3 (the scales are tuned by
KL(softmax(z_M / T) || softmax(z_M^ / T))). The pages keep all of a teacher's
distribution; here it is cut to K words, so the formulas of the cut are plain
readings:

    z = scale H W^T, lse = log sum exp z, p = exp(z - lse)
    logprobs   z - lse of given words, -sum p log p, the k largest z (the lower
               word first among equals)
    tail       q = exp logq, r = max(0, 1 - sum q), rest = log sum exp z over the
               words that are not listed:
               loss = sum q (logq - z + lse) + r (log r - rest + lse)
    no tail    q = softmax logq over the entries, loss = sum q (log q - z + lse)
    gradient   dz = (sum q + r) p - q - r exp(z - rest) [not listed],
               G = dz dloss scale, dH = G W, dW = G^T H
"""
from __future__ import annotations

import numpy as np


def logits(H, W, scale=1.0):
    return scale * (np.asarray(H, np.float64) @ np.asarray(W, np.float64).T)


def lse_of(z):
    top = z.max(1)
    return top + np.log(np.exp(z - top[:, None]).sum(1))


def vocab_logprobs(H, W, tokens=None, k=0, scale=1.0):
    """(logprobs, entropy, lse, top_ids, top_logprobs); logprobs None without tokens."""
    z = logits(H, W, scale)
    T, V = z.shape
    lse = lse_of(z)
    logp = z - lse[:, None]
    given = None
    if tokens is not None:
        tokens = np.asarray(tokens)
        at = tokens.reshape(T, -1)
        given = np.take_along_axis(logp, np.clip(at, 0, V - 1), 1)
        given = np.where(at < 0, 0.0, np.where(at < V, given, np.nan)).reshape(tokens.shape)
    best = np.argsort(-z, axis=1, kind="stable")[:, :k]
    return given, -(np.exp(logp) * logp).sum(1), lse, best, np.take_along_axis(logp, best, 1)


def teacher(ids, logq, tail=True):
    """(q, log q, r) of each entry and token; q = 0, log q = 0 for no entry."""
    ids, logq = np.asarray(ids), np.asarray(logq, np.float64)
    on = ids >= 0
    if not tail:
        top = np.where(on, logq, -np.inf).max(1, keepdims=True, initial=-1e300)
        total = np.where(on, np.exp(np.where(on, logq, -np.inf) - top), 0.0).sum(1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            logq = logq - top - np.log(total)
    q = np.where(on, np.exp(np.where(on, logq, 0.0)), 0.0)
    r = np.maximum(0.0, 1.0 - q.sum(1)) if tail else np.zeros(len(ids))
    return q, np.where(on, logq, 0.0), r


def vocab_distill(H, W, ids, logq, scale=1.0, tail=True):
    """(loss, lse, rest, hit); rows without entries are not looked at."""
    ids = np.asarray(ids)
    T, K = ids.shape
    loss, lse, rest, hit = np.zeros(T), np.zeros(T), np.zeros(T), np.zeros((T, K))
    q, lq, r = teacher(ids, logq, tail)
    for t in np.flatnonzero((ids >= 0).any(1)):
        z = logits(np.asarray(H)[t:t + 1], W, scale)
        lse[t] = lse_of(z)[0]
        mine = ids[t][ids[t] >= 0]
        others = np.delete(z[0], np.unique(mine))
        if not tail:
            rest[t] = lse[t]
        else:
            rest[t] = lse_of(others[None])[0] if others.size else -np.inf
        for k in range(K):
            if ids[t, k] < 0:
                continue
            hit[t, k] = z[0, ids[t, k]]
            if q[t, k] > 0:
                loss[t] += q[t, k] * (lq[t, k] - hit[t, k] + lse[t])
        if r[t] > 0 and others.size:
            loss[t] += r[t] * (np.log(r[t]) - rest[t] + lse[t])
    return loss, lse, rest, hit


def vocab_distill_backward(H, W, ids, logq, dloss, scale=1.0, tail=True):
    """(dH, dW, G); G (T x V) is zero for rows without entries."""
    H, W, ids = np.asarray(H, np.float64), np.asarray(W, np.float64), np.asarray(ids)
    dloss = np.asarray(dloss, np.float64)
    q, _, r = teacher(ids, logq, tail)
    G = np.zeros((len(H), len(W)))
    for t in np.flatnonzero((ids >= 0).any(1)):
        z = logits(H[t:t + 1], W, scale)[0]
        p = np.exp(z - lse_of(z[None])[0])
        mine = ids[t] >= 0
        out = np.ones(len(W), bool)
        out[ids[t][mine]] = False
        rt = r[t] if out.any() else 0.0
        g = (q[t].sum() + rt) * p
        np.subtract.at(g, ids[t][mine], q[t][mine])
        if tail and out.any():
            g[out] -= rt * np.exp(z[out] - lse_of(z[None, out])[0])
        G[t] = g * dloss[t] * scale
    use = (ids >= 0).any(1)
    return np.where(use[:, None], G @ W, 0.0), G[use].T @ H[use], G
