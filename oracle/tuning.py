"""Plain CPU oracle of the operators that tune a packed model (test
infrastructure): 8-bit activation checkpoints, the gradient of a packed layer
from such a checkpoint, and softmax cross entropy over a vocabulary with its
gradient. float64 NumPy; it shares no code with the GPU library.

Source: the digest's section 方法步骤详情, stage 3 (the binary factors are
frozen and the scales tuned, there by the KL divergence from the original
model's outputs); the pages give no formula of a layer's gradient, nor of
checkpoints and of the cross entropy against labels that a model is scored by,
so these are the plain ones:

    checkpoint   e = least integer with max|x| <= 127 2^e over 32 columns of a
                 row, clamped to -126 .. 121 (9 for float16); c = x / 2^e to
                 even, in -127 .. 127; the value is c 2^e, NaN in a group that
                 held a NaN or an infinity
    layer        a = s2 * x, p = S_V^T a, q = S_U p, y = s1 * q:
                 ds1 = sum_t dy q, dp = S_U^T (s1 dy), da = S_V dp,
                 dx = s2 da, ds2 = sum_t da x
    loss         z = scale H W^T, lse = log sum exp z, loss = lse - z[label];
                 G = (exp(z - lse) - [label]) dloss scale, dH = G W, dW = G^T H
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def act8_quantize(x, top=121):
    """(codes int8, exps uint8) of x (rows x cols, any float type)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    g = np.zeros((rows, groups * GROUP))
    g[:, :cols] = x
    g = g.reshape(rows, groups, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    big = np.abs(g).max(-1)
    e = np.full(big.shape, -126)
    for k in range(-126, top):   # raise e while the step is too small
        e = np.where(big > 127.0 * 2.0 ** k, k + 1, e)
    c = np.clip(np.rint(g / np.exp2(e.astype(float))[..., None]), -127, 127)
    codes = c.reshape(rows, groups * GROUP)[:, :cols].astype(np.int8)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def act8_steps(exps):
    e = np.asarray(exps).astype(int)
    return np.where(e == 255, np.nan, np.exp2((e - 127).astype(float)))


def act8_values(codes, exps):
    cols = codes.shape[1]
    return codes.astype(np.float64) * np.repeat(act8_steps(exps), GROUP, 1)[:, :cols]


def layer_backward(SU, SV, s1, s2, x, dy):
    """(dx, ds1, ds2) for +-1 matrices SU (m x r), SV (n x r)."""
    SU, SV, s1, s2, x, dy = (np.asarray(v, np.float64) for v in (SU, SV, s1, s2, x, dy))
    q = ((x * s2) @ SV) @ SU.T
    da = ((dy * s1) @ SU) @ SV.T
    return da * s2, (dy * q).sum(0), (da * x).sum(0)


def vocab_loss(H, W, labels, scale=1.0):
    """(loss, lse); rows with a negative label are not looked at."""
    labels = np.asarray(labels)
    loss, lse = np.zeros(len(labels)), np.zeros(len(labels))
    use = labels >= 0
    if use.any():
        z = scale * np.asarray(H, np.float64)[use] @ np.asarray(W, np.float64).T
        top = z.max(1)
        lse[use] = top + np.log(np.exp(z - top[:, None]).sum(1))
        loss[use] = lse[use] - z[np.arange(len(z)), labels[use]]
    return loss, lse


def vocab_loss_backward(H, W, labels, dloss, scale=1.0):
    """(dH, dW, G) of sum dloss * loss, G for the used rows only."""
    H, W, labels = np.asarray(H, np.float64), np.asarray(W, np.float64), np.asarray(labels)
    dH, dW = np.zeros(H.shape), np.zeros(W.shape)
    use = labels >= 0
    _, lse = vocab_loss(H, W, labels, scale)
    G = np.exp(scale * H[use] @ W.T - lse[use][:, None])
    G[np.arange(len(G)), labels[use]] -= 1.0
    G *= np.asarray(dloss, np.float64)[use][:, None] * scale
    dH[use] = G @ W
    dW += G.T @ H[use]
    return dH, dW, G
