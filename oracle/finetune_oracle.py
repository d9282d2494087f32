"""CPU oracle (numpy, fp64) of the gated feed-forward and fine-tuning calls,
written from their formulas in include/mbok.h.  Test infrastructure only; it
shares no code with the library.  Every function returns, beside its values,
the sum of absolute terms that an error bound scales with.
"""
from __future__ import annotations

import numpy as np

from oracle import mbok_oracle as O


def _sigmoid(a: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def planes(packed: np.ndarray, K: int, M: int, N: int) -> np.ndarray:
    """fp64 [K][M][N] of +-1."""
    return O.unpack_bits(packed, K, M, N).astype(np.float64)


def project(packed, alpha_mgk, K, M, N, x):
    """W x for each row of x, and sum_k sum_j |alpha_k x_j| (every term of
    every kernel: what a sum taken kernel by kernel rounds against)."""
    a = np.repeat(np.asarray(alpha_mgk, dtype=np.float64), 128, axis=1)      # [M][N][K]
    W = np.einsum("mnk,kmn->mn", a, planes(packed, K, M, N))
    return x @ W.T, np.abs(x) @ np.abs(a).sum(2).T


def silu(a: np.ndarray) -> np.ndarray:
    return a * _sigmoid(a)


def gated_grad(dh, g, u):
    """dgate, dup, h and the absolute terms of dgate."""
    s = _sigmoid(g)
    return dh * u * (s + g * s * (1 - s)), dh * g * s, g * s * u, np.abs(dh * u) * (s + np.abs(g) * s * (1 - s))


def layer_grad(mats, N, X, dYs):
    """mats: (packed, alpha [M][G][K], K, M) of matrices that share X [T][N];
    dYs their output gradients [T][M].  Returns dX with its absolute terms, and
    per matrix dalpha [M][G][K] with its absolute terms."""
    dX, E = np.zeros_like(X), np.zeros_like(X)
    das = []
    for (packed, alpha, K, M), dY in zip(mats, dYs):
        B = planes(packed, K, M, N)
        a = np.repeat(np.asarray(alpha, dtype=np.float64), 128, axis=1)
        W = np.einsum("mnk,kmn->mn", a, B)
        dX += dY @ W
        E += np.abs(dY) @ np.abs(a).sum(2)
        C, A = dY.T @ X, np.abs(dY).T @ np.abs(X)
        G = N // 128
        das.append(((B * C).reshape(K, M, G, 128).sum(3).transpose(1, 2, 0),
                    np.repeat(A.reshape(M, G, 128).sum(2)[:, :, None], K, axis=2)))
    return dX, E, das


def distill(z, teacher, index, tau, weight, grad):
    """loss, lse, dz, and the probabilities q and listed p [T][V] (dense)."""
    T, V = z.shape
    loss, lse_out, dz = np.zeros(T), np.zeros(T), np.zeros((T, V))
    q_all, p_all = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        listed = (index[t] >= 0) & (index[t] < V) & (teacher[t] != -np.inf)
        if weight[t] == 0 or not listed.any():
            continue
        v = teacher[t][listed] / tau
        e = np.exp(v - v.max())
        p = e / e.sum()
        logp = v - v.max() - np.log(e.sum())
        y = z[t] / tau
        with np.errstate(invalid="ignore"):
            lse = y.max() + np.log(np.exp(y - y.max()).sum())
        c = index[t][listed]
        with np.errstate(invalid="ignore"):
            loss[t] = weight[t] * sum(pi * (lp - (y[ci] - lse)) for pi, lp, ci in zip(p, logp, c) if pi != 0)
        lse_out[t] = lse
        q_all[t] = np.exp(y - lse)
        np.add.at(p_all[t], c, p)
        dz[t] = grad[t] * weight[t] / tau * (q_all[t] - p_all[t])
    return loss, lse_out, dz, q_all, p_all
