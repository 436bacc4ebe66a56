"""Plain CPU restatement of the training operators — test infrastructure only: SiLU * up with dropout and its
backward, the grouped products for input and weight gradients, the gradient of the router's logits, and the
whole layer's loss gradient.  fp64 throughout; the operators' definitions are those of
``include/training/moe_training.h``.
"""
from __future__ import annotations

import numpy as np

__all__ = ["philox4x32", "dropout_factors", "silu_mul_dropout", "silu_mul_backward", "grouped_dgrad", "grouped_wgrad",
           "route_backward", "train_layer"]


def philox4x32(counter, key):
    """Philox 4x32-10 (Salmon et al., SC 2011): four counter words and two key words to four random words, on
    Python ints or arrays of them (as uint64)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k0, k1 = (int(v) for v in key)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        hi0, lo0 = np.divmod(c[0] * np.uint64(0xD2511F53), np.uint64(1 << 32))
        hi1, lo1 = np.divmod(c[2] * np.uint64(0xCD9E8D57), np.uint64(1 << 32))
        c = [hi1 ^ c[1] ^ np.uint64(k0), lo1, hi0 ^ c[3] ^ np.uint64(k1), lo0]
        k0, k1 = (k0 + 0x9E3779B9) % 2**32, (k1 + 0xBB67AE85) % 2**32
    return [v & low for v in c]


def dropout_factors(pairs, n: int, p: float, seed: int, offset: int) -> np.ndarray:
    """[len(pairs), n]: 0 or 1 / (1 - p), p taken to a multiple of 2^-16."""
    below = min(65535, int(np.floor(p * 65536 + 0.5)))
    if below == 0:
        return np.ones((len(pairs), n))
    seed, offset = seed % 2**64, offset % 2**64
    chunk, pair = np.meshgrid(np.arange(-(-n // 8)), np.asarray(pairs), indexing="xy")
    one = np.ones_like(chunk).astype(np.uint64)
    w = philox4x32((chunk, pair, one * np.uint64(offset % 2**32), one * np.uint64(offset >> 32)),
                   (seed % 2**32, seed >> 32))
    r = np.stack([w[c // 2] >> np.uint64(16 * (c % 2)) & np.uint64(0xFFFF) for c in range(8)], axis=2)
    keep = r.reshape(len(pairs), 8 * r.shape[1])[:, :n] >= below
    return keep / (1.0 - below / 65536.0)


def _sigmoid(g):
    return 0.5 * (1.0 + np.tanh(0.5 * g))


def silu_mul_dropout(g, u, factors):
    return g * _sigmoid(g) * u * factors


def silu_mul_backward(g, u, d, w, factors):
    """(d_gate, d_up, w * h, d_w) of rows whose h is multiplied by w [rows] after the down projection."""
    s = _sigmoid(g)
    h = g * s * u * factors
    dh = w[:, None] * d * factors
    return dh * u * (s + g * s * (1.0 - s)), dh * g * s, w[:, None] * h, (d * h).sum(axis=1)


def _pairs_of(sorted_ids, offsets, e, num_pairs):
    """Sorted rows of expert e that hold a pair, and the pairs."""
    rows = np.arange(offsets[e], offsets[e + 1])
    p = sorted_ids[rows]
    real = (p >= 0) & (p < num_pairs)
    return rows[real], p[real]


def grouped_dgrad(dys, ws, sorted_ids, offsets, num_pairs, top_k, by_token):
    """sum over the pairs (dy, W [E, N, K]) of dy(r) W_e, and the same sum of magnitudes; zero rows elsewhere."""
    out = np.zeros((len(sorted_ids), ws[0].shape[2]))
    size = np.zeros_like(out)
    for e in range(ws[0].shape[0]):
        rows, p = _pairs_of(sorted_ids, offsets, e, num_pairs)
        for dy, w in zip(dys, ws):
            a = dy[p // top_k if by_token else rows]
            out[rows] += a @ w[e]
            size[rows] += np.abs(a) @ np.abs(w[e])
    return out, size


def grouped_wgrad(dy, x, sorted_ids, offsets, num_pairs, top_k, dy_by_token, x_by_token):
    """dy_e^T x_e for every expert, and the same sum of magnitudes."""
    E = len(offsets) - 1
    out = np.zeros((E, dy.shape[1], x.shape[1]))
    size = np.zeros_like(out)
    for e in range(E):
        rows, p = _pairs_of(sorted_ids, offsets, e, num_pairs)
        a, b = dy[p // top_k if dy_by_token else rows], x[p // top_k if x_by_token else rows]
        out[e] = a.T @ b
        size[e] = np.abs(a).T @ np.abs(b)
    return out, size


def route_backward(ids, w, dw, num_experts, logits=None):
    T, k = ids.shape
    out = np.zeros((T, num_experts))
    for t in range(T):
        ok = (ids[t] >= 0) & (ids[t] < num_experts)
        dot = (w[t] * dw[t])[ok].sum()
        if logits is None:
            np.add.at(out[t], ids[t][ok], (w[t] * (dw[t] - dot))[ok])
        else:
            np.add.at(out[t], ids[t][ok], dw[t][ok])
            p = np.exp(logits[t] - logits[t].max())
            out[t] = p / p.sum() * (out[t] - dot)
    return out


def train_layer(x, wg, wu, wd, ids, w, factors, d_out):
    """Output and gradients (d_x, d_w, d_wg, d_wu, d_wd) of out[t] = sum_j w[t, j] E_ids[t, j](x[t]), token by token
    and pair by pair, without a sorted layout.  ``factors`` [T * k, I]: dropout of each pair's hidden values."""
    T, k = ids.shape
    out, d_x, d_w = np.zeros_like(x), np.zeros_like(x), np.zeros((T, k))
    d_wg, d_wu, d_wd = np.zeros_like(wg), np.zeros_like(wu), np.zeros_like(wd)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if not 0 <= e < len(wg):
                continue
            g, u, f = wg[e] @ x[t], wu[e] @ x[t], factors[t * k + j]
            s = _sigmoid(g)
            h = g * s * u * f
            y = wd[e] @ h
            out[t] += w[t, j] * y
            d_w[t, j] = d_out[t] @ y
            dy = w[t, j] * d_out[t]
            d_wd[e] += np.outer(dy, h)
            dh = wd[e].T @ dy * f
            dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
            d_wg[e] += np.outer(dg, x[t])
            d_wu[e] += np.outer(du, x[t])
            d_x[t] += wg[e].T @ dg + wu[e].T @ du
    return out, d_x, d_w, d_wg, d_wu, d_wd
