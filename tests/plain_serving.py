"""Plain 64-bit forms of the serving-step operators (shared-prefix decode, rotary queries, rotating
append), written from their definitions in numpy. Test infrastructure only."""
import math

import numpy as np

D_QK, D_V, BLK = 576, 512, 64


def visible(n, s_q, t, causal):
    n = max(int(n), 0)
    return min(max(n - s_q + t + 1, 0), n) if causal else n


def decode_shared(q, kv, shared_table, block_table, seqlens, scale, causal):
    """q float64 [b, s_q, h, 576], kv float64 [blocks, 64, 576]. Returns out, lse, mix (the probability-
    weighted mean of |value|) and span (the largest scale * sum |q_i k_i| of the row)."""
    b, s_q, h, _ = q.shape
    nb = len(shared_table)
    out, mix = np.zeros((b, s_q, h, D_V)), np.zeros((b, s_q, h, D_V))
    lse, span = np.full((b, h, s_q), -np.inf), np.zeros((b, s_q, h))
    for i in range(b):
        n = max(int(seqlens[i]), 0)
        w = (n + BLK - 1) // BLK
        table = [int(shared_table[j]) if j < nb else int(block_table[i, j]) for j in range(w)]
        keys = kv[table].reshape(-1, D_QK)[:n] if w else np.zeros((0, D_QK))
        for t in range(s_q):
            k = keys[:visible(n, s_q, t, causal)]
            if not len(k):
                continue
            s = scale * (q[i, t] @ k.T)
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(axis=1, keepdims=True)
            out[i, t] = (e / l) @ k[:, :D_V]
            mix[i, t] = (e / l) @ np.abs(k[:, :D_V])
            lse[i, :, t] = (m + np.log(l))[:, 0]
            span[i, t] = (scale * (np.abs(q[i, t]) @ np.abs(k).T)).max(axis=1)
    return out, lse, mix, span


def inv_freq(base=10000.0, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    out = []
    for i in range(32):
        f = base ** (-2.0 * i / 64)
        if factor > 1.0:
            share = 1.0
            if original_len:
                pair_of = lambda turns: 64 * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
                low = min(max(math.floor(pair_of(beta_fast)), 0), 63)
                high = min(max(math.ceil(pair_of(beta_slow)), 0), 63)
                high = high if high > low else low + 0.001
                share = min(max((i - low) / (high - low), 0.0), 1.0)
            f = f * (1 - share) + f / factor * share
        out.append(f)
    return np.array(out)


def rotate(x, pos, freq, interleaved, magnitude=1.0):
    """x float64 [..., 64] turned to positions pos (broadcast against x[..., 0])."""
    a = np.asarray(pos, dtype=np.float64)[..., None] * freq
    c, s = magnitude * np.cos(a), magnitude * np.sin(a)
    y = np.empty(np.broadcast_shapes(x.shape[:-1], a.shape[:-1]) + (64,))
    first, second = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


def append_values(x, pos, freq, interleaved, magnitude=1.0, weight=None, eps=1e-6):
    """The 576 values (float64, unrounded) that token rows x [tokens, 576] are stored as."""
    lat = x[:, :D_V]
    if weight is not None:
        lat = lat / np.sqrt((lat ** 2).mean(axis=1, keepdims=True) + eps) * weight
    return np.concatenate([lat, rotate(x[:, D_V:], pos, freq, interleaved, magnitude)], axis=1)
