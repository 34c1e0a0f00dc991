"""CPU oracle for linear attention with one decay per head and for the state pool's 8-bit
cache.

TEST INFRASTRUCTURE ONLY, like ``gdr_oracle``: plain NumPy in float64, written from the
definitions, a token at a time, with no code of the package. Rounds nothing unless
``round_out``: callers compare within bounds that count the roundings of the CUDA path.

    S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T       o_t = scale S_t^T q_t

Conventions are those of the gated delta rule's oracle: value head h reads query/key head
h // (H_v / H_qk); lengths are clamped to [0, T]; tokens behind the length are not read and
give zeros; an item whose slot is outside the pool is skipped; ``accepted`` selects how many
leading tokens the slot receives (None: all).
"""
from __future__ import annotations

import numpy as np

__all__ = ["linear_attention", "quantize", "dequantize", "E4M3_VALUES"]


def linear_attention(query, key, value, log_decay, pool, lengths, indices, accepted=None,
                     scale=1.0):
    """(out [B, H_v, T, D_v], pool after the call), both float64."""
    query, key, value = (np.asarray(x, np.float64) for x in (query, key, value))
    pool = np.array(pool, np.float64)
    B, H_qk, T, D_k = query.shape
    H_v, D_v = value.shape[1], value.shape[3]
    group = H_v // H_qk
    with np.errstate(over="ignore"):
        decay = np.exp(np.asarray(log_decay, np.float64))
    out = np.zeros((B, H_v, T, D_v))
    for b in range(B):
        s = int(indices[b])
        if not 0 <= s < pool.shape[0]:
            continue
        L = min(max(int(lengths[b]), 0), T)
        n = L if accepted is None else min(max(int(accepted[b]), 0), L)
        for h in range(H_v):
            S = pool[s, h].copy()
            kept = S.copy()
            for t in range(L):
                # a decay of 0 forgets even an infinite state
                S = decay[h] * S if decay[h] != 0 else np.zeros_like(S)
                S = S + np.outer(key[b, h // group, t], value[b, h, t])
                out[b, h, t] = scale * (query[b, h // group, t] @ S)
                if t + 1 == n:
                    kept = S.copy()
            pool[s, h] = kept
    return out, pool


def _e4m3_values():
    """The 127 finite magnitudes of e4m3 (codes 0 .. 126), ascending."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


E4M3_VALUES = _e4m3_values()
FLOOR = 2.0 ** -100


def _nearest_e4m3(x):
    """Codes (uint8) of the e4m3 values nearest to x, ties to the even code; |x| <= 448."""
    mag = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3_VALUES, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - E4M3_VALUES[lo], E4M3_VALUES[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantize(x, kind):
    """(codes, scales) of float values whose last axis is whole groups of 64, with the
    arithmetic of the definition in float32: scale = m / top, code = nearest(x * (top / m)).
    Codes are int8, or uint8 bit patterns for "e4m3"."""
    top = np.float32(448.0 if kind == "e4m3" else 127.0)
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    m = np.abs(g).max(-1)
    bad = ~np.isfinite(g).all(-1)
    some = ~bad & (m >= np.float32(FLOOR))
    safe = np.where(some, m, np.float32(1.0)).astype(np.float32)
    scale = np.where(some, (safe / top).astype(np.float32), np.float32(0.0))
    factor = np.where(some, (top / safe).astype(np.float32), np.float32(0.0))
    y = (np.where(bad[..., None], np.float32(0.0), g) * factor[..., None]).astype(np.float32)
    if kind == "e4m3":
        codes = _nearest_e4m3(np.clip(y.astype(np.float64), -448.0, 448.0))
    else:
        codes = np.rint(y).astype(np.int8)
    scale = np.where(bad, np.float32("nan"), scale).astype(np.float32)
    return codes.reshape(x.shape), scale


def dequantize(codes, scales, kind):
    """float64 values code * scale (the product rounded to float32, as stored scales are)."""
    codes = np.asarray(codes)
    if kind == "e4m3":
        u = codes.view(np.uint8)
        table = np.append(E4M3_VALUES, np.nan)
        values = table[u & 127] * np.where(u & 128, -1.0, 1.0)
    else:
        values = codes.astype(np.float64)
    scales = np.repeat(np.asarray(scales, np.float32), 64, -1)
    return (values.astype(np.float32) * scales).astype(np.float64)
