"""CPU oracle of the rotary positions, the rotated int8 key/value cache and attention over it (NumPy, float64).

TEST INFRASTRUCTURE ONLY, as the other oracles. The pages describe neither
positions nor a cache. Readings (listed in the design notes):
  * A pair of channels turns by position * frequency on the pair's own axis.
  * A cell holds a head vector as the linear layer holds a token: rotated by
    H_128/sqrt(128), int8 codes, one float32 scale absmax/127, ties to even.
  * Attention takes its queries, keys and softmax as the INT8 attention does;
    the values are what their cells stand for.
"""

from __future__ import annotations

import numpy as np

from .attention_oracle import quantize_heads
from .convrot_oracle import rotate


def rope(x: np.ndarray, positions: np.ndarray, freq: np.ndarray, axis: np.ndarray, interleaved: bool = False,
         inverse: bool = False) -> np.ndarray:
    """x [B, S, H, D], positions [axes, B, S]; the turn as a complex product, pair by pair."""
    out = np.array(x, np.float64)
    half = len(freq)
    for i in range(half):
        if not 0 <= axis[i] < len(positions):
            continue
        angle = positions[axis[i]].astype(np.float64) * freq[i]
        turn = np.exp((-1j if inverse else 1j) * angle)[..., None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        z = (np.float64(1) * x[..., a] + 1j * x[..., b]) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


def cache_write(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Head vectors [..., 128] -> (codes int8, scale float32) of their cells."""
    return quantize_heads(x, 128)


def cache_value(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """What cells stand for: (codes * scale) R, in float64."""
    return rotate(np.asarray(codes, np.float64) * np.asarray(scale, np.float64)[..., None], 128)


def seen(length: int, news: int, tree=None) -> np.ndarray:
    """[news, length]: which keys the new tokens of a sequence see (the news are its last keys)."""
    out = np.zeros((news, max(length, 0)), bool)
    context = length - news
    for i in range(news):
        for j in range(length):
            m = j - context
            if m < 0:
                out[i, j] = True
            elif tree is None:
                out[i, j] = m <= i
            else:
                out[i, j] = m < 64 and bool((int(tree[i]) >> m) & 1)
    return out


def cache_attention(q: np.ndarray, k_codes, k_scale, v_codes, v_scale, see: np.ndarray, softmax_scale: float):
    """One sequence: q [news, Hq, 128]; codes [Hkv, length, 128], scales [Hkv, length].

    Returns (O [news, Hq, 128], weights [news, Hq, length] with rows of zeros where nothing is seen,
    the rotated queries' codes and scales)."""
    news, hq, _ = q.shape
    hkv, length, _ = k_codes.shape
    qc, sq = quantize_heads(q, 128)
    o = np.zeros(q.shape, np.float64)
    w = np.zeros((news, hq, length), np.float64)
    for h in range(hq):
        kv = h // (hq // hkv)
        s = (qc[:, h].astype(np.float64) @ k_codes[kv].astype(np.float64).T) * sq[:, h].astype(np.float64)[:, None] \
            * k_scale[kv].astype(np.float64)[None, :] * softmax_scale
        for i in range(news):
            on = see[i]
            if not on.any():
                continue
            e = np.exp(s[i, on] - s[i, on].max())
            w[i, h, on] = e / e.sum()
            o[i, h] = w[i, h, on] @ cache_value(v_codes[kv][on], v_scale[kv][on])
    return o, w, qc, sq
