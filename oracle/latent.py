"""RMS norm, the FP8 latent cache and latent attention in float64 (oracle; test infrastructure only).

All inputs are float64 arrays holding the exact values of the tensors' elements. Definitions:
  y = x / sqrt(mean(x^2) + eps) * w                                     (rmsnorm_ref)
  a token's scale = max(amax, 1e-10) / 448 rounded up to a power of two, held within
  2^-42 .. 2^40, as its exponent byte                                   (token_code_ref)
  o = softmax(scale q k^T over the keys a row sees) v; a row that sees none is zero
                                                                        (attention_ref)
Pinned by ``tests/test_oracle_latent.py``.
"""

from __future__ import annotations

import numpy as np


def rmsnorm_ref(x: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w


def token_code_ref(y: np.ndarray) -> np.ndarray:
    """UE8M0 codes of tokens y [T, D]; 255 for a token that is not finite."""
    amax = np.abs(y).max(axis=1)
    ok = np.isfinite(amax)
    mant, exp = np.frexp(np.maximum(np.where(ok, amax, 1.0), 1e-10) / 448.0)  # mant in [0.5, 1)
    code = 127 + exp - (mant == 0.5)
    return np.where(ok, np.clip(code, 127 - 42, 127 + 40), 255)


def e8m0_value(codes: np.ndarray) -> np.ndarray:
    codes = np.asarray(codes).astype(np.int64)
    return np.where(codes == 255, np.nan, np.exp2(np.where(codes == 255, 0, codes) - 127.0))


def attention_ref(q: np.ndarray, k: np.ndarray, v: np.ndarray, sees: np.ndarray, scale: float):
    """q [R, D], k [L, D], v [L, E]; row r sees keys 0 .. sees[r] - 1. Returns (o [R, E], the same
    average of |v|, the largest scale * sum |q||k| of a row), the latter two for error bounds."""
    o = np.zeros((q.shape[0], v.shape[1]))
    mag = np.zeros_like(o)
    reach = np.zeros(q.shape[0])
    for r in range(q.shape[0]):
        n = int(max(0, min(sees[r], k.shape[0])))
        if n == 0:
            continue
        s = scale * (k[:n] @ q[r])
        p = np.exp(s - s.max())
        p /= p.sum()
        o[r] = p @ v[:n]
        mag[r] = p @ np.abs(v[:n])
        reach[r] = abs(scale) * (np.abs(k[:n]) @ np.abs(q[r])).max()
    return o, mag, reach
