"""CPU oracle of 4-bit weights with group scales (numpy, float64).

TEST INFRASTRUCTURE ONLY, like moe_oracle.py.  Plain definitions; pinned by
tests/test_few_host.py against exact rational arithmetic and hand-worked cases.
"""
from __future__ import annotations

import numpy as np


def q4_values(codes, scales, zeros, group: int) -> np.ndarray:
    """W[..., n, k] = s (q - z) of codes [..., N, K] (one number each), scales and zeros
    [..., N, groups] (zeros None: 8)."""
    K = codes.shape[-1]
    wide = lambda a: np.repeat(np.asarray(a, dtype=np.float64), group, axis=-1)[..., :K]
    return wide(scales) * (np.asarray(codes, dtype=np.float64) - (8.0 if zeros is None else wide(zeros)))


def q4_unpair(pairs) -> np.ndarray:
    """Codes of row-major bytes: input 2j in the low half of byte j."""
    p = np.asarray(pairs, dtype=np.int64)
    return np.stack([p % 16, p // 16], axis=-1).reshape(*p.shape[:-1], -1)


def q4_tile(codes, N: int, K: int) -> np.ndarray:
    """The library's order of one matrix's codes [N, K]: bytes of 1 KB tiles of 16 x 128,
    codes outside the matrix 0."""
    nt, kt = -(-N // 16), -(-K // 128)
    out = np.zeros((nt, kt, 256), dtype=np.uint32)
    for n in range(N):
        for k in range(K):
            r, c = n % 16, k % 128
            word = ((c // 8 % 4) * 16 + r) * 4 + c // 32
            out[n // 16, k // 128, word] |= np.uint32(int(codes[n, k]) << (4 * (c % 8 // 2) + 16 * (c % 2)))
    return out.reshape(-1).view(np.uint8)


def q4_quantise(w, group: int, zeros: bool, to_elt):
    """Codes [..., N, K], scales and zero points [..., N, groups] of weights w; `to_elt` rounds
    float64 values to the element type (and returns float64)."""
    w = np.asarray(w, dtype=np.float64)
    K = w.shape[-1]
    codes = np.zeros(w.shape, dtype=np.int64)
    ng = -(-K // group)
    scales, zp = np.zeros((*w.shape[:-1], ng)), np.zeros((*w.shape[:-1], ng), dtype=np.int64)
    for g in range(ng):
        v = w[..., g * group:(g + 1) * group]
        if zeros:
            lo, hi = np.minimum(v.min(-1), 0.0), np.maximum(v.max(-1), 0.0)
            s = to_elt((hi - lo) / 15.0)
        else:
            s = to_elt(np.abs(v).max(-1) / 7.0)
        one = np.where(s == 0, np.inf, s)
        z = np.clip(np.rint(-lo / one), 0, 15) if zeros else np.full(s.shape, 8.0)
        q = np.clip(np.rint(v / one[..., None]) + z[..., None], 0 if zeros else 1, 15)
        codes[..., g * group:(g + 1) * group] = q
        scales[..., g], zp[..., g] = s, z
    return codes, scales, zp if zeros else None
