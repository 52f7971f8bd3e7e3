"""Plain CPU oracle of the block-scaled E4M3 operators of the experts.

TEST INFRASTRUCTURE. Imported only by the tests and ``__graft_entry__.smoke()``; it shares no code
with the CUDA path.

Format (the header ``include/moe.h`` states it): E4M3 codes and one E8M0 byte b per block of 128
values, worth 2^(b - 127), the least power of two with amax / scale <= 448, not below 2^-126, and 1
for an all-zero block; a code is the nearest E4M3 value to v / scale, ties to the even code.
Everything below is evaluated in fp64: scales by comparing amax with 448 * 2^j, codes by
:func:`oracle.moe_fp8.e4m3_encode` on the exact quotient, products as fp64 matrix products of the
values the codes stand for.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

from .moe_fp8 import e4m3_decode, e4m3_encode

__all__ = ["BLOCK", "scale_bytes", "scale_values", "quantize_rows", "quantize_weight",
           "quantize_tokens", "token_blocks", "values_rows", "values_weight", "values_tokens",
           "experts_of", "gemm", "wgrad", "swiglu", "swiglu_backward"]

BLOCK = 128
_LIMIT = np.ldexp(448.0, np.arange(-126, 128))       # 448 * 2^j


def scale_bytes(amax) -> np.ndarray:
    """E8M0 byte of blocks with these largest magnitudes."""
    amax = np.asarray(amax, np.float64)
    j = np.searchsorted(_LIMIT, amax, side="left") - 126   # least j with 448 2^j >= amax
    return np.where(amax > 0, j + 127, 127).astype(np.uint8)


def scale_values(b) -> np.ndarray:
    return np.ldexp(1.0, np.asarray(b, np.int64) - 127)


def _nblocks(n: int) -> int:
    return -(-n // BLOCK)


def _spread(s, n: int, axis: int) -> np.ndarray:
    """Block scales repeated to `n` values along `axis`."""
    return np.take(np.repeat(s, BLOCK, axis=axis), np.arange(n), axis=axis)


def quantize_rows(M) -> Tuple[np.ndarray, np.ndarray]:
    M = np.asarray(M, np.float64)
    R, C = M.shape
    b = np.stack([scale_bytes(np.abs(M[:, i:i + BLOCK]).max(axis=1)) for i in range(0, C, BLOCK)], 1) \
        if R else np.zeros((0, _nblocks(C)), np.uint8)
    return e4m3_encode(M / _spread(scale_values(b), C, 1)), b


def quantize_weight(W) -> Tuple[np.ndarray, np.ndarray]:
    W = np.asarray(W, np.float64)
    E, R, C = W.shape
    b = np.zeros((E, _nblocks(R), _nblocks(C)), np.uint8)
    for i in range(b.shape[1]):
        for j in range(b.shape[2]):
            blk = W[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            b[:, i, j] = scale_bytes(np.abs(blk).max(axis=(1, 2)))
    return e4m3_encode(W / _spread(_spread(scale_values(b), R, 1), C, 2)), b


def experts_of(offsets: Sequence[int]) -> List[Tuple[int, int]]:
    return [(int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def token_blocks(rows: int, E: int) -> int:
    """The most blocks that any split of `rows` rows among E experts fills: each of the
    min(rows, E) experts with a row wastes at most 127 places."""
    return (rows + 127 * min(rows, E)) // BLOCK


def quantize_tokens(M, offsets) -> Tuple[np.ndarray, np.ndarray]:
    """Codes [C, 128 n] and bytes [n, C] of the n blocks that the experts' rows fill."""
    M = np.asarray(M, np.float64)
    codes, bytes_ = [], []
    for a, z in experts_of(offsets):
        for r in range(a, z, BLOCK):
            blk = M[r:min(r + BLOCK, z)]
            b = scale_bytes(np.abs(blk).max(axis=0))
            q = np.zeros((M.shape[1], BLOCK), np.uint8)
            q[:, :blk.shape[0]] = e4m3_encode(blk / scale_values(b)).T
            codes.append(q)
            bytes_.append(b)
    if not codes:
        return np.zeros((M.shape[1], 0), np.uint8), np.zeros((0, M.shape[1]), np.uint8)
    return np.concatenate(codes, 1), np.stack(bytes_)


def values_rows(q, b) -> np.ndarray:
    q = np.asarray(q)
    return e4m3_decode(q) * _spread(scale_values(b), q.shape[1], 1)


def values_weight(q, b) -> np.ndarray:
    q = np.asarray(q)
    s = _spread(_spread(scale_values(b), q.shape[1], 1), q.shape[2], 2)
    return e4m3_decode(q) * s


def values_tokens(q_t, b_t) -> np.ndarray:
    q_t = np.asarray(q_t)
    return e4m3_decode(q_t) * _spread(scale_values(b_t).T, q_t.shape[1], 1)


def gemm(A, W, offsets, absolute: bool = False) -> np.ndarray:
    """A [R, k] per expert against W [E, n, k]; rows outside every expert are NaN. `absolute`: the
    sums of magnitudes, which bound the rounding of any order of summation."""
    A, W = (np.abs(A), np.abs(W)) if absolute else (A, W)
    out = np.full((A.shape[0], W.shape[1]), np.nan)
    for e, (a, z) in enumerate(experts_of(offsets)):
        out[a:z] = A[a:z] @ W[e].T
    return out


def wgrad(A, B, offsets, absolute: bool = False) -> np.ndarray:
    """Per expert A^T B over its rows, from values in row order."""
    A, B = (np.abs(A), np.abs(B)) if absolute else (A, B)
    return np.stack([A[a:z].T @ B[a:z] for a, z in experts_of(offsets)])


def swiglu(gu) -> np.ndarray:
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    return g / (1.0 + np.exp(-np.clip(g, -700, None))) * u


def swiglu_backward(gu, dh) -> Tuple[np.ndarray, np.ndarray]:
    """([d_gate | d_up], h)."""
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    dh = np.asarray(dh, np.float64)
    s = 1.0 / (1.0 + np.exp(-np.clip(g, -700, None)))
    return np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], 1), g * s * u
