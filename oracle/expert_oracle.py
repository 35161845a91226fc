"""fp64 oracle of the expert-layer operators (test infrastructure; shares no code
with the library): tokens sorted by expert and back, 8-bit operands with block
scales, and their products.  Plain NumPy, written from the definitions.

8-bit values are held as the numbers they stand for; rounding to the 8-bit grid
is done on exact numbers, from the definition of the type (e4m3: 3 mantissa bits,
smallest normal 2^-6, largest 448; e5m2: 2 bits, 2^-14, 57344).
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
F8 = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


def up128(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK * BLOCK


def expert_sort(ids: np.ndarray, E: int):
    """(offsets [E + 1], rows [T, k], tokens [T k]) of a stable sort by expert."""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            lists[e].append(p)
    offsets = np.zeros(E + 1, dtype=np.int64)
    rows = np.full(T * k, -1, dtype=np.int64)
    tokens = np.full(T * k, -1, dtype=np.int64)
    r = 0
    for e in range(E):
        for p in lists[e]:
            rows[p], tokens[r] = r, p // k
            r += 1
        offsets[e + 1] = r
    return offsets, rows.reshape(T, k), tokens


def dispatch(x: np.ndarray, tokens: np.ndarray) -> np.ndarray:
    out = np.zeros((len(tokens), x.shape[1]))
    for r, t in enumerate(tokens):
        if 0 <= t < len(x):
            out[r] = x[t]
    return out


def combine(y: np.ndarray, rows: np.ndarray, w=None):
    """(out [T, C], sum of the terms' sizes)."""
    T, k = rows.shape
    out = np.zeros((T, y.shape[1]))
    size = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < len(y):
                term = (1.0 if w is None else float(w[t, j])) * y[rows[t, j]]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_backward(dout: np.ndarray, y: np.ndarray, rows: np.ndarray, w=None):
    """(dy, dw, sum of the sizes of dw's terms)."""
    dy = np.zeros_like(y)
    dw = np.zeros(rows.shape)
    size = np.zeros(rows.shape)
    for t in range(rows.shape[0]):
        for j in range(rows.shape[1]):
            r = rows[t, j]
            if 0 <= r < len(y):
                dy[r] = (1.0 if w is None else float(w[t, j])) * dout[t]
                dw[t, j] = dout[t] @ y[r]
                size[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, size


def round8(v: np.ndarray, f8: str) -> np.ndarray:
    """Nearest number of the 8-bit type, ties to even; NaN stays, infinities (and
    what rounds past the largest number) become NaN in e4m3, infinities in e5m2."""
    bits, low, top = F8[f8]
    v = np.asarray(v, dtype=np.float64)
    out = np.array(v)
    fine = np.isfinite(v) & (v != 0)
    e = np.floor(np.log2(np.abs(v[fine])))
    e = np.where(np.exp2(e) > np.abs(v[fine]), e - 1, np.where(np.exp2(e + 1) <= np.abs(v[fine]), e + 1, e))
    step = np.exp2(np.maximum(e, low) - bits)
    out[fine] = np.rint(v[fine] / step) * step
    over = np.abs(out) > top
    out[over] = np.nan if f8 == "e4m3" else np.sign(out[over]) * np.inf
    return out


def _block(v: np.ndarray, f8: str, axes):
    """The library's fp32 arithmetic on blocks along `axes`: (q, scale with those axes kept)."""
    top = np.float32(F8[f8][2])
    a = np.abs(v)
    a = np.where(np.isfinite(a), a, np.float32(0)).astype(np.float32)
    s = np.maximum(a.max(axis=axes, keepdims=True) / top, np.float32(2.0 ** -126)).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        y = (v * (np.float32(1) / s)).astype(np.float32)
    return round8(y, f8), s


def quantize_rows(x: np.ndarray, f8: str):
    """x [R, C] float32: (q [R, Cp], scale [Cp/128, R])."""
    R, C = x.shape
    v = np.zeros((R, up128(C)), dtype=np.float32)
    v[:, :C] = x
    q, s = _block(v.reshape(R, -1, BLOCK), f8, (2,))
    return q.reshape(R, -1), s[:, :, 0].T


def quantize_tiles(x: np.ndarray, f8: str):
    """x [R, C] float32: (q [R, Cp], scale [Cp/128, Rp/128])."""
    R, C = x.shape
    v = np.zeros((up128(R), up128(C)), dtype=np.float32)
    v[:R, :C] = x
    q, s = _block(v.reshape(up128(R) // BLOCK, BLOCK, up128(C) // BLOCK, BLOCK), f8, (1, 3))
    return q.reshape(v.shape)[:R], s[:, 0, :, 0].T


def quantize_columns(x: np.ndarray, offsets, f8: str):
    """Sorted rows x [P, C] float32: (qt [C, cap], scale [cap/128, C])."""
    P, C = x.shape
    cap = BLOCK * (P // BLOCK + len(offsets) - 1)
    v = np.zeros((cap, C), dtype=np.float32)
    at = 0
    for a, b in zip(offsets[:-1], offsets[1:]):
        v[at:at + b - a] = x[a:b]
        at += up128(int(b - a))
    q, s = _block(v.reshape(-1, BLOCK, C), f8, (1,))
    return q.reshape(cap, C).T, s[:, 0]


def values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    """The fp64 values of a 2-D operand with row or tile scales."""
    R, K = q.shape
    r = np.arange(R) if s.shape[1] == R else np.arange(R) // BLOCK
    return q * s.astype(np.float64).T[r][:, np.arange(K) // BLOCK]


def product(a: np.ndarray, b: np.ndarray):
    """(A B^T, sum of the terms' sizes) of values."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def cut_off(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """What the 8-bit matrix instructions may lose: in every group of 8 consecutive
    k, each of the 7 products besides the largest, less than 2^-13 of it."""
    lost = np.zeros((len(a), len(b)))
    for k in range(0, a.shape[1], 8):
        lost += np.max(np.abs(a[:, None, k:k + 8] * b[None, :, k:k + 8]), axis=2, initial=0.0)
    return 7 * 2.0 ** -13 * lost
