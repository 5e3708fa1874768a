"""Oracle of the e4m3 block format, its product and the routing of tokens to experts (NumPy).

Written from the definitions alone: the codes by searching the table of e4m3 values, the
products and sums in float64, the sort by Python's stable order.
"""
import numpy as np

MAX = 448.0


def _table():
    """Value of each code 0x00 .. 0x7e (the non-negative finite ones, ascending)."""
    v = []
    for c in range(0x7F):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


TABLE = _table()


def encode(q):
    """e4m3 codes nearest to q, ties to the even code, magnitudes above 448 held there."""
    q = np.asarray(q, np.float64)
    a = np.minimum(np.abs(q), MAX)
    hi = np.clip(np.searchsorted(TABLE, a), 1, len(TABLE) - 1)
    lo = hi - 1
    dl, dh = a - TABLE[lo], TABLE[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def decode(codes):
    codes = np.asarray(codes, np.uint8)
    full = np.concatenate([TABLE, [np.nan], -TABLE, [np.nan]])
    return full[codes]


def blocks(n):
    return -(-n // 128)


def spread(scales, n, axis):
    return np.take(np.repeat(scales, 128, axis=axis), np.arange(n), axis=axis)


def pack(x, rows=1):
    """(codes, scales) of x [M, K] float32 in blocks of rows x 128, by fp32 divisions."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    P, Q = -(-M // rows), blocks(K)
    pad = np.zeros((P * rows, Q * 128), np.float32)
    pad[:M, :K] = x
    pad = pad.reshape(P, rows, Q, 128)
    scales = (np.abs(pad).max(axis=(1, 3)) / np.float32(MAX)).astype(np.float32)
    scales[scales == 0] = 1.0
    with np.errstate(over="ignore", under="ignore"):
        q = (pad / scales[:, None, :, None]).astype(np.float32)
    return encode(q).reshape(P * rows, Q * 128)[:M, :K], scales


def dequant(codes, scales, rows=1):
    M, K = codes.shape
    s = scales.astype(np.float64)
    if rows > 1:
        s = np.take(np.repeat(s, rows, axis=0), np.arange(M), axis=0)
    return decode(codes) * spread(s, K, 1)


def gemm(x, xs, w, ws):
    """(y, sum of the products' magnitudes), both float64."""
    a, b = dequant(x, xs), dequant(w, ws, 128)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def silu_mul(x):
    x = np.asarray(x, np.float64)
    g, u = x[:, :x.shape[1] // 2], x[:, x.shape[1] // 2:]
    return g / (1 + np.exp(-g)) * u


def sort(ids, E):
    """(tokens, pos, offsets) of ids [T, k]."""
    T, k = ids.shape
    flat = [int(e) for e in ids.reshape(-1)]
    live = sorted((s for s in range(T * k) if 0 <= flat[s] < E), key=lambda s: flat[s])
    tokens = np.full(T * k, -1, np.int32)
    pos = np.full(T * k, -1, np.int32)
    for p, s in enumerate(live):
        tokens[p], pos[s] = s // k, p
    offsets = np.array([sum(1 for s in live if flat[s] < e) for e in range(E + 1)] if E <= 64 else
                       np.concatenate([[0], np.cumsum(np.bincount([flat[s] for s in live], minlength=E))]), np.int32)
    return tokens, pos.reshape(T, k), offsets


def combine(ys, pos, weights=None):
    """(out, sum of magnitudes), float64."""
    ys = np.asarray(ys, np.float64)
    T, k = pos.shape
    w = np.ones((T, k)) if weights is None else np.asarray(weights, np.float64)
    out, mag = np.zeros((T, ys.shape[1])), np.zeros((T, ys.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < len(ys):
                out[t] += w[t, j] * ys[pos[t, j]]
                mag[t] += np.abs(w[t, j] * ys[pos[t, j]])
    return out, mag
