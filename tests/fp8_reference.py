"""The FP8 block-scaled matmul from its definition, in NumPy: codes by the f32 steps the
definition names, contractions in 64 bits. Shares no code with the library."""
import numpy as np

F = np.float32


def e4m3_value(v):
    """v (f64) rounded to the nearest e4m3 value (3 mantissa bits, ties to even, spacing 2^-9
    below 2^-6), saturating at 448; NaN stays NaN."""
    v = np.clip(np.asarray(v, dtype=np.float64), -448.0, 448.0)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(v)
        step = np.exp2(np.maximum(e - 1, -6) - 3.0)
        return np.rint(v / step) * step


def decode(codes):
    """e4m3 code bytes -> values."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def _scale(amax):
    with np.errstate(over="ignore", invalid="ignore"):
        return np.maximum((amax.astype(F) / F(448.0)).astype(F), F(2.0 ** -126)).astype(F)


def _amax(a, axis):
    return np.max(np.where(np.isnan(a), F(0), np.abs(a)), axis=axis)


def quant_rows(x):
    """Values of the codes and scales of x (M, K), one scale per row and 128 columns."""
    x = np.asarray(x, dtype=F)
    M, K = x.shape
    nb = -(-K // 128)
    q, s = np.empty((M, K)), np.empty((M, nb), dtype=F)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for b in range(nb):
            xb = x[:, 128 * b: 128 * b + 128]
            s[:, b] = _scale(_amax(xb, 1))
            q[:, 128 * b: 128 * b + 128] = e4m3_value(xb * (F(1) / s[:, b: b + 1]))
    return q, s


def pack(w):
    """Values of the codes and scales of w (N, K), one scale per 128 x 128 tile."""
    w = np.asarray(w, dtype=F)
    N, K = w.shape
    q, s = np.empty((N, K)), np.empty((-(-N // 128), -(-K // 128)), dtype=F)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(s.shape[0]):
            for j in range(s.shape[1]):
                t = w[128 * i: 128 * i + 128, 128 * j: 128 * j + 128]
                s[i, j] = _scale(_amax(t, None))
                q[128 * i: 128 * i + 128, 128 * j: 128 * j + 128] = e4m3_value(t * (F(1) / s[i, j]))
    return q, s


def dequant(q, s):
    """Weight values of codes and tile scales (f64)."""
    N, K = q.shape
    return q * np.repeat(np.repeat(s.astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]


def gemm(x, wq, ws, bias=None):
    """(y, T): x quantised and multiplied with W^T; T = sum of the terms' magnitudes."""
    q, s = quant_rows(x)
    v = q * np.repeat(s.astype(np.float64), 128, 1)[:, : q.shape[1]]
    w = dequant(wq, ws)
    y, T = v @ w.T, np.abs(v) @ np.abs(w).T
    if bias is not None:
        y, T = y + bias, T + np.abs(bias)
    return y, T


def backward(dy, wq, ws):
    """(dx, T): dy quantised along N and multiplied with W."""
    q, s = quant_rows(dy)
    v = q * np.repeat(s.astype(np.float64), 128, 1)[:, : q.shape[1]]
    w = dequant(wq, ws)
    return v @ w, np.abs(v) @ np.abs(w)
