"""The mixture-of-experts layer from its definition, in NumPy: Q4_0 weights and Q8_0 codes
by the f32 steps the definitions name, sums in 64 bits, with a bound on what f32 sums and the
rounding of h to int8 may change. Shares no code with the library."""
import numpy as np

F = np.float32


def dequant_q4_0(qs, d):
    """Codes (rows, K/2) bytes and fp16 scale bits (rows, K/32) -> (rows, K) f64."""
    q = np.asarray(qs, dtype=np.uint8).reshape(qs.shape[0], -1, 16).astype(np.int64)
    w = np.concatenate([q & 15, q >> 4], axis=2) - 8
    s = np.asarray(d).view(np.float16).astype(np.float64)
    return (w * s[:, :, None]).reshape(qs.shape[0], -1)


def q8_0(x):
    """(codes, scales) of f32 rows: d = amax/127, codes x * (1/d) rounded half away from zero."""
    b = np.asarray(x, dtype=F).reshape(x.shape[0], -1, 32)
    d = (np.max(np.abs(b), axis=2) / F(127)).astype(F)
    inv = np.where(d > 0, F(1) / np.where(d > 0, d, F(1)), F(0)).astype(F)
    v = (b * inv[:, :, None]).astype(F).astype(np.float64)
    return np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127), d


def values(codes, d):
    return (codes * d.astype(np.float64)[:, :, None]).reshape(codes.shape[0], -1)


def route(x, wr, top_k, renorm):
    """(ids, weights, logits): largest logits first, the lower index on ties."""
    logits = np.asarray(x, dtype=np.float64) @ np.asarray(wr, dtype=np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    e = np.exp(logits - logits.max(1, keepdims=True))
    chosen = np.take_along_axis(e, ids, 1)
    return ids, chosen / (chosen if renorm else e).sum(1, keepdims=True), logits


def experts(x, ids, weights, gu, dn, rel):
    """(y, bound): the layer for dequantised experts gu (E, 2I, H) and dn (E, H, I). `rel` is
    the error of one f32 dot relative to the sum of its terms' magnitudes. The bound follows
    that error through h = g / (1 + exp(-g)) * u (|silu'| < 1.1; expf, the division and the
    product within 4 steps of 2^-24 each), through the scale of a 32-block of h, and counts
    a whole step of the code for every h that lies so close to a rounding border that its
    error may carry it across."""
    T, H = x.shape
    E, I = gu.shape[0], gu.shape[1] // 2
    xv = values(*q8_0(x))
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for s in range(ids.shape[1]):
            e = ids[t, s]
            if e < 0 or e >= E:
                continue
            gus, size = gu[e] @ xv[t], rel * (np.abs(gu[e]) @ np.abs(xv[t]))
            g, u, dg, du = gus[:I], gus[I:], size[:I], size[I:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = silu * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 16 * 2.0 ** -24 * np.abs(h) + 2.0 ** -120
            hb, db = h.reshape(-1, 32), dh.reshape(-1, 32)
            amax = np.abs(hb).max(1, keepdims=True)
            d = amax / 127
            dd = db.max(1, keepdims=True) / 127 + 2.0 ** -23 * d
            inv = np.where(d > 0, 1 / np.where(d > 0, d, 1), 0)
            v = hb * inv
            dv = db * inv + np.abs(v) * dd * inv + 2.0 ** -22 * np.abs(v)
            codes = np.sign(v) * np.floor(np.abs(v) + 0.5)
            near = np.abs(np.abs(v) - np.floor(np.abs(v)) - 0.5) <= dv
            flip = np.where(near, np.ceil(dv), 0) * (d + dd) + np.abs(codes) * dd
            hv = (codes * d).reshape(-1)
            w = weights[t, s]
            y[t] += w * (dn[e] @ hv)
            A = np.abs(dn[e])
            bound[t] += abs(w) * (A @ flip.reshape(-1) + rel * (A @ np.abs(hv + flip.reshape(-1))))
    return y, bound + 8 * 2.0 ** -24 * np.abs(y) + 2.0 ** -120
