"""Plain definitions, in 64 bits and on the CPU, of the microscaled 4-bit format, the expert product
over it and the balance loss, for the tests of the library's operators."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x):
    """[R, C] float32 values -> (codes [R, C/2], scales [R, C/32]), one value after the other's definition."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    v = x.astype(np.float64).reshape(R, C // 32, 32)
    amax = np.abs(v).max(2)
    bad = ~np.isfinite(v).all(2)
    amax = np.where(bad | (amax == 0), 1.0, amax)
    power = np.where(np.abs(v).max(2) == 0, -127, np.frexp(amax)[1] - 1 - 2)
    power = np.maximum(power, -127)
    with np.errstate(invalid="ignore"):
        m = np.abs(v) / np.exp2(power.astype(np.float64))[..., None]
        far = np.abs(m[..., None] - GRID)
    # The nearest grid value; of two equally near ones the one whose mantissa bit (the code's lowest) is 0.
    best = far.min(-1, keepdims=True)
    near = far == best
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1)) | (np.signbit(v).astype(np.int64) << 3)
    code = np.where(bad[..., None], 0, code).reshape(R, C).astype(np.uint8)
    scales = np.where(bad, 255, power + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """-> float64 [..., C]; NaN where the scale byte is 255."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    q = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(q & 8, -GRID[q & 7], GRID[q & 7])
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def experts(w, x, offsets, src, dst, row_scale, y_rows, swiglu):
    """w[e] [n, k], x [x_rows, k] float64; src[i], dst[i] rows or out of range.
    -> y [y_rows, n_out] (NaN: not written), and a bound of its fp32 rounding errors."""
    n, K = w[0].shape
    n_out = n // 2 if swiglu else n
    y = np.full((y_rows, n_out), np.nan)
    err = np.zeros((y_rows, n_out))
    u = 2.0 ** -24
    for e in range(len(offsets) - 1):
        i = np.arange(offsets[e], offsets[e + 1])
        i = i[(0 <= dst[i]) & (dst[i] < y_rows)]
        if len(i) == 0:
            continue
        there = (0 <= src[i]) & (src[i] < len(x))
        rows, to, we = np.where(there[:, None], x[np.where(there, src[i], 0)], 0), dst[i], w[e].T
        z = rows @ we
        # K exact products summed in fp32 in some order: K roundings, each of at most one step (2 u)
        # of a partial sum that sum |w x| bounds.
        dz = 2 * (K + 8) * u * (np.abs(rows) @ np.abs(we))
        if swiglu:
            g, p, dg, dp = z[:, :n_out], z[:, n_out:], dz[:, :n_out], dz[:, n_out:]
            with np.errstate(over="ignore"):
                s = g / (1 + np.exp(-g))
            h = s * p
            # |silu'| <= 1.1; exp and reciprocal instructions a few steps, exp's argument |g| steps more.
            dh = 1.1 * dg * (np.abs(p) + dp) + np.abs(s) * dp + (16 + 4 * np.abs(g)) * u * np.abs(h)
            z, dz = h, dh
        if row_scale is not None:
            f = row_scale[to].astype(np.float64)[:, None]
            z, dz = z * f, dz * np.abs(f) + u * np.abs(z * f)
        y[to], err[to] = z, dz
    return y, err


def balance(logits, ids, valid, a, b, grad=1.0):
    """float64 -> losses [3], counts [E], mean_prob [E], n, dlogits [T, E]."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = ids.shape[1]
    keep = np.ones(T, bool) if valid is None else np.asarray(valid).astype(bool)
    counts = np.zeros(E, np.int64)
    for t in np.nonzero(keep)[0]:
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
    n = int(keep.sum())
    with np.errstate(invalid="ignore", divide="ignore"):
        top = logits.max(1, keepdims=True) if E else logits
        top = np.where(np.isneginf(top), 0, top)
        ex = np.exp(logits - top)
        tot = ex.sum(1, keepdims=True)
        p = np.where(tot == 0, 0, ex / tot)
        lse = np.where(tot[:, 0] == 0, 0, top[:, 0] + np.log(tot[:, 0]))
    if n == 0:
        return np.zeros(3), counts, np.zeros(E), 0, np.zeros_like(p)
    f = counts / (n * k)
    mean_prob = p[keep].sum(0) / n
    bal, z = E * (f * mean_prob).sum(), (lse[keep] ** 2).sum() / n
    d = grad * p * (a * E / n * (f - (p * f).sum(1, keepdims=True)) + 2 * b * lse[:, None] / n)
    return np.array([a * bal + b * z, bal, z]), counts, mean_prob, n, np.where(keep[:, None], d, 0)
