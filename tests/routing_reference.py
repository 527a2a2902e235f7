"""Plain definitions, in 64 bits and on the CPU, of routing from scores, the order of assignments by expert,
the combination of routed rows and low-rank adapters, with bounds of a float32 evaluation's rounding errors,
for the tests of the library's operators."""
import numpy as np

U = 2.0 ** -24  # a float32 rounding, relative


def scores(logits, softmax):
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if not softmax:
            return np.where(l >= 0, 1 / (1 + np.exp(-l)), np.exp(l) / (1 + np.exp(l)))
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0, top))
        total = e.sum(1, keepdims=True)
        return np.where(total == 0, 0, e / np.where(total == 0, 1, total))


def select(logits, k, softmax, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, bias=None, valid=None):
    """-> ids [T, k] (-1: none), weights [T, k], rows that hold what no choice is made from (weights NaN)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids, w = np.full((T, k), -1), np.zeros((T, k))
    bad = np.isnan(l).any(1) | (softmax & np.isposinf(l).any(1))
    s = scores(np.where(bad[:, None], 0, l), softmax)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    per = E // groups
    for t in range(T):
        if valid is not None and not valid[t]:
            bad[t] = False
            continue
        if bad[t]:
            w[t] = np.nan
            continue
        out = np.isneginf(l[t]) | np.isneginf(b) | np.isnan(b)
        c = np.where(out, -np.inf, s[t] + np.nan_to_num(b, nan=0.0, posinf=np.inf, neginf=0.0))
        # Experts of equal score in 64 bits (a sigmoid near 1) but other logits: the logits decide where there is no bias.
        key = c if bias is not None else np.where(out, -np.inf, l[t])
        if top_groups < groups:
            sums = []
            for g in range(groups):
                first = sorted((c if best == 2 or bias is not None else key)[g * per:(g + 1) * per], reverse=True)[:best]
                first = [v for v in first if v > -np.inf]
                sums.append(sum(first) if first else -np.inf)
            stay = [g for g in sorted(range(groups), key=lambda g: (-sums[g], g)) if sums[g] > -np.inf][:top_groups]
            key = np.where(np.isin(np.arange(E) // per, stay), key, -np.inf)
        chosen = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:k]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        lj, sj = l[t, chosen], s[t, chosen]
        if renorm and softmax:
            e = np.exp(lj - lj.max())
            w[t, :len(chosen)] = scale * e / e.sum()
        elif renorm:  # logs, as the scores may be smaller than any double
            g = np.minimum(lj, 0) - np.log1p(np.exp(-np.abs(lj)))
            e = np.exp(g - g.max())
            w[t, :len(chosen)] = scale * e / e.sum()
        else:
            w[t, :len(chosen)] = scale * sj
    return ids, w, bad


def select_gradient(logits, ids, w, dw, softmax, renorm, scale):
    """-> dlogits [T, E] and the sum of the magnitudes of its terms."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(np.where(np.isnan(l), 0, l), softmax)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        D = sum(dw[t, j] * w[t, j] for j in at)
        Da = sum(abs(dw[t, j] * w[t, j]) for j in at)
        for j in at:
            e = ids[t, j]
            v, m = w[t, j] * dw[t, j], abs(w[t, j] * dw[t, j])
            if renorm:
                v, m = v - w[t, j] * D / scale, m + abs(w[t, j] / scale) * Da
            f = 1.0 if softmax else 1 - s[t, e]
            if not softmax:
                f = np.exp(-l[t, e]) / (1 + np.exp(-l[t, e])) if l[t, e] >= 0 else 1 / (1 + np.exp(l[t, e]))
            d[t, e] += v * f
            size[t, e] += m * f
        if softmax and not renorm and at:
            d[t] -= s[t] * D
            size[t] += s[t] * Da
    return d, size


def order(ids, E):
    """-> counts [E], offsets [E + 1], the places of ids 0 .. E - 1 in a stable order."""
    flat = np.asarray(ids).reshape(-1)
    known = np.nonzero((flat >= 0) & (flat < E))[0]
    counts = np.bincount(flat[known], minlength=E)
    return counts, np.concatenate(([0], np.cumsum(counts))), known[np.argsort(flat[known], kind="stable")]


def combine(rows, ids, w, base, k):
    """rows [T * k, H] -> y [T, H] and a bound of its float32 error before the last rounding."""
    T, H = len(rows) // k, rows.shape[1]
    on = np.ones((T, k), bool) if ids is None else np.asarray(ids).reshape(T, k) >= 0
    w = np.ones((T, k)) if w is None else np.asarray(w, np.float64).reshape(T, k)
    r = np.where(on[:, :, None], np.asarray(rows, np.float64).reshape(T, k, H), 0)
    w = np.where(on, w, 0)
    b = np.zeros((T, H)) if base is None else np.asarray(base, np.float64)
    y = b + (w[:, :, None] * r).sum(1)
    return y, (k + 2) * U * (np.abs(b) + np.abs(w[:, :, None] * r).sum(1))


def combine_gradient(dy, rows, ids, w, k):
    """-> drows [T * k, H] (one rounding away from float32's), dweights [T, k] and its error bound."""
    T, H = dy.shape
    on = np.ones((T, k), bool) if ids is None else np.asarray(ids).reshape(T, k) >= 0
    w = np.ones((T, k)) if w is None else np.asarray(w, np.float64).reshape(T, k)
    r = np.where(on[:, :, None], np.asarray(rows, np.float64).reshape(T, k, H), 0)
    dy = np.asarray(dy, np.float64)[:, None, :]
    drows = np.where(on[:, :, None], w[:, :, None] * dy, 0)
    p = np.where(on[:, :, None], dy * r, 0)
    # H products of one rounding each and the sums, in some order.
    return drows.reshape(T * k, H), p.sum(2), (H + 8) * U * np.abs(p).sum(2)


def adapters(a, b, s, x, offsets, src, src_div, dst, base, y_rows, dy=None, f32=True):
    """a [n, r, K], b [n, N, r] float64, s [n]; src, dst by position.
    -> dict of y, h and, with dy, dx (rows named by src before the division), da, db: (values, bound) each, NaN where
    nothing is written.  f32: y is float32, h enters the second product with 24 bits instead of 16."""
    n, r, K = a.shape
    N, P = b.shape[1], len(src)
    part = 2.0 ** -23 if f32 else 2.0 ** -16
    out = {"y": [np.full((y_rows, N), np.nan), np.zeros((y_rows, N))], "h": [np.full((P, r), np.nan), np.zeros((P, r))]}
    if dy is not None:
        D = len(x) * src_div
        out["dx"] = [np.full((D, K), np.nan), np.zeros((D, K))]
        out["da"], out["db"] = [np.zeros((n, r, K)), np.zeros((n, r, K))], [np.zeros((n, N, r)), np.zeros((n, N, r))]
    for e in range(n):
        i = np.arange(offsets[e], offsets[e + 1])
        if not len(i):
            continue
        from_ok = (src[i] >= 0) & (src[i] // src_div < len(x))
        to_ok = (dst[i] >= 0) & (dst[i] < y_rows)
        xi = np.where(from_ok[:, None], x[np.where(from_ok, src[i] // src_div, 0)], 0)
        A, B = a[e], b[e]
        h = xi @ A.T
        # Exact products summed in float32: a rounding a sum, each of at most one step (2 U) of what the terms sum to.
        dh = 2 * (K + 8) * U * (np.abs(xi) @ np.abs(A).T)
        out["h"][0][i], out["h"][1][i] = h, dh
        hs, hd = s[e] * h, abs(s[e]) * dh + U * np.abs(s[e] * h)
        d = hs @ B.T
        # The parts of h (three products a rank where two or three parts), then their sum.
        dd = hd @ np.abs(B).T + (part + 2 * (3 * r + 8) * U) * (np.abs(hs) @ np.abs(B).T)
        to = dst[i[to_ok]]
        bb = np.zeros((len(to), N)) if base is None else base[to]
        out["y"][0][to] = bb + d[to_ok]
        out["y"][1][to] = dd[to_ok] + U * (np.abs(bb) + np.abs(d[to_ok]))
        if dy is None:
            continue
        g = np.where(to_ok[:, None], dy[np.where(to_ok, dst[i], 0)], 0)
        q = s[e] * (g @ B)
        qd = abs(s[e]) * 2 * (3 * N + 8) * U * (np.abs(g) @ np.abs(B)) + U * np.abs(q)
        v = q @ A
        rows = src[i[from_ok]]
        out["dx"][0][rows] = v[from_ok]
        out["dx"][1][rows] = (qd @ np.abs(A) + (2.0 ** -16 + 2 * (2 * r + 8) * U) * (np.abs(q) @ np.abs(A)))[from_ok]
        terms = 2.0 ** -23 + 2 * (6 * len(i) + 16) * U
        out["da"][0][e] = q.T @ xi
        out["da"][1][e] = qd.T @ np.abs(xi) + terms * (np.abs(q).T @ np.abs(xi))
        out["db"][0][e] = s[e] * (g.T @ h)
        out["db"][1][e] = abs(s[e]) * (np.abs(g).T @ dh + (terms + U) * (np.abs(g).T @ np.abs(h)))
    return out
