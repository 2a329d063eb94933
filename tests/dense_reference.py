"""Plain 64-bit forms of the paged cache, the dense attention and the draft verification, in
numpy, for the tests: loops over sequences, heads and tokens, written from the formulas."""
import numpy as np

E4M3 = None  # the 256 values, filled on first use


def e4m3_values():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; no
    infinities, 0x7f and 0xff are NaN."""
    global E4M3
    if E4M3 is None:
        v = np.zeros(256)
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            if e == 15 and m == 7:
                x = np.nan
            v[c] = -x if c & 128 else x
        E4M3 = v
    return E4M3


def encode_row(x):
    """(codes as values, exponent) of one row: the least e in [-100, 100] with
    max|x| <= 448 * 2^e over the finite values, each value to the nearest code, ties to the code
    whose last mantissa bit is 0."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    top = np.abs(x[fine]).max() if fine.any() else 0.0
    e = -100
    while e < 100 and top > 448.0 * 2.0 ** e:
        e += 1
    grid = e4m3_values()[:127]  # ascending, even codes have last bit 0
    y = np.abs(np.where(fine, x, 0.0)) * 2.0 ** -e
    hi = np.clip(np.searchsorted(grid, y), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - grid[lo], grid[hi] - y
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(y >= 448.0, 126, pick)
    out = np.where(fine, np.copysign(grid[pick], x), np.nan)
    return out, e


def attend(q, k, v, first, scale, causal=True):
    """q [m][H_q][d] at positions first .., k, v [n][H_kv][d]: (out, lse) in 64 bits; a token
    that sees nothing gives 0 and -inf, and a cell a token does not see is never touched."""
    m, H_q, d = q.shape
    n, H_kv = k.shape[:2]
    out, lse = np.zeros((m, H_q, d)), np.full((m, H_q), -np.inf)
    for i in range(m):
        see = min(n, max(0, first + i + 1)) if causal else n
        if see == 0:
            continue
        for h in range(H_q):
            g = h * H_kv // H_q
            s = scale * (k[:see, g].astype(np.float64) @ q[i, h].astype(np.float64))
            t = s.max()
            w = np.exp(s - t)
            out[i, h] = (w @ v[:see, g].astype(np.float64)) / w.sum()
            lse[i, h] = t + np.log(w.sum())
    return out, lse


def attend_weights_abs(q, k, v, first, scale, causal=True):
    """sum_j softmax_j |v_j|, the magnitude that bounds the roundings of an output."""
    return attend(q, k, np.abs(v), first, scale, causal)[0]


def verify(p, q, tokens, n_draft, u):
    """One sequence: p [n+1 or more][V], q [n][V] or None.  (tokens out, accepted)."""
    D, V = p.shape[0] - 1, p.shape[1]
    n = min(max(int(n_draft), 0), D)
    a = n
    for j in range(n):
        t = int(tokens[j])
        ok = 0 <= t < V
        if ok:
            qt = 1.0 if q is None else float(q[j, t])
            ok = float(u[j]) * qt < float(p[j, t])
        if not ok:
            a = j
            break
    w = p[a].astype(np.float64)
    w = np.where(w > 0, w, 0.0)
    if a < n:
        if q is None:
            rest = w.copy()
            if 0 <= tokens[a] < V:
                rest[tokens[a]] = 0
        else:
            rest = p[a].astype(np.float64) - q[a].astype(np.float64)
            rest = np.where(rest > 0, rest, 0.0)
        if rest.sum() > 0:
            w = rest
    c = np.cumsum(w)
    out = np.full(D + 1, -1, np.int32)
    out[:a] = tokens[:a]
    if c[-1] > 0:
        over = np.flatnonzero(c > float(u[D]) * c[-1])
        out[a] = over[0] if over.size else np.flatnonzero(w > 0)[-1]
    return out, a
