"""The vocabulary operators in 64 bits (numpy, row by row), with bounds of the fp32 error of the
kernels' arithmetic. u = 2^-24 is the fp32 unit roundoff."""
import numpy as np

U = 2.0 ** -24
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rounding(x, dtype):
    """Half a spacing of the storage type at |x|: what one rounding to it can move a value."""
    x = np.abs(x)
    if dtype == "float32":
        return x * U + 2.0 ** -150
    if dtype == "float16":
        return np.maximum(x * 2.0 ** -11, 2.0 ** -25)
    return x * 2.0 ** -8 + 2.0 ** -134


def process_logits(z, prompt, output, rep, freq, pres, bias, mask):
    """z [B, V] float64, lists of ids per row, bias lists of (id, value). Returns (y, error bound)."""
    y = z.copy()
    mag = np.abs(z)
    for b in range(z.shape[0]):
        count = {}
        for v in output[b]:
            count[v] = count.get(v, 0) + 1
        for v in set(prompt[b]) | set(count):
            y[b, v] = y[b, v] / rep[b] if y[b, v] > 0 else y[b, v] * rep[b]
            mag[b, v] = abs(y[b, v])
        for v, c in count.items():
            y[b, v] = y[b, v] - freq[b] * c - pres[b]
            mag[b, v] += abs(freq[b] * c) + abs(pres[b])
        for v, x in bias[b]:
            y[b, v] += x
            mag[b, v] += abs(x)
    most = 5 + max([len(x) for x in bias] + [0])
    if mask is not None:
        v = np.arange(z.shape[1])
        keep = (mask.astype(np.int64)[:, v // 32] >> (v % 32)) & 1
        y[keep == 0] = -np.inf
    return y, most * U * np.where(np.isfinite(mag), mag, 0.0)


def distill(z, ids, t, tau, lse, weight):
    """Per row: loss, stats (largest, sum, coefficient, L), gradient, and bounds of the fp32 error of loss,
    coefficient and gradient.

    Exponents: y = z c - M c carries two roundings of values up to m = 2 max|z| c, so 2^y is off by a
    factor 1 + e_y, e_y = 2 u m ln 2 + 2^-22 (the exponential itself). A sum of V positive terms by at
    least 128 threads, each in turn, then a tree, adds at most (V / 128 + 32) u."""
    N, V = z.shape
    out = dict(loss=np.zeros(N), stats=np.tile([0.0, 1.0, 0.0, 0.0], (N, 1)), grad=np.zeros((N, V)),
               loss_tol=np.zeros(N), coef_tol=np.zeros(N), grad_tol=np.zeros((N, V)))
    for n in range(N):
        on = ids[n] >= 0
        if not on.any():
            continue
        lt = t[n][on] / tau
        at = ids[n][on]
        if lse is None:
            if np.all(lt == -np.inf):
                continue
            big = lt.max()
            L = big + np.log(np.exp(lt - big).sum())
        else:
            L = lse[n]
            if L == -np.inf:
                continue
        with np.errstate(divide="ignore", invalid="ignore"):
            M = z[n].max()
            e = np.exp((z[n] - M) / tau)
            S = e.sum()
            p = e / S
            logp = (z[n] - M) / tau - np.log(S)
            q = np.exp(lt - L)
            loss = sum(qk * ((x - L) - logp[v]) for qk, x, v in zip(q, lt, at) if qk > 0)
            coef, r, u = 1.0, 0.0, np.nan
            off = np.ones(V, bool)
            off[at] = False
            if lse is not None:
                r, u = max(0.0, 1.0 - q.sum()), p[off].sum()
                if r > 0:
                    loss += r * (np.log(r) - np.log(u))
                    coef = 1.0 - r / u
            g = p * np.where(off, coef, 1.0)
            np.subtract.at(g, at, q)
        out["loss"][n] = tau * tau * loss
        out["stats"][n] = M, S, coef, L
        out["grad"][n] = weight[n] * tau * g
        K = len(at)
        finite = z[n][np.isfinite(z[n])]
        m = 2 * np.abs(finite).max() * 1.4427 / tau if finite.size else 0.0
        e_p = 2 * (2 * U * m * 0.7 + 2.0 ** -22) + (V / 128 + 32) * U
        e_q = (K + 16) * U + 4 * U * (np.abs(lt[np.isfinite(lt)]).max(initial=0.0) + abs(L))
        e_log = e_p + 4 * U * (m + abs(np.log(S)) + 1)
        d_r = q.sum() * (e_q + (K + 2) * U)
        tol = (q.sum() + abs(loss)) * (e_log + e_q) * 2 + e_q * np.abs(q[q > 0] * np.log(q[q > 0])).sum()
        tol += sum(abs(qk * (x - L - logp[v])) * e_q for qk, x, v in zip(q, lt, at) if qk > 0)
        d_coef = 0.0
        if r > 0:
            tol += d_r * (abs(np.log(r) - np.log(u)) + 1) + r * (e_p + 8 * U * (1 + abs(np.log(r)) + abs(np.log(u))))
            d_coef = (d_r + r * (e_p + 4 * U)) / u
        out["loss_tol"][n] = tau * tau * tol * (1 + 8 * U)
        out["coef_tol"][n] = d_coef + 2 * U
        d = p * np.where(off, abs(coef), 1.0) * (e_p + 8 * U) + np.where(off, p * d_coef, 0.0)
        np.add.at(d, at, q * (e_q + (K + 4) * U))
        out["grad_tol"][n] = abs(weight[n]) * tau * d
    return out


def e4m3(x):
    """x >= 0 rounded to the nearest E4M3 value (ties to even), saturating at 448."""
    if x <= 0:
        return 0.0
    e = max(int(np.floor(np.log2(x))), -6)
    return min(448.0, float(np.round(x / 2.0 ** (e - 3))) * 2.0 ** (e - 3))


def decode(codes, scales, rows, cols, fmt, g):
    """Values [rows, cols] in 64 bits, element by element from the documented layout; and codes and block scales."""
    n = 32 if fmt == "mx" else 16
    codes, flat = codes.reshape(rows, -1), scales.reshape(-1)
    tiles = -(-(-(-cols // 32) * (32 // n)) // 4)
    r, k = np.arange(rows)[:, None], np.arange(cols)[None]
    code = (codes[r, k // 2] >> (4 * (k % 2))) & 15
    j = k // n
    b = flat[((r // 128) * tiles + j // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4].astype(np.int64)
    if fmt == "mx":
        s = np.where(b == 255, np.nan, 2.0 ** (b.astype(float) - 127))
    else:
        e, f = (b >> 3) & 15, b & 7
        s = np.where(b == 0x7f, np.nan, np.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7.0), f * 2.0 ** -9))
    v = np.where(code >= 8, -GRID[code & 7], GRID[code & 7])
    return v * s * g, code, s
