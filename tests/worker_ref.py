"""Plain 64-bit forms of the operators that a worker runs before its gradients
are averaged (8-bit quantisation and product, distillation, balance loss), on
numpy arrays.  Written from the formulas in gar.h; no code of the package."""
import numpy as np

BLOCK = 128
# format -> (largest value, significand bits after the point, smallest normal exponent)
FORMATS = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}


def round_to_format(v, fmt):
    """v (float64) to the format's grid, ties to even; |v| within its range."""
    _, bits, emin = FORMATS[fmt]
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(v == 0, emin, np.floor(np.log2(np.abs(np.where(v == 0, 1.0, v)))))
    e = np.maximum(e, emin)
    quantum = np.exp2(e - bits)
    return np.rint(v / quantum) * quantum


def block_scales(x, fmt, square):
    """Scale bytes [rows, blocks] of x (float64), blocks of 128 columns (or 128 x 128)."""
    top = FORMATS[fmt][0]
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    out = np.zeros((rows, nb), np.int64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    for b in range(nb):
        m = a[:, b * BLOCK:(b + 1) * BLOCK].max(axis=1)
        if square:
            m = np.concatenate([np.full(min(BLOCK, rows - r), m[r:r + BLOCK].max()) for r in range(0, rows, BLOCK)])
        k = np.full(rows, -126)
        for i in range(rows):
            while m[i] > top * 2.0 ** k[i]:
                k[i] += 1
        out[:, b] = k + 127
    return out


def quantize(x, fmt, square):
    """(values / scale as float64 with NaN for NaN and infinities, scale bytes) of x (any float array)."""
    x = np.asarray(x, np.float64)
    s = block_scales(x, fmt, square)
    scale = np.repeat(np.exp2(s - 127.0), BLOCK, axis=1)[:, :x.shape[1]]
    v = np.where(np.isfinite(x), x, 0.0) / scale
    return np.where(np.isfinite(x), round_to_format(v, fmt), np.nan), s


def pack_scales(s):
    """[rows, blocks] -> the library's [ceil(blocks / 4), rows, 4], 1 past the end."""
    rows, nb = s.shape
    g = -(-nb // 4)
    out = np.ones((g, rows, 4), np.uint8)
    for b in range(nb):
        out[b // 4, :, b % 4] = s[:, b]
    return out


def distill(z, index, teacher, tau, weight):
    """(loss, lse, dz, q, p per entry) in float64."""
    z = np.asarray(z, np.float64)
    rows, vocab = z.shape
    loss, lse = np.zeros(rows), np.zeros(rows)
    dz, q = np.zeros_like(z), np.zeros_like(z)
    p = np.zeros(index.shape)
    with np.errstate(all="ignore"):
        for r in range(rows):
            on = (index[r] >= 0) & (index[r] < vocab) & (teacher[r] > -np.inf)
            if weight[r] == 0 or not on.any():
                continue
            t = teacher[r][on].astype(np.float64) / tau
            lp = t - t.max() - np.log(np.exp(t - t.max()).sum())
            y = z[r] / tau
            m = y.max()
            if m == -np.inf:
                lse[r], loss[r] = -np.inf, np.inf
            else:
                log_sum = np.log(np.exp(y - m).sum())  # kept apart from m, which may be too large to add it to
                lse[r] = m + log_sum
                q[r] = np.exp(y - m - log_sum)
                e = np.exp(lp)
                loss[r] = sum(e[j] * (lp[j] + log_sum - (y[i] - m)) for j, i in enumerate(index[r][on]) if e[j] > 0)
            p[r, on] = np.exp(lp)
            dz[r] = q[r]
            np.subtract.at(dz[r], index[r][on], np.exp(lp))
            dz[r] *= weight[r] / tau
    return loss, lse, dz, q, p


def balance(z, k, alpha, valid=None):
    """(choices, counts, loss, dz, scale) over the list of workers' logits, in
    float64; scale[w][t, e] = coef p max |c - mean|, what dz's error is measured in."""
    z = [np.asarray(a, np.float64) for a in z]
    E = z[0].shape[1]
    choices, counts, ps = [], [], []
    n = 0
    with np.errstate(invalid="ignore"):
        for w, a in enumerate(z):
            c = np.full((a.shape[0], k), -1, np.int32)
            p = np.zeros_like(a)
            cnt = np.zeros(E, np.int64)
            for t in range(a.shape[0]):
                usable = [e for e in range(E) if a[t, e] > -np.inf]
                if (valid is not None and not valid[w][t]) or not usable:
                    continue
                n += 1
                best = sorted(usable, key=lambda e: (-a[t, e], e))[:k]
                c[t, :len(best)] = best
                cnt[best] += 1
                x = np.exp(a[t] - np.max(a[t][usable]))
                p[t] = x / x.sum()
            choices.append(c)
            counts.append(cnt)
            ps.append(p)
    total = np.sum(counts, axis=0).astype(np.float64)
    if n == 0:
        return choices, counts, 0.0, [np.zeros_like(a) for a in z], [np.zeros_like(a) for a in z]
    f, mean_p = total / (k * n), np.sum([p.sum(axis=0) for p in ps], axis=0) / n
    loss = alpha * E * float((f * mean_p).sum())
    coef = alpha * E / (k * n * n)
    dz = [coef * p * (total - (p @ total)[:, None]) for p in ps]
    spread = np.abs(total - total.mean()).max() + 1e-3
    return choices, counts, loss, dz, [abs(coef) * p * spread for p in ps]
