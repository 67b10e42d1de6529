"""The 8-bit products with block scales and the layer of experts around them, in binary64 with
numpy, from their definitions; test infrastructure only."""
import numpy as np

from oracle.fp8_paged import e4m3_decode


def spread(scales, width, axis=-1):
    """Scales of blocks of 128 for every element; a single column stands for all."""
    s = np.asarray(scales, np.float64)
    if axis == -1 and s.shape[-1] == 1:
        return np.broadcast_to(s, (*s.shape[:-1], width))
    return np.take(np.repeat(s, 128, axis), np.arange(width), axis)


def values(codes, scales, rows_in_blocks):
    s = spread(scales, codes.shape[-2], -2) if rows_in_blocks else scales
    return e4m3_decode(codes) * spread(s, codes.shape[-1])


def matmul(a, a_scales, b, b_scales):
    """(a @ b.T, the same of magnitudes)."""
    x, w = values(a, a_scales, False), values(b, b_scales, True)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def by_expert(a, a_scales, b, b_scales, offsets, rows, num_rows):
    """As matmul, with NaN where no expert has the row."""
    n = b.shape[1]
    y, mass = (np.full((num_rows, n), np.nan) for _ in range(2))
    off = np.clip(np.asarray(offsets), 0, num_rows)
    for e in range(b.shape[0]):
        for i in range(off[e], off[e + 1]):
            r = i if rows is None else int(rows[i])
            if 0 <= r < a.shape[0]:
                y[i:i + 1], mass[i:i + 1] = matmul(a[r:r + 1], a_scales[r:r + 1], b[e], b_scales[e])
            else:
                y[i], mass[i] = 0, 0
    return y, mass


def gated(y, mass):
    """(z, scales, bound on |z|'s error for an error of 1 mass in y)."""
    n = y.shape[1] // 2
    g, u, mg, mu = y[:, :n], y[:, n:], mass[:, :n], mass[:, n:]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    z = silu * u
    per = 1.1 * mg * np.abs(u) + np.abs(silu) * mu
    scales = np.maximum(np.abs(z).reshape(len(z), -1, 128).max(2), 1e-4) / 448
    return z, scales, per


def route(logits, top_k, score, bias, groups, top_groups, renormalize, scale):
    x = np.minimum(np.where(np.isnan(logits), -np.inf, logits).astype(np.float64),
                   np.finfo(np.float32).max)
    tokens, experts = x.shape
    chosen, weights = np.zeros((tokens, top_k), np.int64), np.zeros((tokens, top_k))
    for t in range(tokens):
        row = x[t]
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-row))
            elif row.max() == -np.inf:
                s = np.zeros(experts)
            else:
                s = np.exp(row - row.max())
                s /= s.sum()
        biased = s + (0 if bias is None else np.asarray(bias, np.float64))
        key = row if bias is None else biased
        taken = range(groups)
        if groups > 1:
            v = [sum(sorted(biased.reshape(groups, -1)[g])[-2:]) for g in range(groups)]
            taken = sorted(range(groups), key=lambda g: (-v[g], g))[:top_groups]
        within = [e for e in range(experts) if e // (experts // groups) in taken]
        pick = sorted(within, key=lambda e: (-key[e], e))[:top_k]
        w = s[pick]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        chosen[t], weights[t] = pick, w * scale
    return chosen, weights


def sort_by_expert(chosen, experts):
    """Offsets, rows, places by walking the pairs expert by expert."""
    tokens, top_k = chosen.shape
    offsets, rows, places = [0], [], np.full((tokens, top_k), -1, np.int64)
    flat = chosen.reshape(-1)
    for e in range(experts):
        for i in np.nonzero(flat == e)[0]:
            places.reshape(-1)[i] = len(rows)
            rows.append(i // top_k)
        offsets.append(len(rows))
    rows += [-1] * (tokens * top_k - len(rows))
    return np.array(offsets, np.int64), np.array(rows, np.int64).reshape(-1), places


def combine(y, places, weights, base):
    out = np.zeros((places.shape[0], y.shape[1])) if base is None else base.astype(np.float64).copy()
    mass = np.abs(out)
    for t in range(places.shape[0]):
        for p, w in zip(places[t], weights[t]):
            if 0 <= p < y.shape[0]:
                out[t] += np.float64(w) * y[p]
                mass[t] += np.abs(np.float64(w) * y[p])
    return out, mass
