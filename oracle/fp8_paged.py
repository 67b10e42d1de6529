"""Plain definitions of the operators on the paged E4M3 cache with grouped
heads, in numpy: the append in binary32 (its codes are defined bit for bit),
attention and the norm in binary64."""
import math

import numpy as np

_E4M3 = None


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    """E4M3 codes as float64 (0x7F / 0xFF are NaN)."""
    global _E4M3
    if _E4M3 is None:
        c = np.arange(256)
        e, m = (c >> 3) & 15, c & 7
        v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
        v = np.where(c & 128, -v, v)
        v[[0x7F, 0xFF]] = np.nan
        _E4M3 = v
    return _E4M3[codes]


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code, ties to the even one, saturating; NaN -> 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    r = np.rint(a / step) * step                    # numpy rounds ties to even
    _, e = np.frexp(r)
    normal = ((e + 6) << 3) | (np.rint(np.ldexp(r, 4 - e)).astype(np.int64) - 8)
    codes = np.where(r < 2.0 ** -6, np.rint(r * 512).astype(np.int64), normal)
    codes = codes | (np.signbit(x).astype(np.int64) << 7)
    return np.where(np.isnan(x), 0x7F, codes).astype(np.uint8)


def ceil_log2_f32(v) -> int:
    """Smallest e with 2**e >= v for a positive binary32 v."""
    m, e = math.frexp(float(v))
    return e - 1 if m == 0.5 else e


def rotate(x, cos_sin_row, rotary_dim, interleaved):
    """One token's heads [heads, dim] (float32), every product and sum rounded."""
    x = x.copy()
    half = rotary_dim // 2
    c, s = cos_sin_row[:half], cos_sin_row[half:rotary_dim]
    i, j = (slice(0, rotary_dim, 2), slice(1, rotary_dim, 2)) if interleaved else \
        (slice(0, half), slice(half, rotary_dim))
    a, b = x[:, i].copy(), x[:, j].copy()
    x[:, i] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    x[:, j] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return x


def append(k, v, caches, scales, table, ctx_lens, starts, cos_sin, rotary_dim, interleaved,
           positions=None, q=None):
    """k, v [tokens, heads, dim] and q float32; caches: two uint8 [pages, heads,
    slots, dim], scales: two uint8 [pages, heads], both updated in place.
    Returns (rotated queries float32, bool [tokens]: which rows are written);
    rows that are skipped are as they were."""
    pages, heads, page, dim = caches[0].shape
    q_out = None if q is None else q.copy()
    written = np.zeros(k.shape[0], bool)
    capacity = table.shape[1] * page
    for b in range(len(ctx_lens)):
        n = int(starts[b + 1] - starts[b])
        c = min(max(int(ctx_lens[b]), 0), capacity)
        by_page = {}
        for i in range(n):
            t, p = int(starts[b]) + i, c + i
            written[t] = True
            if rotary_dim:
                r = int(positions[t]) if positions is not None else p
                if not 0 <= r < cos_sin.shape[0]:
                    written[t] = False
                    continue
                if q is not None:
                    q_out[t] = rotate(q[t], cos_sin[r], rotary_dim, interleaved)
                kt = rotate(k[t], cos_sin[r], rotary_dim, interleaved)
            else:
                kt = k[t]
            if p >= capacity or not 0 <= table[b, p // page] < pages:
                continue
            by_page.setdefault(p // page, []).append((p % page, kt, v[t]))
        for column, rows in by_page.items():
            g = table[b, column]
            kept = max(0, c - column * page)
            for which in (0, 1):
                for h in range(heads):
                    vals = np.stack([r[1 + which][h] for r in rows])
                    amax = np.float32(np.nanmax(np.append(np.abs(vals).ravel(), np.float32(1e-4))))
                    with np.errstate(over="ignore"):
                        scaled = np.float32(amax * np.float32(1 / np.float32(448)))
                    e = 120 if np.isinf(scaled) else min(ceil_log2_f32(scaled), 120)
                    if kept:
                        old = int(scales[which][g, h]) - 127
                        if old >= e:
                            e = old
                        else:
                            was = e4m3_decode(caches[which][g, h, :kept])
                            caches[which][g, h, :kept] = e4m3_encode(was * 2.0 ** (old - e))
                    scales[which][g, h] = e + 127
                    for (slot, *_), x in zip(rows, vals):
                        caches[which][g, h, slot] = e4m3_encode(x.astype(np.float64) * 2.0 ** -e)
    return q_out, written


def attention(q, caches, scales, table, seq_lens, starts, sm_scale, causal=True, window=0):
    """float64 (out, lse, mass, spread): mass = sum_j softmax_j |v_j|; spread
    [tokens, heads] = the largest sm_scale * sum_d |q_d k_jd| over visible keys
    (what rounding of the scores scales with); rows past the sequences NaN."""
    pages, heads, page, dim = caches[0].shape
    group = q.shape[1] // heads
    q = q.astype(np.float64)
    out = np.full(q.shape, np.nan)
    mass = np.zeros(q.shape)
    lse = np.full(q.shape[:2], np.nan)
    spread = np.zeros(q.shape[:2])
    capacity = table.shape[1] * page
    for b in range(len(seq_lens)):
        first, n = int(starts[b]), int(starts[b + 1] - starts[b])
        total = min(max(int(seq_lens[b]), 0), capacity)
        tokens = np.arange(total)
        g = table[b, tokens // page]
        ok = (g >= 0) & (g < pages)
        gc = np.where(ok, g, 0)
        for h in range(heads):
            def values(which):
                sc = scales[which][gc, h].astype(np.int64)
                two = np.where(sc == 255, np.nan, np.exp2(sc - 127.0))
                return e4m3_decode(caches[which][gc, h, tokens % page]) * two[:, None]
            k, v = values(0), values(1)
            for i in range(n):
                p = total - n + i
                see = ok.copy()
                if causal:
                    see &= tokens <= p
                if window:
                    see &= tokens > p - window
                hs = slice(h * group, (h + 1) * group)
                if not see.any():
                    out[first + i, hs], lse[first + i, hs] = 0, -np.inf
                    continue
                qi = q[first + i, hs]
                x = qi @ k[see].T * sm_scale
                spread[first + i, hs] = (np.abs(qi) @ np.abs(k[see]).T * sm_scale).max(1)
                m = x.max(1, keepdims=True)
                e = np.exp(x - m)
                s = e.sum(1, keepdims=True)
                out[first + i, hs] = e @ v[see] / s
                mass[first + i, hs] = e @ np.abs(v[see]) / s
                lse[first + i, hs] = (m + np.log(s))[:, 0]
    return out, lse, mass, spread


def add_rmsnorm(x, residual, weight, eps, group):
    """float64 (y, scales, h): y the normalised values, scales per group."""
    h = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight.astype(np.float64)
    g = group or y.shape[1]
    amax = np.abs(y.reshape(y.shape[0], -1, g)).max(2)
    return y, np.maximum(amax, 1e-4) / 448.0, h
