"""Float64 CPU restatement of the cache operators (test infrastructure only).

Everything is loops over (sequence, kv head) with NumPy; codes are E4M3 values as
floats, so nothing of the library's packing or tiling is repeated here.
"""
import math

import numpy as np

SCALE_FLOOR = 2.0 ** -100


def e4m3_round(x):
    """Nearest E4M3 value, ties to even, saturating at 448; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    ax = np.abs(np.where(np.isfinite(x), x, 0.0))
    e = np.maximum(np.floor(np.log2(np.where(ax > 0, ax, 1.0))), -6.0)
    step = np.exp2(e - 3)
    y = np.clip(np.rint(np.where(np.isfinite(x), x, 0.0) / step) * step, -448.0, 448.0)
    return np.where(np.isnan(x), np.nan, np.where(np.isinf(x), np.sign(x) * 448.0, y))


def scale_for(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s."""
    if not amax > 0:
        return SCALE_FLOOR
    e = math.ceil(math.log2(amax / 448.0))
    while amax > 448.0 * 2.0 ** e:
        e += 1
    while amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return max(2.0 ** e, SCALE_FLOOR)


def clamp_lens(lens, B, Nk):
    return [Nk] * B if lens is None else [min(max(int(n), 0), Nk) for n in lens]


def store64(x, codes, scales, block, lens):
    """x [B, H, n_new, d] appended to (codes, scales), which are copied; per tensor."""
    codes, scales = np.array(codes, np.float64), np.array(scales, np.float64)
    B, H, Nk, _ = codes.shape
    n_new = x.shape[2]
    for b, n in enumerate(clamp_lens(lens, B, Nk)):
        start = n - n_new
        for h in range(H):
            for j in range(scales.shape[2]):
                p0, p1 = j * block, min((j + 1) * block, n)
                first = max(p0, start, 0)
                if first >= p1:
                    continue
                fresh = np.asarray(x[b, h, first - start:p1 - start], np.float64)
                fin = np.abs(fresh[np.isfinite(fresh)])
                s = scale_for(float(fin.max()) if fin.size else 0.0)
                if p0 < start:
                    s = max(s, scales[b, h, j])
                    codes[b, h, p0:start] = e4m3_round(codes[b, h, p0:start] * (scales[b, h, j] / s))
                codes[b, h, first:p1] = e4m3_round(fresh / s)
                scales[b, h, j] = s
    return codes, scales


def dequantised(codes, scales, block):
    """Real values of a cache."""
    codes = np.asarray(codes, np.float64)
    if scales is None:
        return codes
    return codes * np.repeat(np.asarray(scales, np.float64), block, axis=2)[:, :, :codes.shape[2], None]


def bounds64(k, block, lens):
    """[B, H, n_blocks, 2, d] minima and maxima (NaN skipped); zeros where a block holds nothing."""
    B, H, Nk, d = k.shape
    nb = -(-Nk // block)
    out = np.zeros((B, H, nb, 2, d))
    for b, n in enumerate(clamp_lens(lens, B, Nk)):
        for j in range(nb):
            held = np.asarray(k[b, :, j * block:min((j + 1) * block, n)], np.float64)
            if held.shape[1]:
                out[b, :, j, 0], out[b, :, j, 1] = np.nanmin(held, 1), np.nanmax(held, 1)
    return out


def last_seen(n, Nq, i, causal):
    return n - Nq + i if causal else n - 1


def select64(q, bounds, scales, n_select, block, Nk, lens, n_first, n_last, causal=True):
    """The selection by brute force: sorted by (not forced, -score, index)."""
    q, bounds = np.asarray(q, np.float64), np.asarray(bounds, np.float64)
    B, Hq, Nq, _ = q.shape
    H = bounds.shape[1]
    g = Hq // H
    idx = np.full((B, H, Nq, n_select), -1, np.int64)
    for b, n in enumerate(clamp_lens(lens, B, Nk)):
        for h in range(H):
            for i in range(Nq):
                last = last_seen(n, Nq, i, causal)
                count = last // block + 1 if last >= 0 else 0
                u = np.full(count, -np.inf)
                for r in range(g):
                    x = q[b, h * g + r, i]
                    with np.errstate(invalid="ignore"):
                        v = np.where(x >= 0, x * bounds[b, h, :count, 1], x * bounds[b, h, :count, 0]).sum(-1)
                    if scales is not None:
                        v = v * np.asarray(scales[b, h, :count], np.float64)
                    u = np.fmax(u, v)
                order = sorted(range(count), key=lambda j: (not (j < n_first or j >= count - n_last), -u[j], j))
                top = sorted(order[:n_select])
                idx[b, h, i, :len(top)] = top
    return idx


def attend64(q, k, v, scale, causal, lens, idx=None, block=0):
    """O, LSE, and per output sum_j p_j |v_j| and max_j sum_c |q_c k_jc| scale, from which
    the tests derive their tolerances. k, v are real values; idx restricts a query's keys."""
    q = np.asarray(q, np.float64)
    B, Hq, Nq, d = q.shape
    H, Nk = k.shape[1], k.shape[2]
    g, nb = Hq // H, -(-Nk // block) if block else 0
    o, lse = np.zeros((B, Hq, Nq, d)), np.full((B, Hq, Nq), -np.inf)
    pv, size = np.zeros((B, Hq, Nq, d)), np.zeros((B, Hq, Nq))
    for b, n in enumerate(clamp_lens(lens, B, Nk)):
        for hq in range(Hq):
            h = hq // g
            for i in range(Nq):
                last = last_seen(n, Nq, i, causal)
                keys = np.arange(max(last + 1, 0))
                if idx is not None:
                    at = [int(j) for j in idx[b, h, i] if 0 <= j < nb]
                    keys = np.concatenate([np.arange(j * block, (j + 1) * block) for j in at] + [np.zeros(0, np.int64)])
                    keys = keys[keys <= last].astype(np.int64)
                if not keys.size:
                    continue
                kk, vv = k[b, h, keys], v[b, h, keys]
                s = scale * (kk @ q[b, hq, i])
                m = s.max()
                e = np.exp(s - m)
                l = e.sum()
                o[b, hq, i] = (e / l) @ vv
                lse[b, hq, i] = m + math.log(l)
                pv[b, hq, i] = (e / l) @ np.abs(vv)
                size[b, hq, i] = scale * (np.abs(kk) @ np.abs(q[b, hq, i])).max()
    return o, lse, pv, size


def weights64(q, k, lse, scale, causal, lens):
    """The sums that cache_weights adds, [B, H, Nk], and for each key the largest
    sum_c |q_c k_c| scale of a row that sees it."""
    q = np.asarray(q, np.float64)
    B, Hq, Nq, d = q.shape
    H, Nk = k.shape[1], k.shape[2]
    g = Hq // H
    add, size = np.zeros((B, H, Nk)), np.zeros((B, H, Nk))
    for b, n in enumerate(clamp_lens(lens, B, Nk)):
        for hq in range(Hq):
            for i in range(Nq):
                last = last_seen(n, Nq, i, causal)
                if last < 0 or lse[b, hq, i] == -np.inf:
                    continue
                kk = k[b, hq // g, :last + 1]
                add[b, hq // g, :last + 1] += np.exp(scale * (kk @ q[b, hq, i]) - float(lse[b, hq, i]))
                size[b, hq // g, :last + 1] = np.maximum(size[b, hq // g, :last + 1],
                                                         scale * (np.abs(kk) @ np.abs(q[b, hq, i])))
    return add, size


def evict64(acc, keep, recent, lens):
    """Kept positions [B, H, keep] (-1 behind them) and the new lengths."""
    B, H, Nk = acc.shape
    idx, out = np.full((B, H, keep), -1, np.int64), []
    for b, n in enumerate(clamp_lens(lens, B, Nk)):
        m = min(n, keep)
        r = min(recent, m)
        for h in range(H):
            a = [float(x) for x in acc[b, h, :n - r]]
            order = sorted(range(n - r), key=lambda j: (math.isnan(a[j]), 0.0 if math.isnan(a[j]) else -a[j], j))
            idx[b, h, :m] = sorted(order[:m - r]) + list(range(n - r, n))
        out.append(m)
    return idx, out
