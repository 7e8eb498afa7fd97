"""fp64 definitions of the multi-axis rotary, the block-scaled int8 cache and its eviction (numpy).

Written from the formulas of include/gqa.h, one (sequence, KV head) at a time; shares nothing with the GPU path.
"""

from __future__ import annotations

import math

import numpy as np

F32 = np.float32


def axis_of_pair(sections, interleaved: bool) -> list[int]:
    """Axis of every rotated pair."""
    pairs, axes = sum(sections), len(sections)
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    out = []
    for d in range(pairs):
        r = d % axes
        out.append(r if r > 0 and d < axes * sections[r] else 0)
    return out


def rotary_axes(x, heads, positions, cos, sin, sections, interleaved=False, weight=None, eps=1e-6):
    """x (B, S, heads*H) rotated in fp64; cos / sin (R, pairs) as stored."""
    B, S = x.shape[:2]
    y = np.asarray(x, np.float64).reshape(B, S, heads, -1).copy()
    H = y.shape[-1]
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    pairs = sum(sections)
    out = y.copy()
    for d, a in enumerate(axis_of_pair(sections, interleaved)):
        c = np.asarray(cos, np.float64)[positions[a], d][:, :, None]
        s = np.asarray(sin, np.float64)[positions[a], d][:, :, None]
        out[..., d] = y[..., d] * c - y[..., d + pairs] * s
        out[..., d + pairs] = y[..., d + pairs] * c + y[..., d] * s
    return out.reshape(B, S, heads * H)


def nearest_code(x, scale):
    """Integer nearest to x / scale, ties to even, within +-127. The 64-bit quotient of two 24-bit (or a 31- and a
    24-bit) numbers lies on the right side of every border."""
    if not scale > 0:
        return np.zeros(x.shape, np.int8)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.rint(np.asarray(x, np.float64) / np.float64(scale))
    q = np.where(np.isnan(q), 0.0, np.clip(q, -127, 127))
    return q.astype(np.int8)


def append(codes, scales, rows, past, block_size):
    """Store rows (n, H) of one head behind `past` rows: codes (C, H) and scales (blocks) in place."""
    n = rows.shape[0]
    for blk in range(past // block_size, (past + n - 1) // block_size + 1 if n else 0):
        a, z = blk * block_size, (blk + 1) * block_size
        lo, hi = max(a, past), min(z, past + n)
        x = np.asarray(rows[lo - past:hi - past], F32)
        mag = np.abs(x[np.isfinite(x)])
        s = F32(F32(mag.max() if mag.size else 0.0) * F32(1.0 / F32(127.0)))
        if past > a:
            s0 = scales[blk]
            if s > s0:
                codes[a:past] = nearest_code(codes[a:past].astype(np.float64) * np.float64(s0), s)
            else:
                s = s0
        scales[blk] = s
        codes[lo:hi] = nearest_code(x, s)


def values(codes, scales, rows, block_size):
    """Rows [0, rows) of one head in fp64."""
    return codes[:rows].astype(np.float64) * scales[np.arange(rows) // block_size].astype(np.float64)[:, None]


def step(query, key, value, seqlens_k, new_lens, cache, block_size, num_heads, kv_num_heads, scale=0.0, softcap=0.0,
         window=-1, sink=None, smooth=False, past_weights=None, weights=None):
    """One step; cache = (key_codes, value_codes, key_scales, value_scales) is updated in place, and `weights`
    (B, N_kv, C fp64) if given. Returns output, and bounds for tolerances: sum_j p_j |v_j| (shaped as
    output) and the largest max_d |q_d| sum_d |k_jd| scale of every query row (B, S, N)."""
    B, S = query.shape[:2]
    H = query.shape[2] // num_heads
    G = num_heads // kv_num_heads
    kc, vc, ks, vs = cache
    scale = scale or 1.0 / math.sqrt(H)
    out = np.zeros((B, S, num_heads, H))
    mag = np.zeros((B, S, num_heads, H))
    reach = np.zeros((B, S, num_heads))
    for b in range(B):
        total = int(seqlens_k[b]) + 1
        new = S if new_lens is None else int(new_lens[b])
        past = total - new
        for g in range(kv_num_heads):
            if key is not None:
                for x, c, s in ((key, kc, ks), (value, vc, vs)):
                    rows = np.asarray(x[b, :new], F32).reshape(new, kv_num_heads, H)[:, g]
                    append(c[b, g], s[b, g], rows, past, block_size)
            k, v = values(kc[b, g], ks[b, g], total, block_size), values(vc[b, g], vs[b, g], total, block_size)
            av, size = np.abs(v), np.abs(k).sum(-1)
            got = np.zeros(total)
            for i in range(new):
                p = past + i
                lo = 0 if window < 0 else max(0, p - window)
                for h in range(g * G, (g + 1) * G):
                    q = np.asarray(query[b, i], np.float64).reshape(num_heads, H)[h]
                    z = k[lo:p + 1] @ q * scale
                    if softcap > 0:
                        z = softcap * np.tanh(z / softcap)
                    extra = [] if sink is None and not smooth else [0.0 if sink is None else float(sink[h])]
                    m = max([z.max(), *extra])
                    e = np.exp(z - m)
                    e = e / (e.sum() + sum(math.exp(x - m) for x in extra))
                    out[b, i, h] = e @ v[lo:p + 1]
                    mag[b, i, h] = e @ av[lo:p + 1]
                    reach[b, i, h] = size[lo:p + 1].max() * np.abs(q).max() * scale
                    got[lo:p + 1] += e
            if weights is not None:
                had = 0.0 if past_weights is None else np.where(np.arange(total) < past, past_weights[b, g, :total], 0.0)
                weights[b, g, :total] = had + got
    return out.reshape(B, S, -1), mag.reshape(B, S, -1), reach


def kept_rows(weights, total, keep, recent, first):
    """Rows of one head that stay: first, recent and the largest weights between (lower row first on a tie)."""
    if total <= keep:
        return np.arange(total)
    mid = np.arange(first, total - recent)
    w = np.asarray(weights, np.float64)[mid]
    w = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(np.asarray(weights, np.float64)[mid])
    best = sorted(range(len(mid)), key=lambda i: (nan[i], -w[i], mid[i]))[:keep - first - recent]
    return np.concatenate([np.arange(first), np.sort(mid[np.array(best, int)]), np.arange(total - recent, total)])


def evict(cache, weights, seqlens_k, keep, recent, first, block_size, into, into_weights=None):
    """Copy the kept rows of every (sequence, head) to `into` (in place). Returns kept (B, N_kv, keep), seqlens."""
    B, Nkv = weights.shape[:2]
    kept = np.full((B, Nkv, keep), -1, np.int32)
    lens = np.zeros(B, np.int32)
    for b in range(B):
        total = int(seqlens_k[b]) + 1
        lens[b] = min(total, keep) - 1
        for g in range(Nkv):
            rows = kept_rows(weights[b, g], total, keep, recent, first)
            kept[b, g, :len(rows)] = rows
            if into_weights is not None:
                into_weights[b, g, :len(rows)] = weights[b, g, rows]
            for c, s, tc, ts in ((cache[0], cache[2], into[0], into[2]), (cache[1], cache[3], into[1], into[3])):
                for a in range(0, len(rows), block_size):
                    src = rows[a:a + block_size]
                    sc = s[b, g, src // block_size]
                    top = sc.max()
                    ts[b, g, a // block_size] = top
                    for j, r in enumerate(src):
                        x = c[b, g, r].astype(np.float64) * np.float64(sc[j])
                        tc[b, g, a + j] = c[b, g, r] if sc[j] == top else nearest_code(x, top)
    return kept, lens
