"""fp64 definitions of the drafted-token operators: tree attention, verification, the move of accepted rows (numpy).

Written from the formulas of include/gqa.h, one (sequence, head, node) at a time; shares nothing with the GPU path.
"""

from __future__ import annotations

import math

import numpy as np


def parent(parents, b, i) -> int:
    """Parent of node i as the operators read it: one outside [-1, i) is -1."""
    a = int(parents[b if parents.shape[0] > 1 else 0, i])
    return a if -1 <= a < i else -1


def ancestors(parents, b, i) -> list[int]:
    """The node itself and its ancestors, from the node up."""
    out = []
    while i >= 0:
        out.append(i)
        i = parent(parents, b, i)
    return out


def forward(query, key, value, parents, seqlens_k, new_lens, present_key, present_value, num_heads, kv_num_heads,
            scale=0.0, softcap=0.0, window=-1, sink=None, smooth=False):
    """One step; the caches (B, N_kv, C, H) are updated in place. Returns output, and bounds for tolerances:
    sum_j p_j |v_j| (shaped as output) and the largest max_d |q_d| sum_d |k_jd| scale of every query row (B, S, N)."""
    B, S = query.shape[:2]
    H = query.shape[2] // num_heads
    G = num_heads // kv_num_heads
    scale = scale or 1.0 / math.sqrt(H)
    out, mag, reach = np.zeros((B, S, num_heads, H)), np.zeros((B, S, num_heads, H)), np.zeros((B, S, num_heads))
    for b in range(B):
        n = S if new_lens is None else int(new_lens[b])
        past = int(seqlens_k[b]) + 1 - n
        for g in range(kv_num_heads):
            for x, c in ((key, present_key), (value, present_value)):
                c[b, g, past:past + n] = x[b, :n].reshape(n, kv_num_heads, H)[:, g]
            k, v = (c[b, g, :past + n].astype(np.float64) for c in (present_key, present_value))
            size = np.abs(k).sum(-1)
            for i in range(n):
                up = ancestors(parents, b, i)
                first = max(0, past + len(up) - 1 - window) if window >= 0 else 0
                rows = list(range(first, past)) + [past + a for d, a in enumerate(up) if window < 0 or d <= window]
                for h in range(g * G, (g + 1) * G):
                    q = np.asarray(query[b, i], np.float64).reshape(num_heads, H)[h]
                    z = k[rows] @ q * scale
                    if softcap > 0:
                        z = softcap * np.tanh(z / softcap)
                    extra = [] if sink is None and not smooth else [0.0 if sink is None else float(sink[h])]
                    m = max([z.max(), *extra])
                    e = np.exp(z - m)
                    e = e / (e.sum() + sum(math.exp(x - m) for x in extra))
                    out[b, i, h], mag[b, i, h] = e @ v[rows], e @ np.abs(v[rows])
                    reach[b, i, h] = size[rows].max() * np.abs(q).max() * abs(scale)
    return out.reshape(B, S, -1), mag.reshape(B, S, -1), reach


def _proper(row):
    row = np.asarray(row, np.float64)
    return np.where((row > 0) & (row < 2.0 ** 40), row, 0.0)


def verify(tokens, parents, target_probs, accept_uniforms, sample_uniforms, draft_probs=None, new_lens=None):
    """Returns path (B, S), path_lens (B) and next_token (B)."""
    B, S, V = target_probs.shape
    path, lens, token = np.full((B, S), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        n = S if new_lens is None else int(new_lens[b])
        if not 0 < n <= S:
            continue
        at, nodes = 0, [0]
        while True:
            p = _proper(target_probs[b, at])
            q = None if draft_probs is None else _proper(draft_probs[b, at])
            left, z, found = p.copy(), 1.0, None
            for i in range(1, n):
                if parent(parents, b, i) != at:
                    continue
                x = int(tokens[b, i])
                inside = 0 <= x < V
                r, qx = (left[x], 1.0 if q is None else q[x]) if inside else (0.0, 1.0)
                if z > 0 and float(accept_uniforms[b, i]) * qx * z < r:
                    found = i
                    break
                if q is not None:
                    left = np.maximum(left / (z if z > 0 else 1.0) - q, 0.0)
                elif inside:
                    left[x] = 0.0
                z = math.fsum(left)
            if found is None:
                break
            at = found
            nodes.append(at)
        if not left.any():
            left = p
        path[b, :len(nodes)], lens[b] = nodes, len(nodes)
        if left.any():
            above = np.flatnonzero(np.cumsum(left) > float(sample_uniforms[b]) * math.fsum(left))
            token[b] = above[0] if len(above) else np.flatnonzero(left)[-1]
    return path, lens, token


def accept(caches, path, path_lens, seqlens_k, new_lens=None):
    """Moves the rows of every cache (B, N_kv, C, H) in place; returns the new seqlens_k."""
    B, S = path.shape
    out = np.full(B, -1, np.int32)
    for b in range(B):
        n = S if new_lens is None else int(new_lens[b])
        total, k, C = int(seqlens_k[b]) + 1, int(path_lens[b]), caches[0].shape[2]
        if not (0 <= n <= S and n <= total <= C and 0 <= k <= n):
            continue
        rows = [int(x) for x in path[b, :k]]
        if any(not 0 <= x < n for x in rows) or any(x >= y for x, y in zip(rows, rows[1:])):
            continue
        past = total - n
        for c in caches:
            c[b, :, past:past + k] = c[b][:, [past + x for x in rows]]
        out[b] = past + k - 1
    return out
