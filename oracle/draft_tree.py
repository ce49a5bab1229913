"""Oracle for the speculative step with trees of drafted tokens (numpy, float64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages name speculative decoding ("Cache KV, attention et optimisation de
l'inference", section "Decodage speculatif": guess several next tokens, check
them in one pass) without a tree.  Readings taken: a tree's nodes are the last
positions of the context in the order they were drafted; a node attends the
committed positions, its ancestors and itself; its position (for the rotation)
is the committed length plus its depth.
"""

from __future__ import annotations

import numpy as np

from .paged_attention import _as_f64, gather_sequence_kv


def rope_table(positions: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """[positions, rot] float32: cos then sin of position * base^(-2 i / rot),
    the angles in float64."""
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    angle = np.arange(positions, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def norm_rope(x, weight, positions, table, eps, interleaved) -> np.ndarray:
    """``x [T, H, d]``: RMS norm per head (``weight`` None: none), then each
    pair of the first rot elements turned by its token's angle."""
    x = _as_f64(x).copy()
    if weight is not None:
        x /= np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
        x *= _as_f64(weight)
    rot = table.shape[1]
    out = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = table[positions, i].astype(np.float64)[:, None]
        s = table[positions, rot // 2 + i].astype(np.float64)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def tree_layout(parents, q_start, context_lens):
    """(masks uint64, positions int64) of every node, walking up from each."""
    masks = np.zeros(len(parents), dtype=np.uint64)
    positions = np.zeros(len(parents), dtype=np.int64)
    for s in range(len(context_lens)):
        lo, hi = int(q_start[s]), int(q_start[s + 1])
        for t in range(hi - lo):
            word, depth, u = 0, -1, t
            while u >= 0:
                word |= 1 << u
                depth += 1
                u = int(parents[lo + u])
            masks[lo + t] = word
            positions[lo + t] = int(context_lens[s]) - (hi - lo) + depth
    return masks, positions


def tree_attention(q, q_start, masks, k_cache, v_cache, block_tables, context_lens, scale):
    """``q [total, Hq, d]``: softmax(q K^T * scale) V over each row's visible
    keys only (hidden keys are left out, not weighted by zero); a row without
    any is zero.  ``scale`` is taken as the float32 the kernels receive."""
    q = _as_f64(q)
    out = np.zeros(q.shape)
    scale = float(np.float32(scale))
    for s in range(len(context_lens)):
        lo, n, L = int(q_start[s]), int(q_start[s + 1]) - int(q_start[s]), int(context_lens[s])
        if n == 0:
            continue
        k = _as_f64(gather_sequence_kv(k_cache, block_tables[s], L))
        v = _as_f64(gather_sequence_kv(v_cache, block_tables[s], L))
        group = q.shape[1] // k.shape[1]
        for t in range(n):
            word = int(masks[lo + t])
            keys = list(range(L - n)) + [L - n + u for u in range(n) if word >> u & 1]
            if not keys:
                continue
            for h in range(k.shape[1]):
                rows = slice(h * group, (h + 1) * group)
                x = q[lo + t, rows] @ k[keys, h].T * scale
                p = np.exp(x - x.max(-1, keepdims=True))
                out[lo + t, rows] = (p / p.sum(-1, keepdims=True)) @ v[keys, h]
    return out


def accept_rows(pool, block_tables, context_lens, q_start, accepted, num_accepted):
    """(a copy of ``pool [layers, NB, bs, ...]`` with the accepted rows moved
    up, the new context lengths)."""
    out, bs = pool.copy(), pool.shape[2]
    lens = np.array(context_lens, dtype=np.int64)
    for s in range(len(lens)):
        base = int(context_lens[s]) - (int(q_start[s + 1]) - int(q_start[s]))
        for i in range(int(num_accepted[s])):
            a, b = base + i, base + int(accepted[s][i])
            out[:, block_tables[s][a // bs], a % bs] = pool[:, block_tables[s][b // bs], b % bs]
        lens[s] = base + int(num_accepted[s])
    return out, lens
