"""Oracle for the block-scaled FP8 cache: e4m3 codes with one float32 scale for
each block of 16 tokens and KV head, and of prompt attention.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A code c of block b and head h stands for ``e4m3(c) * scales[b, h]``.  The
append gives a block that receives rows the scale ``max(old, 2^e)``, 2^e the
least power of two (e >= -126) with ``max |new element| <= 448 * 2^e`` over the
finite elements; ``old`` counts only where rows of the sequence lie before the
new ones, which are moved to the new scale.
"""

from __future__ import annotations

import numpy as np

from .fp8_cache import E4M3_MAX, e4m3_bits_to_f64, f32_to_e4m3_bits
from .paged_attention import bf16_bits_to_f64

BLOCK = 16


def block_scale(x) -> float:
    """The scale that new elements ask for, by trial from the smallest."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    top = x.max() if x.size else 0.0
    e = -126
    while E4M3_MAX * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def append_block_scaled(k_bits, v_bits, q_start, tables, lens, k_codes, v_codes, k_scales,
                        v_scales):
    """New pools and scales (copies); rows and pools as bits, a call at a time."""
    out = []
    for rows, codes, scales in ((k_bits, k_codes, k_scales), (v_bits, v_codes, v_scales)):
        rows = bf16_bits_to_f64(rows)
        codes, scales = np.array(codes), np.array(scales, dtype=np.float32)
        for s, length in enumerate(lens):
            n = int(q_start[s + 1]) - int(q_start[s])
            for j in range(int(length - n) // BLOCK, -(-int(length) // BLOCK)):
                first = max(int(length) - n, j * BLOCK)
                last = min(int(length), (j + 1) * BLOCK)
                if first >= last:
                    continue
                b, a = int(tables[s][j]), first - j * BLOCK
                at = int(q_start[s]) + first - (int(length) - n)
                new = rows[at:at + last - first]
                for h in range(codes.shape[2]):
                    old = float(scales[b, h]) if a else 0.0
                    f = max(old, block_scale(new[:, h]))
                    if a and f != old:
                        codes[b, :a, h] = f32_to_e4m3_bits(
                            e4m3_bits_to_f64(codes[b, :a, h]) * (old / f))
                    codes[b, a:a + len(new), h] = f32_to_e4m3_bits(new[:, h] / f)
                    scales[b, h] = f
        out += [codes, scales]
    return out[0], out[2], out[1], out[3]


def dequantize_blocks(codes, scales) -> np.ndarray:
    """The float64 values that codes ``[NB, 16, Hkv, d]`` stand for."""
    return e4m3_bits_to_f64(codes) * np.asarray(scales, dtype=np.float64)[:, None, :, None]


def attend(q, k, v, scale, first):
    """Rows q ``[n, Hq, d]`` over k, v ``[L, Hkv, d]`` in float64; row i sees keys
    ``0 .. first + i`` (``first`` None: all).  Returns the result and
    sum_j w_j |v_j|, the size that rounding the weights is relative to."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    group = hq // hkv
    out, size = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        seen = L if first is None else min(L, first + i + 1)
        if seen <= 0:
            continue
        for h in range(hq):
            x = k[:seen, h // group] @ q[i, h] * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[i, h] = w @ v[:seen, h // group]
            size[i, h] = w @ np.abs(v[:seen, h // group])
    return out, size
