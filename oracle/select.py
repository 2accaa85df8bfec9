"""Block summaries, block scores and block selection, float64 (oracle; test infrastructure).

A summary is the mean of a block's keys, each rotated by its slot; its product with the query rotated by (query
position - block start) is the mean of the block's scores (the score equation of the MiniPIC summary, gist.science
2606.13126, section 2.1, summed over the block).  Plain loops.
"""

from __future__ import annotations

import math

import numpy as np

from .rope import rope_rotate


def block_means(k, means, cu, start, tables, base, bs=16):
    """``means`` [num_blocks, Hkv, d] after summarising the blocks that an append of cu[r+1] - cu[r] keys from key
    start[r] on wrote into; k float64 values [num_blocks, Hkv, bs, d]."""
    means = np.array(means, dtype=np.float64)
    for r in range(len(cu) - 1):
        end = int(start[r]) + int(cu[r + 1]) - int(cu[r])
        if end == int(start[r]):
            continue
        for b in range(int(start[r]) // bs, -(-end // bs)):
            p, n = int(tables[r][b]), min(bs, end - b * bs)
            means[p] = rope_rotate(k[p][:, :n], np.arange(n), base).mean(1)
    return means


def block_scores(q, means, tables, starts, lens, q_pos, base, scale=0.0, max_pos=1 << 30, bs=16):
    """(scores [B, Hkv, mb], size of the vectors' product |q| |m| scale of the same shape)."""
    q, means = np.asarray(q, dtype=np.float64), np.asarray(means, dtype=np.float64)
    B, Hq, d = q.shape
    num, Hkv = means.shape[:2]
    mb = np.asarray(tables).shape[1]
    sc = scale if scale > 0 else 1.0 / math.sqrt(d)
    out = np.full((B, Hkv, mb), -np.inf)
    size = np.zeros((B, Hkv, mb))
    for r in range(B):
        qr = rope_rotate(q[r], np.full(Hq, int(q_pos[r])), base).reshape(Hkv, Hq // Hkv, d)
        for b in range(-(-int(lens[r]) // bs)):
            p, st = int(tables[r][b]), int(starts[r][b])
            if not (0 <= p < num and 0 <= st < max_pos):
                continue
            m = rope_rotate(means[p], np.full(Hkv, st), base)
            for g in range(Hkv):
                s = qr[g] @ m[g] * sc
                out[r, g, b] = np.nan if np.isnan(s).any() else s.max()
                size[r, g, b] = np.linalg.norm(qr[g], axis=1).max() * np.linalg.norm(m[g]) * sc
    return out, size


def block_select(scores, lens, budget, first=1, last=1, bs=16):
    """selected [B, Hkv, budget] int32."""
    scores = np.asarray(scores)
    B, Hkv, _ = scores.shape
    out = np.full((B, Hkv, budget), -1, np.int32)
    for r in range(B):
        n = -(-int(lens[r]) // bs)
        for g in range(Hkv):
            s = scores[r, g, :n]
            keep = list(range(n))
            if n > budget:
                always = [b for b in range(n) if b < first or b >= n - last]
                held = set(always)
                others = sorted((b for b in range(n) if b not in held),
                                key=lambda b: (np.isnan(s[b]), -s[b] if not np.isnan(s[b]) else 0.0, b))
                keep = sorted(always + others[:budget - len(always)])
            out[r, g, :len(keep)] = keep
    return out
