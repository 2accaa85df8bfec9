"""8-bit cache, block weights and eviction, float64 (oracle; test infrastructure).

Storage: OCP e4m3 (1 sign, 4 exponent bits of bias 7, 3 mantissa bits; no
infinities; 0x7f and 0xff are NaN), one scale per (block, kv head) and pool.
Attention: the score equation of the MiniPIC summary (gist.science 2606.13126,
section 2.1) over the values that the bytes stand for.  Plain loops, nothing
blocked or fused.
"""

from __future__ import annotations

import math

import numpy as np

from .attention import attend, key_index_map
from .rope import rope_rotate

MIN_EXP = -100
MAX = 448.0


def _value(b: int) -> float:
    sign = -1.0 if b & 0x80 else 1.0
    e, m = (b >> 3) & 15, b & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))


VALUES = np.array([_value(b) for b in range(256)])
_POS = VALUES[:127]  # 0 .. 448 ascending


def decode_bytes(b: np.ndarray) -> np.ndarray:
    return VALUES[np.asarray(b, dtype=np.uint8)]


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte, ties to the even byte; beyond 448 (infinity too) saturates."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), MAX)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    b = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    b = np.where(_POS[hi] == a, hi, b)
    b = b | np.where(np.signbit(x), 0x80, 0)
    return np.where(nan, 0x7f | np.where(np.signbit(x), 0x80, 0), b).astype(np.uint8)


def scale_for(x: np.ndarray) -> float:
    """2^k, the least k >= -100 with max|x| <= 448 * 2^k over the finite values."""
    f = np.abs(np.asarray(x, dtype=np.float64))
    f = f[np.isfinite(f)]
    amax = float(f.max()) if f.size else 0.0
    k = MIN_EXP
    while MAX * 2.0 ** k < amax:
        k += 1
    return 2.0 ** k


def append(pool, scale, new, cu, start, tables):
    """(pool bytes, scales) after the quantising append of ``new`` [total, Hkv, d]."""
    pool, scale = np.array(pool), np.array(scale, dtype=np.float64)
    bs = pool.shape[2]
    for r in range(len(cu) - 1):
        i, n = 0, int(cu[r + 1]) - int(cu[r])
        while i < n:
            j = int(start[r]) + i
            b, s0 = int(tables[r][j // bs]), j % bs
            m = min(n - i, bs - s0)
            for h in range(pool.shape[1]):
                rows = np.asarray(new[int(cu[r]) + i:int(cu[r]) + i + m, h], dtype=np.float64)
                s = scale_for(rows)
                if s0:
                    s = max(float(scale[b, h]), s)
                    if s > scale[b, h]:
                        pool[b, h, :s0] = encode(decode_bytes(pool[b, h, :s0]) * (scale[b, h] / s))
                pool[b, h, s0:s0 + m] = encode(rows / s)
                scale[b, h] = s
            i += m
    return pool, scale


def values(pool, scale):
    """float64 values of a quantised pool."""
    return decode_bytes(pool) * np.asarray(scale, dtype=np.float64)[..., None, None]


def _request(k, v, tables, starts, n, base, num_blocks, max_pos, bs=16):
    """Rotated keys, values [Hkv, n, d] and which of the n keys are usable."""
    phys, slot, pos = key_index_map(tables, starts, n, bs)
    ok = (phys >= 0) & (phys < num_blocks) & (pos >= 0) & (pos < max_pos)
    kk = np.where(ok[:, None, None], k[np.clip(phys, 0, num_blocks - 1), :, slot], 0.0)
    vv = np.where(ok[:, None, None], v[np.clip(phys, 0, num_blocks - 1), :, slot], 0.0)
    kr = rope_rotate(kk.transpose(1, 0, 2), np.where(ok, pos, 0), base)
    return kr, vv.transpose(1, 0, 2), ok


def attention(q, cu, q_pos, k, v, tables, starts, lens, base, scale=0.0, causal=False, max_pos=1 << 30):
    """q [total, Hq, d], k / v float64 values of the pools.  ``causal``: the
    rows of request r are its last keys' queries; else one row per request that
    sees every key.  Returns a dict with out, lse, block weights [B, Hkv, mb]
    (non-causal), and what error bounds need: spread = sum_j p_j |v_j - out|,
    mass = sum_j p_j |v_j|, smax = max_j |q| |k_j| scale per (row, head)."""
    q = np.asarray(q, dtype=np.float64)
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    G, mb = Hq // Hkv, np.asarray(tables).shape[1]
    sc = scale if scale > 0 else 1.0 / math.sqrt(d)
    res = {"out": np.zeros((total, Hq, d)), "lse": np.full((total, Hq), -np.inf),
           "weights": np.zeros((len(lens), Hkv, mb)), "spread": np.zeros((total, Hq, d)),
           "mass": np.zeros((total, Hq, d)), "smax": np.zeros((total, Hq))}
    for r in range(len(lens)):
        q0, q1 = int(cu[r]), int(cu[r + 1])
        n = int(lens[r])
        if q1 == q0 or n == 0:
            continue
        kr, vr, ok = _request(k, v, tables[r], starts[r], n, base, k.shape[0], max_pos)
        qr = rope_rotate(q[q0:q1].transpose(1, 0, 2), np.asarray(q_pos[q0:q1], dtype=np.int64), base)
        qr = qr.transpose(1, 0, 2)
        seen = np.broadcast_to(ok, (q1 - q0, n))
        if causal:
            i = np.arange(q1 - q0)[:, None]
            seen = seen & (np.arange(n) <= n - (q1 - q0) + i)
        for h in range(Hq):
            g = h // G
            o, lse = attend(qr[:, h], kr[g], vr[g], sc, seen)
            s = np.where(seen, (qr[:, h] @ kr[g].T) * sc, -np.inf)
            p = np.exp(s - np.where(np.isfinite(lse), lse, 0.0)[:, None]) * np.isfinite(lse)[:, None]
            res["out"][q0:q1, h], res["lse"][q0:q1, h] = o, lse
            res["mass"][q0:q1, h] = p @ np.abs(vr[g])
            for t in range(q1 - q0):
                res["spread"][q0 + t, h] = p[t] @ np.abs(vr[g] - o[t])
            norms = np.where(seen, np.linalg.norm(kr[g], axis=1), 0.0).max(1)
            res["smax"][q0:q1, h] = np.linalg.norm(qr[:, h], axis=1) * norms * sc
            if not causal:
                w = np.zeros(-(-n // 16) * 16)
                w[:n] = p[0]
                res["weights"][r, g, :w.size // 16] += w.reshape(-1, 16).sum(1)
    return res


def evict(scores, tables, starts, lens, budget, first, last, weights=None, decay=1.0, bs=16):
    """Dict of the outputs of one eviction step (ranking on scores kept in float32)."""
    scores, tables, starts = np.asarray(scores), np.asarray(tables), np.asarray(starts)
    B, mb = tables.shape
    o = {"scores": np.zeros((B, mb), np.float32), "block_tables": np.full((B, mb), -1, np.int32),
         "block_starts": np.zeros((B, mb), np.int32), "seq_lens": np.array(lens, dtype=np.int32),
         "evicted": np.full((B, mb), -1, np.int32), "n_evicted": np.zeros(B, np.int32)}
    for r in range(B):
        n = -(-int(lens[r]) // bs)
        s = scores[r, :n].astype(np.float64) * float(np.float32(decay))
        if weights is not None:
            s = s + np.asarray(weights[r], dtype=np.float64)[:, :n].sum(0)
        s = s.astype(np.float32)
        rank = np.where(np.isnan(s), -np.inf, s)
        always = [b for b in range(n) if b < first or b >= n - last]
        others = sorted((b for b in range(n) if b not in set(always)), key=lambda b: (-rank[b], np.isnan(s[b]), b))
        room = budget - len(always)
        keep = list(range(n)) if n <= budget else sorted(always + others[:room])
        gone = [b for b in range(n) if b not in set(keep)]
        o["scores"][r, :len(keep)] = s[keep]
        o["block_tables"][r, :len(keep)] = tables[r, keep]
        o["block_starts"][r, :len(keep)] = starts[r, keep]
        o["evicted"][r, :len(gone)] = tables[r, gone]
        o["n_evicted"][r] = len(gone)
        o["seq_lens"][r] -= bs * len(gone)
    return o
