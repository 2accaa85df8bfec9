"""Batches for the tests of selected blocks and shared prefixes, and float64 results of decode over given keys."""

import numpy as np

from list_util import f64, make_batch


def batch(torch, dev, lens, Hq, Hkv, d, kv, seed, base=1e4):
    """list_util.make_batch, also with pools of float32 (kv "f32", and then the query)."""
    t = make_batch(torch, dev, lens, Hq, Hkv, d, "bf16" if kv == "f32" else kv, seed, base)
    t["kv"] = kv
    if kv == "f32":
        g = torch.Generator(device=dev).manual_seed(seed + 1)
        for x in ("k_pool", "v_pool", "q"):
            t[x] = torch.randn(t[x].shape, generator=g, device=dev)
    return t


def pools(t):
    names = ("k_pool", "v_pool", "k_scale", "v_scale") if t["kv"] == "e4m3" else ("k_pool", "v_pool")
    return tuple(t[n] for n in names)


def turned(torch, x, pos, base):
    """x [..., n, d] in float64 rotated at pos [n]."""
    h = x.shape[-1] // 2
    freq = base ** (-2 * torch.arange(h, device=x.device, dtype=torch.float64) / (2 * h))
    a = pos.double()[:, None] * freq
    c, s, u, w = a.cos(), a.sin(), x[..., :h], x[..., h:]
    return torch.cat([u * c - w * s, w * c + u * s], -1)


def held(torch, t, x, blk, g, slot):
    """float64 values [n, d] of pool x ("k" or "v") at (block, kv head, slot)."""
    p = t[x + "_pool"]
    if p.dtype == torch.float8_e4m3fn:
        return p.view(torch.uint8)[blk, g, slot].view(p.dtype).double() * t[x + "_scale"].double()[blk, g][:, None]
    return p[blk, g, slot].double()


def reference(torch, t, keys, scale=None):
    """What oracle.cache8.attention returns for one query a request, with `keys(r, g)` the indices of the keys that kv
    head g of request r attends to (a tensor; repeated ones count again)."""
    q, Hkv = t["q"].double(), t["Hkv"]
    B, Hq, d = q.shape
    G, nb = Hq // Hkv, t["k_pool"].shape[0]
    scale = scale or d ** -0.5
    res = {k: np.zeros((B, Hq, d)) for k in ("out", "spread", "mass")}
    res.update(lse=np.full((B, Hq), -np.inf), smax=np.zeros((B, Hq)))
    for r in range(B):
        qr = turned(torch, q[r], t["q_pos"][r].expand(Hq), t["base"])
        for g in range(Hkv):
            j = keys(r, g)
            blk = t["block_tables"][r].long()[j // 16]
            pos = t["block_starts"][r].long()[j // 16] + j % 16
            use = ((blk >= 0) & (blk < nb) & (pos >= 0) & (pos < t["max_pos"])).nonzero()[:, 0]
            if not len(use):
                continue
            j, blk, pos = j[use], blk[use], pos[use]
            k = turned(torch, held(torch, t, "k", blk, g, j % 16), pos, t["base"])
            v = held(torch, t, "v", blk, g, j % 16)
            h = slice(g * G, (g + 1) * G)
            s = qr[h] @ k.T * scale
            p = torch.softmax(s, 1)
            o = p @ v
            res["out"][r, h], res["lse"][r, h] = f64(o), f64(torch.logsumexp(s, 1))
            res["mass"][r, h] = f64(p @ v.abs())
            for i in range(G):
                res["spread"][r, g * G + i] = f64(p[i] @ (v - o[i]).abs())
            res["smax"][r, h] = f64(qr[h].norm(dim=1) * k.norm(dim=1).max() * scale)
    return res


def keys_of(torch, t, selected):
    """keys(r, g) of a selection [B, Hkv, n] (a list or tensor of block numbers, -1: unused)."""
    def keys(r, g):
        L = int(t["seq_lens"][r])
        n = -(-L // 16)
        s = torch.as_tensor(selected[r][g], device=t["q"].device).long()[:n]
        s = s[(s >= 0) & (s < n)]
        j = (s[:, None] * 16 + torch.arange(16, device=s.device)).view(-1)
        return j[j < L]
    return keys
