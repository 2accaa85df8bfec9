"""Batches on the GPU for the decode over one list of blocks, and their float64 results."""

import numpy as np


def f64(t):
    return t.double().cpu().numpy()


def make_batch(torch, dev, lens, Hq, Hkv, d, kv, seed, base=1e4):
    """Random pools ("e4m3" with power-of-two scales, or "bf16"), each block in one place, starts with gaps."""
    g = torch.Generator(device=dev).manual_seed(seed)
    B, mb = len(lens), -(-max(lens) // 16)
    n = torch.tensor(lens, device=dev)
    nb = int(((n + 15) // 16).sum()) + 1
    used = torch.arange(mb, device=dev) * 16 < n[:, None]
    tables = torch.full((B, mb), -1, dtype=torch.int32, device=dev)
    tables[used] = torch.randperm(nb, generator=g, device=dev)[:int(used.sum())].int()
    gaps = torch.randint(0, 3, (B, mb), generator=g, device=dev).cumsum(1)
    starts = torch.where(used, torch.arange(mb, device=dev) * 16 + gaps, 0).int()
    t = dict(kv=kv, base=base, Hkv=Hkv)
    for x in "kv":
        y = torch.randn(nb, Hkv, 16, d, generator=g, device=dev)
        if kv == "e4m3":
            s = torch.exp2(torch.ceil(torch.log2(y.abs().amax((2, 3)) / 448)))
            t[x + "_scale"], t[x + "_pool"] = s, (y / s[..., None, None]).to(torch.float8_e4m3fn)
        else:
            t[x + "_scale"], t[x + "_pool"] = torch.ones(nb, Hkv, device=dev), y.bfloat16()
    last = (n - 1).clamp(min=0)
    t.update(q=torch.randn(B, Hq, d, generator=g, device=dev).bfloat16(), block_tables=tables, block_starts=starts,
             seq_lens=n.int(), q_pos=(starts.long().gather(1, (last // 16)[:, None])[:, 0] + last % 16 + 1).int(),
             max_pos=int(starts.max()) + 40)
    return t


def call(mp, torch, t, rope, out, lse, bw, ws, **kw):
    """The call that records block weights (over the e4m3 cache also without them: bw None)."""
    if t["kv"] == "e4m3":
        return mp.attn_decode_q8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["block_tables"],
                                 t["block_starts"], t["seq_lens"], t["q_pos"], rope, out=out, lse=lse,
                                 block_weights=bw, workspace=ws, **kw)
    return mp.attn_decode_weights(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"],
                                  t["seq_lens"], t["q_pos"], rope, bw, out=out, lse=lse, workspace=ws, **kw)


def workspace_size(mp, t):
    f = mp.attn_decode_q8_workspace_size if t["kv"] == "e4m3" else mp.attn_decode_weights_workspace_size
    B, Hq, d = t["q"].shape
    return f(B, Hq, t["Hkv"], d, t["block_tables"].shape[1])


def reference(torch, t):
    """out, lse, block weights and the sizes that error bounds need (as oracle.cache8.attention returns them), with
    every product and sum in float64; keys with an unusable block or position are left out."""
    q, Hkv, base = t["q"].double(), t["Hkv"], t["base"]
    B, Hq, d = q.shape
    G, mb = Hq // Hkv, t["block_tables"].shape[1]
    nb = t["k_pool"].shape[0]
    res = {k: np.zeros((B, Hq, d)) for k in ("out", "spread", "mass")}
    res.update(lse=np.full((B, Hq), -np.inf), smax=np.zeros((B, Hq)), weights=np.zeros((B, Hkv, mb)))
    freq = base ** (-2 * torch.arange(d // 2, device=q.device, dtype=torch.float64) / d)

    def turn(x, pos):   # [..., n, d] rotated at pos [n]
        angle = pos.double()[:, None] * freq
        c, s, u, w = angle.cos(), angle.sin(), x[..., :d // 2], x[..., d // 2:]
        return torch.cat([u * c - w * s, w * c + u * s], -1)

    def bytes_of(p):
        return p.view(torch.uint8) if t["kv"] == "e4m3" else p
    for r in range(B):
        n = int(t["seq_lens"][r])
        if not n:
            continue
        j = torch.arange(n, device=q.device)
        blk = t["block_tables"][r].long()[j // 16]
        pos = t["block_starts"][r].long()[j // 16] + j % 16
        use = ((blk >= 0) & (blk < nb) & (pos >= 0) & (pos < t["max_pos"])).nonzero()[:, 0]
        if not len(use):
            continue
        j, blk, pos = j[use], blk[use], pos[use]
        qr = turn(q[r], t["q_pos"][r].expand(Hq))
        for g in range(Hkv):
            k, v = (bytes_of(t[x + "_pool"])[blk, g, j % 16].view(t[x + "_pool"].dtype).double() *
                    t[x + "_scale"].double()[blk, g][:, None] for x in "kv")
            k = turn(k, pos)
            h = slice(g * G, (g + 1) * G)
            s = qr[h] @ k.T / d ** 0.5
            p = torch.softmax(s, 1)
            o = p @ v
            res["out"][r, h], res["lse"][r, h] = f64(o), f64(torch.logsumexp(s, 1))
            res["mass"][r, h] = f64(p @ v.abs())
            for i in range(G):
                res["spread"][r, g * G + i] = f64(p[i] @ (v - o[i]).abs())
            res["smax"][r, h] = f64(qr[h].norm(dim=1) * k.norm(dim=1).max() / d ** 0.5)
            w = torch.zeros(mb * 16, dtype=torch.float64, device=q.device)
            w[j] = p.sum(0)
            res["weights"][r, g] = f64(w.view(-1, 16).sum(1))
    return res
