"""Measured cases of the 8-bit cache, the attention that reads it, and eviction by attention weight.

Operators (``op`` of a case):

``append``   new keys and values quantised into the paged e4m3 pools: one power-of-two scale for each block
             and kv head, which grows (and the block's earlier rows are re-rounded) when a new row needs it.
``decode``   one token per request over a paged position-free cache: keys rotated at their logical positions,
             softmax, values; with ``weights`` also each block's share of the attention, summed over the query
             heads of a kv head.  ``kv`` names the cache: "e4m3" (with scales) or the dtype of q.
``prefill``  a causal chunk of queries per request over the e4m3 cache (the chunk's own keys are its last ones).
``evict``    accumulated block weights are updated and each request keeps its ``budget`` best blocks (the first
             and last ones always), with its tables compacted in order.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits), with ``own`` true the
library's calls.  ``exact`` restates each operator from its definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

BS = 16          # keys per block
E4M3_MAX = 448.0
MIN_EXP = -100   # exponent of the smallest scale


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: two requests of 128 tokens, one shared block at two offsets, full precision
        dict(name="decode e4m3 tiny f32", op="decode", kv="e4m3", dtype="f32", B=2, Hq=4, Hkv=2, d=64, lmin=128,
             lmax=128, span=2, pool_spans=6, base=1e4, weights=False),
        # a RAG batch: 64 requests of 8192 tokens from 512-token spans shared by Zipf popularity
        dict(name="decode e4m3 rag", op="decode", kv="e4m3", dtype="bf16", B=64, Hq=32, Hkv=8, d=128, lmin=8192,
             lmax=8192, span=32, pool_spans=256, base=5e5, weights=False),
        # the largest: 8 contexts of 131072 tokens, 8 query heads a kv head, with the weights eviction needs
        dict(name="decode e4m3 long weights", op="decode", kv="e4m3", dtype="bf16", B=8, Hq=64, Hkv=8, d=128,
             lmin=131072, lmax=131072, span=256, pool_spans=48, base=5e5, weights=True),
        # a continuous batch: ragged private contexts (nothing shared), 7 query heads a kv head
        dict(name="decode e4m3 ragged", op="decode", kv="e4m3", dtype="bf16", B=128, Hq=28, Hkv=4, d=128, lmin=2048,
             lmax=32768, span=64, pool_spans=0, base=1e6, weights=False),
        # the same RAG batch over the bf16 cache, with block weights
        dict(name="decode bf16 rag weights", op="decode", kv="bf16", dtype="bf16", B=64, Hq=32, Hkv=8, d=128,
             lmin=8192, lmax=8192, span=32, pool_spans=256, base=5e5, weights=True),
        # a few short chats, one of them empty, small heads, with block weights
        dict(name="decode bf16 small weights", op="decode", kv="bf16", dtype="bf16", B=5, Hq=4, Hkv=2, d=64, lmin=0,
             lmax=700, span=4, pool_spans=0, base=1e4, weights=True),
        # a decode step's append: one token for each of 128 requests
        dict(name="append step", op="append", dtype="bf16", B=128, Hkv=8, d=128, nmin=1, nmax=1, smax=200),
        # span prefill's append: 16 chunks of up to 2048 tokens at odd offsets
        dict(name="append chunks", op="append", dtype="bf16", B=16, Hkv=4, d=128, nmin=1024, nmax=2048, smax=90),
        # the final prompt of 8 requests (512 tokens) over six cached 1024-token spans
        dict(name="prefill e4m3 rag", op="prefill", dtype="bf16", B=8, Hq=32, Hkv=8, d=128, qmin=512, qmax=512,
             cmin=6144, cmax=6144, span=64, pool_spans=64, base=5e5),
        # short prompts of odd lengths, some without any cached span, small heads
        dict(name="prefill e4m3 small", op="prefill", dtype="bf16", B=3, Hq=8, Hkv=2, d=64, qmin=1, qmax=120,
             cmin=0, cmax=580, span=8, pool_spans=12, base=1e4),
        # the RAG batch's tables cut from 512 to 384 blocks a request
        dict(name="evict rag", op="evict", dtype="bf16", B=64, Hkv=8, lmin=8000, lmax=8192, budget=384, first=4,
             last=8, decay=1.0),
        # the long contexts' tables halved, older weight fading
        dict(name="evict long", op="evict", dtype="bf16", B=8, Hkv=8, lmin=131072, lmax=131072, budget=4096, first=4,
             last=64, decay=0.98),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [(4, 2, 64), (8, 8, 64), (32, 8, 128), (28, 4, 128), (64, 8, 128), (16, 1, 128), (12, 12, 128), (15, 5, 64)]


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "prefill", "evict"])
    if op == "decode":
        kv = rng.choice(["e4m3", "e4m3", "own"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hq, Hkv, d = rng.choice(_HEADS)
        lmax = _log_int(rng, 1, 65536 if dtype == "bf16" else 2048)
        most = (1 << 28) if dtype == "bf16" else (1 << 23)
        B = _log_int(rng, 1, max(1, min(160, most // (lmax * Hkv * d))))
        span = _log_int(rng, 1, 128)
        return dict(op=op, kv="e4m3" if kv == "e4m3" else dtype, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d,
                    lmin=rng.choice([0, 1, lmax // 2, lmax]), lmax=lmax, span=span,
                    pool_spans=rng.choice([0, 5, 64]), base=rng.choice([1e4, 5e5, 1e6]),
                    weights=kv == "own" or rng.random() < 0.5)
    if op == "append":
        Hkv, d = rng.choice([(1, 128), (2, 64), (8, 128), (5, 64), (12, 128)])
        nmax = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(256, 65536 // nmax)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, Hkv=Hkv, d=d,
                    nmin=rng.choice([0, 1, nmax]), nmax=nmax, smax=_log_int(rng, 1, 500))
    if op == "prefill":
        Hq, Hkv, d = rng.choice(_HEADS)
        qmax, cmax = _log_int(rng, 1, 2048), _log_int(rng, 1, 16384)
        most = (1 << 36) // (Hq * d)   # query x key pairs
        B = _log_int(rng, 1, max(1, min(24, most // (qmax * (cmax + qmax)))))
        return dict(op=op, dtype="bf16", B=B, Hq=Hq, Hkv=Hkv, d=d, qmin=rng.choice([1, qmax]), qmax=qmax,
                    cmin=rng.choice([0, cmax]), cmax=cmax, span=_log_int(rng, 1, 64), pool_spans=rng.choice([0, 5, 40]),
                    base=rng.choice([1e4, 5e5]))
    lmax = _log_int(rng, 1, 131072)
    B = _log_int(rng, 1, max(1, min(256, (1 << 20) // lmax)))
    nb = -(-lmax // BS)
    first, last = rng.randint(0, 5), rng.randint(1, 9)
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), B=B, Hkv=rng.choice([1, 2, 8]), lmin=rng.choice([0, lmax]),
                lmax=lmax, budget=max(first + last, int(nb * rng.uniform(0.1, 1.1))), first=first, last=last,
                decay=rng.choice([1.0, 0.9]))


# ---------------------------------------------------------------------------------------------- inputs

def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rand_int(g, lo, hi, shape):
    return torch.randint(int(lo), int(hi) + 1, shape, generator=g, device="cuda")


def _rope_tables(max_pos, d, base):
    """cos | sin in the three stored forms, angles and functions in 64 bits."""
    p = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None]
    a = p * base ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    cs = torch.cat([a.cos(), a.sin()], 1)
    f32 = cs.float()
    c, s = f32[:, :d // 2].bfloat16(), f32[:, d // 2:].bfloat16()
    b16 = torch.stack([torch.cat([c, s, -s], 1), torch.cat([c, -s, s], 1)], 1).contiguous()
    return f32, cs.half(), b16


def _kv_values(g, shape, keys):
    """N(0, 1) values; a few key channels are larger, as key projections have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    if keys:
        x[..., 5::29] *= 3.0
    return x


def _tables(g, B, mb, lens, span, pool_spans):
    """Block tables and starts of B requests: shared spans drawn by Zipf popularity (s = 1.1), or private blocks;
    physical order permuted, spans back to back with small gaps in position."""
    n = -(-mb // span)
    if pool_spans:
        p = 1.0 / torch.arange(1, pool_spans + 1, device="cuda", dtype=torch.float64) ** 1.1
        ids = torch.multinomial(p, B * n, replacement=True, generator=g).view(B, n)
        blocks = (ids[..., None] * span + torch.arange(span, device="cuda")).view(B, n * span)[:, :mb]
        num = pool_spans * span
    else:
        blocks = torch.arange(B * mb, device="cuda").view(B, mb)
        num = B * mb
    blocks = torch.randperm(num, generator=g, device="cuda")[blocks]
    gaps = _rand_int(g, 0, 7, (B, n)).cumsum(1).repeat_interleave(span, 1)[:, :mb]
    starts = torch.arange(mb, device="cuda") * BS + gaps
    used = torch.arange(mb, device="cuda") * BS < lens[:, None]
    tables = torch.where(used, blocks, -1)
    return tables.int().contiguous(), torch.where(used, starts, 0).int().contiguous(), num, starts


def _scale_for(amax):
    """Smallest power of two s with amax <= 448 s (at least 2^-100)."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k.clamp(min=MIN_EXP), MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), k)


def _quantised_pool(g, num, Hkv, d, keys):
    x = _kv_values(g, (num, Hkv, BS, d), keys)
    s = _scale_for(x.abs().amax((2, 3)))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "evict":
        B, mb = case["B"], -(-case["lmax"] // BS)
        lens = _rand_int(g, case["lmin"], case["lmax"], (B,))
        lens[0] = case["lmax"]
        tables, starts, _, _ = _tables(g, B, mb, lens, 32, 0)
        # heavy-tailed block weights, as attention has them
        w = torch.exp(2.0 * torch.randn(B, case["Hkv"], mb, generator=g, device="cuda") - 6.0).to(_dt(case["dtype"]))
        st.update(block_weights=w, scores=torch.exp(2.0 * torch.randn(B, mb, generator=g, device="cuda") - 3.0),
                  block_tables=tables, block_starts=starts, seq_lens=lens.int())
        return st
    d, Hkv, B, dt = case["d"], case["Hkv"], case["B"], _dt(case["dtype"])
    if case["op"] == "append":
        n = _rand_int(g, case["nmin"], case["nmax"], (B,))
        n[0] = case["nmax"]
        start = _rand_int(g, 0, case["smax"], (B,))
        mb = -(-(case["smax"] + case["nmax"]) // BS)
        tables, _, num, _ = _tables(g, B, mb, start + n, 1, 0)
        cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), n.cumsum(0)])
        total = int(cu[-1])
        kp, ks = _quantised_pool(g, num, Hkv, d, True)
        vp, vs = _quantised_pool(g, num, Hkv, d, False)
        # rows of varying size: some need a larger scale than their block has
        size = torch.exp(0.5 * torch.randn(total, Hkv, 1, generator=g, device="cuda"))
        st.update(k_new=(_kv_values(g, (total, Hkv, d), True) * size).to(dt),
                  v_new=(_kv_values(g, (total, Hkv, d), False) * size).to(dt), cu=cu.int(), kv_start=start.int(),
                  block_tables=tables, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs)
        return st
    if case["op"] == "decode":
        lens = _rand_int(g, case["lmin"], case["lmax"], (B,))
        lens[0] = case["lmax"]
        mb = max(1, -(-case["lmax"] // BS))
    else:
        ql = _rand_int(_gen(7), case["qmin"], case["qmax"], (B,))   # the case's own: outputs keep their shape
        ql[0] = case["qmax"]
        ctx = _rand_int(g, case["cmin"], case["cmax"], (B,))
        ctx[0] = case["cmax"]
        lens, mb = ctx + ql, -(-(case["cmax"] + case["qmax"]) // BS)
    tables, starts, num, pos = _tables(g, B, mb, lens, case["span"], case["pool_spans"])
    max_pos = int(pos.max()) + 2 * BS
    last = (lens - 1).clamp(min=0)
    st["q_pos"] = (starts.long().gather(1, (last // BS)[:, None])[:, 0] + last % BS + 1).int()
    st["rope_f32"], st["rope_f16"], st["rope_b16"] = _rope_tables(max_pos, d, case["base"])
    if case["op"] == "decode" and case["kv"] != "e4m3":
        st["k_pool"] = _kv_values(g, (num, Hkv, BS, d), True).to(dt)
        st["v_pool"] = _kv_values(g, (num, Hkv, BS, d), False).to(dt)
    else:
        st["k_pool"], st["k_scale"] = _quantised_pool(g, num, Hkv, d, True)
        st["v_pool"], st["v_scale"] = _quantised_pool(g, num, Hkv, d, False)
    st.update(block_tables=tables, block_starts=starts)
    if case["op"] == "decode":
        st.update(q=torch.randn(B, case["Hq"], d, generator=g, device="cuda").to(dt), seq_lens=lens.int())
        if case["weights"]:
            st["block_weights"] = torch.zeros(B, Hkv, mb, dtype=dt, device="cuda")
    else:
        cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), ql.cumsum(0)])
        total = int(cu[-1])
        row = torch.repeat_interleave(torch.arange(B, device="cuda"), ql)
        j = ctx[row] + torch.arange(total, device="cuda") - cu[row]   # the token's key index
        st.update(q=torch.randn(total, case["Hq"], d, generator=g, device="cuda").to(dt), cu=cu.int(),
                  q_pos=(starts.long()[row, j // BS] + j % BS).int(), kv_lens=lens.int())
    return st


# ---------------------------------------------------------------------------------------------- the operators

def _rotate(x, pos, f32):
    """x [..., d] rotated at pos [...] (half rotation) with the 32-bit table."""
    h = x.shape[-1] // 2
    t = f32[pos.long()]
    c, s = t[..., :h], t[..., h:]
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _gathered(st):
    """Rotated keys and values of every request in 32 bits, [B, Hkv, mb * 16, d], and the key positions."""
    tables, starts = st["block_tables"].long().clamp(min=0), st["block_starts"].long()
    k, v = st["k_pool"].float(), st["v_pool"].float()
    if "k_scale" in st:
        k, v = k * st["k_scale"][..., None, None], v * st["v_scale"][..., None, None]
    B, mb = tables.shape
    pos = (starts[..., None] + torch.arange(BS, device="cuda")).view(B, mb * BS)
    k = k[tables].transpose(1, 2).reshape(B, st["Hkv"], mb * BS, st["d"])
    v = v[tables].transpose(1, 2).reshape(B, st["Hkv"], mb * BS, st["d"])
    return _rotate(k, pos[:, None].expand(B, st["Hkv"], mb * BS), st["rope_f32"]), v


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(m), m, 0.0))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(st):
    dt, B, Hkv, d = _dt(st["dtype"]), st["B"], st["Hkv"], st["d"]
    G = st["Hq"] // Hkv
    k, v = _gathered(st)
    q = st["q"].float()
    q = _rotate(q, st["q_pos"][:, None].expand(B, st["Hq"]), st["rope_f32"]).view(B, Hkv, G, d)
    s = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    s = s.masked_fill(torch.arange(k.shape[2], device="cuda") >= st["seq_lens"][:, None, None, None], -math.inf)
    p = _softmax(s)
    out = {"out": torch.matmul(p, v).view(B, st["Hq"], d).to(dt)}
    if st["weights"]:
        out["block_weights"] = p.view(B, Hkv, G, -1, BS).sum((2, 4)).to(dt)
    return out


def _plain_prefill(st):
    B, Hkv, d, G = st["B"], st["Hkv"], st["d"], st["Hq"] // st["Hkv"]
    cu, qm = st["cu"].long(), st["qmax"]
    ql = cu[1:] - cu[:-1]
    i = torch.arange(qm, device="cuda")
    have = i < ql[:, None]
    at = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = _rotate(st["q"].float()[at], st["q_pos"].long()[at][..., None].expand(B, qm, st["Hq"]), st["rope_f32"])
    k, v = _gathered(st)
    q = q.view(B, qm, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * qm, d)
    s = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, qm, -1) / math.sqrt(d)
    limit = st["kv_lens"].long()[:, None] - ql[:, None] + i   # last key that query i sees
    seen = torch.arange(k.shape[2], device="cuda") <= torch.where(have, limit, -1)[..., None]
    p = _softmax(s.masked_fill(~seen[:, None, None], -math.inf))
    o = torch.matmul(p.view(B, Hkv, G * qm, -1), v).view(B, Hkv, G, qm, d)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, qm, st["Hq"], d)[have].to(torch.bfloat16)}


def _plain_append_one(pool, scale, new, phys, slot, fresh, partial, before):
    """One of the two pools.  fresh / partial [num]: blocks that start with this call's rows, or already held
    `before` rows."""
    need = torch.zeros_like(scale).scatter_reduce(0, phys[:, None].expand(-1, scale.shape[1]),
                                                  new.abs().amax(-1), "amax")
    need = _scale_for(need)
    s = torch.where(fresh[:, None], need, torch.where(partial[:, None], torch.maximum(scale, need), scale))
    earlier = partial[:, None] & (torch.arange(BS, device="cuda") < before[:, None])
    grown = earlier[:, None] & (s > scale)[..., None]
    old = pool.float()
    again = (old * (scale / s)[..., None, None]).to(torch.float8_e4m3fn)
    bits = torch.where(grown[..., None], again.view(torch.uint8), pool.view(torch.uint8))
    bits[phys, :, slot] = (new / s[phys][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    pool.view(torch.uint8).copy_(bits)
    scale.copy_(s)


def _plain_append(st):
    cu, start = st["cu"].long(), st["kv_start"].long()
    total, num = st["k_new"].shape[0], st["k_pool"].shape[0]
    t = torch.arange(total, device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    j = start[r] + t - cu[r]
    phys, slot = st["block_tables"].long()[r, j // BS], j % BS
    fresh = torch.zeros(num, dtype=torch.bool, device="cuda")
    fresh[phys[slot == 0]] = True
    partial = torch.zeros_like(fresh)
    partial[phys] = True
    partial &= ~fresh
    before = torch.zeros(num, dtype=torch.long, device="cuda")
    ends = (start % BS != 0) & (cu[1:] > cu[:-1])
    before[st["block_tables"].long().gather(1, (start // BS)[:, None])[:, 0][ends]] = (start % BS)[ends]
    _plain_append_one(st["k_pool"], st["k_scale"], st["k_new"].float(), phys, slot, fresh, partial, before)
    _plain_append_one(st["v_pool"], st["v_scale"], st["v_new"].float(), phys, slot, fresh, partial, before)


def _plain_evict(st):
    tables, lens = st["block_tables"].long(), st["seq_lens"].long()
    B, mb = tables.shape
    n = (lens + BS - 1) // BS
    b = torch.arange(mb, device="cuda")
    used = b < n[:, None]
    # few terms, but their order must not show in the ranking: summed in 64 bits, kept in 32
    score = (st["scores"].double() * float(np.float32(st["decay"])) + st["block_weights"].double().sum(1)).float()
    held = used & ((b < st["first"]) | (b >= n[:, None] - st["last"]))
    rank = torch.where(held, math.inf, torch.where(used, score, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices   # ties: the lowest index first
    place = torch.empty_like(order).scatter_(1, order, b.expand(B, mb))
    keep = used & (place < st["budget"])
    kept = keep.sum(1)
    to = torch.where(keep, keep.cumsum(1) - 1, mb)                       # column mb takes what is dropped
    gone = used & ~keep
    off = torch.where(gone, gone.cumsum(1) - 1, mb)

    def moved(x, at, fill, dtype):
        y = torch.full((B, mb + 1), fill, device="cuda", dtype=dtype)
        return y.scatter_(1, at, x.to(dtype))[:, :mb].contiguous()

    return {"scores": moved(score, to, 0.0, torch.float32), "block_tables": moved(tables, to, -1, torch.int32),
            "block_starts": moved(st["block_starts"], to, 0, torch.int32),
            "seq_lens": (lens - BS * (n - kept)).int(), "evicted": moved(tables, off, -1, torch.int32),
            "n_evicted": (n - kept).int()}


def _held_values(st):
    """What the 8-bit pools stand for, and their scales."""
    return {"k": st["k_pool"].float() * st["k_scale"][..., None, None],
            "v": st["v_pool"].float() * st["v_scale"][..., None, None], "k_scale": st["k_scale"],
            "v_scale": st["v_scale"]}


def run(st):
    if own:
        import position_independent_kv_paged_gb300 as mp
    if st["op"] == "append":
        if own:
            mp.kv_append_q8(st["k_new"], st["v_new"], st["cu"], st["kv_start"], st["block_tables"], st["k_pool"],
                            st["v_pool"], st["k_scale"], st["v_scale"], max_new_len=st["nmax"])
        else:
            _plain_append(st)
        return _held_values(st)
    if st["op"] == "evict":
        if not own:
            return _plain_evict(st)
        r = mp.kv_evict(st["scores"], st["block_tables"], st["block_starts"], st["seq_lens"], st["budget"],
                        keep_first=st["first"], keep_last=st["last"], block_weights=st["block_weights"],
                        decay=st["decay"])
        return dict(zip(("scores", "block_tables", "block_starts", "seq_lens", "evicted", "n_evicted"), r))
    if not own:
        return _plain_decode(st) if st["op"] == "decode" else _plain_prefill(st)
    rope = mp.RopeTable(st["rope_f32"], st["rope_f16"], st["rope_b16"])
    mb = st["block_tables"].shape[1]
    if st["op"] == "prefill":
        if "workspace" not in st:   # kept from call to call, as a serving loop keeps it
            n = mp.attn_prefill_q8_workspace_size(st["B"], st["Hq"], st["Hkv"], st["d"], st["qmax"], mb)
            st["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        out, _ = mp.attn_prefill_q8(st["q"], st["cu"], st["q_pos"], st["k_pool"], st["v_pool"], st["k_scale"],
                                    st["v_scale"], st["block_tables"], st["block_starts"], st["kv_lens"], rope,
                                    st["qmax"], workspace=st["workspace"])
        return {"out": out}
    if "workspace" not in st:
        size = mp.attn_decode_q8_workspace_size if st["kv"] == "e4m3" else mp.attn_decode_weights_workspace_size
        n = size(st["B"], st["Hq"], st["Hkv"], st["d"], mb)
        st["workspace"] = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
    args = (st["block_tables"], st["block_starts"], st["seq_lens"], st["q_pos"], rope)
    if st["kv"] == "e4m3":
        out, _ = mp.attn_decode_q8(st["q"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], *args,
                                   block_weights=st.get("block_weights"), workspace=st["workspace"])
    else:
        out, _ = mp.attn_decode_weights(st["q"], st["k_pool"], st["v_pool"], *args, st["block_weights"],
                                        workspace=st["workspace"])
    return {"out": out, "block_weights": st["block_weights"]} if st["weights"] else {"out": out}


# ---------------------------------------------------------------------------------------------- work

def _distinct(case, blocks):
    """Blocks of the pool that `blocks` table entries of the batch touch, as expected from the draw."""
    if not case["pool_spans"]:
        return blocks
    p = 1.0 / np.arange(1, case["pool_spans"] + 1) ** 1.1
    p /= p.sum()
    return min(blocks, float((1 - (1 - p) ** (blocks / case["span"])).sum() * case["span"]))


def work(case):
    op = case["op"]
    if op == "evict":
        mb = -(-case["lmax"] // BS)
        elem = 2 if case["dtype"] == "bf16" else 4
        b = case["B"] * ((case["lmin"] + case["lmax"]) / 2 / BS) * (case["Hkv"] * elem + 12) + case["B"] * mb * 16
        return {"bytes": max(b, 1.0), "flops": case["B"] * mb * (case["Hkv"] + 2)}
    d, Hkv, B = case["d"], case["Hkv"], case["B"]
    elem = 2 if case["dtype"] == "bf16" else 4
    if op == "append":
        rows = B * (case["nmin"] + case["nmax"]) / 2 * Hkv * d * 2
        return {"bytes": max(rows * (elem + 1), 1.0), "flops": rows * 3}
    Hq = case["Hq"]
    if op == "decode":
        keys = B * (case["lmin"] + case["lmax"]) / 2
        b = _distinct(case, keys / BS) * BS * Hkv * d * 2 * (1 if case["kv"] == "e4m3" else elem)
        return {"bytes": b + keys / BS * 8 + 2 * B * Hq * d * elem, "flops": 4 * keys * Hq * d}
    q, c = (case["qmin"] + case["qmax"]) / 2, (case["cmin"] + case["cmax"]) / 2
    b = _distinct(case, B * (q + c) / BS) * BS * Hkv * d * 2 + 2 * B * q * Hq * d * elem
    return {"bytes": b, "flops": 4 * B * Hq * d * q * (c + (q + 1) / 2)}


# ---------------------------------------------------------------------------------------------- 64 bits

def _angles(pos, d, base):
    i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    return pos.double()[:, None] * torch.pow(torch.tensor(base, dtype=torch.float64, device="cuda"), -2.0 * i / d)


def _turn(x, pos, base):
    """x [n, heads, d] in 64 bits, as complex numbers times exp(i angle)."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                                            _angles(pos, 2 * h, base))[:, None]
    return torch.cat([z.real, z.imag], -1)


def _request_kv(st, r, n):
    j = torch.arange(n, device="cuda")
    blk = st["block_tables"][r].long()[j // BS]
    pos = st["block_starts"][r].long()[j // BS] + j % BS
    out = []
    for name in ("k", "v"):
        pool = st[name + "_pool"]
        if pool.dtype == torch.float8_e4m3fn:
            x = pool.view(torch.uint8)[blk, :, j % BS].view(torch.float8_e4m3fn).double()
            x = x * st[name + "_scale"].double()[blk][..., None]
        else:
            x = pool[blk, :, j % BS].double()
        out.append(x)
    return _turn(out[0], pos, st["base"]), out[1]


def _exact_attention(st, case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    G = case["Hq"] // Hkv
    decode = case["op"] == "decode"
    lens = (st["seq_lens"] if decode else st["kv_lens"]).tolist()
    cu = list(range(B + 1)) if decode else st["cu"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    w = torch.zeros(B, Hkv, st["block_tables"].shape[1], dtype=torch.float64, device="cuda")
    for r in range(B):
        n, q0, q1 = lens[r], cu[r], cu[r + 1]
        if n == 0 or q1 == q0:
            continue
        k, v = _request_kv(st, r, n)
        q = _turn(st["q"][q0:q1].double(), st["q_pos"][q0:q1], case["base"])
        for h in range(Hkv):
            s = torch.einsum("tgd,kd->tgk", q[:, h * G:(h + 1) * G], k[:, h]) * d ** -0.5
            if not decode:
                t = torch.arange(q1 - q0, device="cuda")
                hidden = torch.arange(n, device="cuda") > (n - (q1 - q0) + t)[:, None]
                s = s.masked_fill(hidden[:, None], -math.inf)
            p = torch.softmax(s, -1)
            out[q0:q1, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", p, v[:, h])
            if decode and case["weights"]:
                share = torch.zeros(-(-n // BS) * BS, dtype=torch.float64, device="cuda")
                share[:n] = p.sum((0, 1))
                w[r, h, :-(-n // BS)] = share.view(-1, BS).sum(1)
    if decode and case["weights"]:
        return {"out": out, "block_weights": w}
    return {"out": out}


def _e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, ties to even."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.rint(x / step) * step


def _exact_append(st, case):
    res = {}
    cu, start = st["cu"].tolist(), st["kv_start"].tolist()
    tables = st["block_tables"].cpu().numpy()
    for name in ("k", "v"):
        held = st[name + "_pool"].float().cpu().numpy().astype(np.float64)
        scale = st[name + "_scale"].cpu().numpy().astype(np.float64)
        new = st[name + "_new"].float().cpu().numpy().astype(np.float64)
        for r in range(case["B"]):
            i, n = 0, cu[r + 1] - cu[r]
            while i < n:
                j = start[r] + i
                b, s0 = tables[r, j // BS], j % BS
                m = min(n - i, BS - s0)
                rows = new[cu[r] + i:cu[r] + i + m].transpose(1, 0, 2)        # [Hkv, m, d]
                amax = np.abs(rows).max((1, 2))
                with np.errstate(divide="ignore"):
                    k = np.maximum(np.ceil(np.log2(amax / E4M3_MAX)), MIN_EXP)
                k = np.where(np.exp2(k) * E4M3_MAX < amax, k + 1, k)
                s = np.exp2(k)
                if s0:
                    s = np.maximum(s, scale[b])
                    for h in np.nonzero(s > scale[b])[0]:
                        held[b, h, :s0] = _e4m3(held[b, h, :s0] * (scale[b, h] / s[h]))
                held[b, :, s0:s0 + m] = _e4m3(rows / s[:, None, None])
                scale[b] = s
                i += m
        res[name] = torch.from_numpy(held * scale[..., None, None])
        res[name + "_scale"] = torch.from_numpy(scale)
    return {n: res[n] for n in ("k", "v", "k_scale", "v_scale")}


def _exact_evict(st, case):
    B, mb = case["B"], st["block_tables"].shape[1]
    w = st["block_weights"].float().cpu().numpy().astype(np.float64)
    old = st["scores"].cpu().numpy().astype(np.float64)
    tables, starts = st["block_tables"].cpu().numpy(), st["block_starts"].cpu().numpy()
    lens = st["seq_lens"].cpu().numpy()
    o = {"scores": np.zeros((B, mb)), "block_tables": np.full((B, mb), -1, np.int32),
         "block_starts": np.zeros((B, mb), np.int32), "seq_lens": lens.copy(),
         "evicted": np.full((B, mb), -1, np.int32), "n_evicted": np.zeros(B, np.int32)}
    decay = float(np.float32(case["decay"]))
    for r in range(B):
        n = -(-int(lens[r]) // BS)
        s = np.array([math.fsum([old[r, b] * decay, *w[r, :, b]]) for b in range(n)])
        always = {b for b in range(n) if b < case["first"] or b >= n - case["last"]}
        ranked = sorted(range(n), key=lambda b: (b not in always, -np.float32(s[b]), b))
        keep = sorted(ranked[:case["budget"]])
        gone = sorted(ranked[case["budget"]:])
        o["scores"][r, :len(keep)] = s[keep]
        o["block_tables"][r, :len(keep)] = tables[r, keep]
        o["block_starts"][r, :len(keep)] = starts[r, keep]
        o["evicted"][r, :len(gone)] = tables[r, gone]
        o["n_evicted"][r] = len(gone)
        o["seq_lens"][r] -= BS * len(gone)
    return o


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(st, case)
    if case["op"] == "append":
        return _exact_append(st, case)
    return _exact_attention(st, case)
