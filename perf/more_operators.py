"""Measured cases of decode that reads less of the cache: attention over selected blocks, and over a shared prefix.

Operators (``op`` of a case):

``means``     summaries of the blocks that new keys were appended to: the mean of a block's keys, each rotated by its
              slot, so that its product with the query rotated by (query position - block start) is the mean score of
              the block's keys wherever the block is read.  ``kv`` names the cache: "e4m3" or the summaries' dtype.
``scores``    one token per request scores every block of its table: the largest product over the query heads of
              a kv head; minus infinity past the request's length.
``select``    the ``budget`` best blocks by score for each request and kv head; the first and last ones always;
              ascending, then -1.  Scores are inputs.
``selected``  one token per request attends to the keys of its selected blocks.  ``kv`` as above.
``prefix``    one token per request attends to all its keys, where groups of consecutive requests begin with the same
              blocks (a system prompt, a document) at the same positions.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits), with ``own`` true the
library's calls.  ``exact`` restates each operator from its definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

BS = 16          # keys per block


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step: the blocks that one new token of each of 128 requests went into
        dict(name="means step", op="means", kv="bf16", dtype="bf16", B=128, Hkv=8, d=128, nmin=1, nmax=1, smax=200),
        # span prefill: 16 chunks of up to 2048 tokens appended at odd offsets
        dict(name="means chunks", op="means", kv="bf16", dtype="bf16", B=16, Hkv=4, d=128, nmin=1024, nmax=2048,
             smax=90),
        # a RAG batch: 64 requests of 8192 tokens from 512-token spans shared by Zipf popularity
        dict(name="scores rag", op="scores", dtype="bf16", B=64, Hq=32, Hkv=8, d=128, lmin=8192, lmax=8192, span=32,
             pool_spans=256, base=5e5),
        # 8 contexts of 131072 tokens, 8 query heads a kv head
        dict(name="scores long", op="scores", dtype="bf16", B=8, Hq=64, Hkv=8, d=128, lmin=131072, lmax=131072,
             span=256, pool_spans=48, base=5e5),
        # the RAG batch's tables: an eighth of 512 blocks
        dict(name="select rag", op="select", B=64, Hkv=8, lmin=8000, lmax=8192, budget=64, first=1, last=4,
             coarse=False),
        # the long contexts' tables: 512 of 8192 blocks, scores of few bits (many ties)
        dict(name="select long", op="select", B=8, Hkv=8, lmin=131072, lmax=131072, budget=512, first=4, last=16,
             coarse=True),
        # the smallest call: two requests of 128 tokens, half of their blocks, full precision
        dict(name="selected tiny f32", op="selected", kv="f32", dtype="f32", B=2, Hq=4, Hkv=2, d=64, lmin=128,
             lmax=128, budget=4, span=2, pool_spans=6, base=1e4),
        # the RAG batch, 64 blocks (1024 tokens) of each context
        dict(name="selected rag", op="selected", kv="bf16", dtype="bf16", B=64, Hq=32, Hkv=8, d=128, lmin=8192,
             lmax=8192, budget=64, span=32, pool_spans=256, base=5e5),
        # ragged long contexts over the 8-bit cache, nothing shared, 512 blocks of each
        dict(name="selected e4m3 long", op="selected", kv="e4m3", dtype="bf16", B=8, Hq=64, Hkv=8, d=128, lmin=65536,
             lmax=131072, budget=512, span=256, pool_spans=0, base=5e5),
        # a few chats behind one short system prompt, small heads
        dict(name="prefix small", op="prefix", dtype="bf16", B=5, Hq=4, Hkv=2, d=64, P=1, pmin=16, pmax=16, omin=0,
             omax=300, pad=False, base=1e4),
        # 64 questions about three documents of up to 8192 tokens, 7 query heads a kv head, ragged own contexts
        dict(name="prefix documents", op="prefix", dtype="bf16", B=64, Hq=28, Hkv=4, d=128, P=3, pmin=256, pmax=512,
             omin=64, omax=2048, pad=False, base=1e6),
        # the largest: 256 requests behind one prompt of 32768 tokens, 8 query heads a kv head
        dict(name="prefix many", op="prefix", dtype="bf16", B=256, Hq=64, Hkv=8, d=128, P=1, pmin=2048, pmax=2048,
             omin=16, omax=512, pad=False, base=5e5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [(4, 2, 64), (8, 8, 64), (32, 8, 128), (28, 4, 128), (64, 8, 128), (16, 1, 128), (12, 12, 128), (15, 5, 64)]


def draw(rng):
    op = rng.choice(["means", "scores", "select", "selected", "selected", "prefix", "prefix"])
    if op == "means":
        Hkv, d = rng.choice([(1, 128), (2, 64), (8, 128), (5, 64), (12, 128)])
        nmax = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(256, 65536 // nmax)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, kv=rng.choice([dtype, "e4m3"]), dtype=dtype, B=B, Hkv=Hkv, d=d,
                    nmin=rng.choice([0, 1, nmax]), nmax=nmax, smax=_log_int(rng, 1, 500))
    if op == "select":
        lmax = _log_int(rng, 400, 262144)
        B = _log_int(rng, 1, max(1, min(256, (1 << 21) // lmax)))
        first, last = rng.randint(0, 5), rng.randint(1, 9)
        return dict(op=op, B=B, Hkv=rng.choice([1, 2, 8]), lmin=rng.choice([0, lmax]), lmax=lmax,
                    budget=max(first + last + 1, int(lmax // BS * rng.uniform(0.03, 0.7))), first=first, last=last,
                    coarse=rng.random() < 0.5)
    Hq, Hkv, d = rng.choice(_HEADS)
    if op == "prefix":
        pmax = _log_int(rng, 1, 1024)
        omax = _log_int(rng, 1, 4096)
        most = (1 << 36) // (Hq * d)   # query x key pairs
        B = _log_int(rng, 1, max(1, min(256, most // (pmax * BS + omax), (1 << 26) // (omax * Hkv * d))))
        return dict(op=op, dtype="bf16", B=B, Hq=Hq, Hkv=Hkv, d=d, P=rng.randint(1, max(1, min(5, B))),
                    pmin=rng.choice([0, 1, pmax]), pmax=pmax, omin=rng.choice([0, 1, omax]), omax=omax,
                    pad=rng.random() < 0.3, base=rng.choice([1e4, 5e5, 1e6]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    lmax = _log_int(rng, 1, 131072)
    most = 1 << 26 if dtype == "bf16" else 1 << 25   # values read, for `scores` halved
    B = _log_int(rng, 1, max(1, min(160, (most * BS // 2 if op == "scores" else most) // (lmax * Hkv * d))))
    case = dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, d=d, lmin=rng.choice([0, 1, lmax // 2, lmax]), lmax=lmax,
                span=_log_int(rng, 1, 128), pool_spans=rng.choice([0, 5, 64]), base=rng.choice([1e4, 5e5, 1e6]))
    if op == "selected":
        nb = min(-(-lmax // BS), 512 if dtype == "bf16" else 64)
        case.update(kv=rng.choice([dtype, "e4m3"]), budget=_log_int(rng, 2, max(2, nb)))
    return case


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


def _quantised_pool(g, num, Hkv, d, keys):
    """e4m3 values with a power-of-two scale for each block and kv head."""
    x = _kv_values(g, (num, Hkv, BS, d), keys)
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448.0)))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn), s


def _pools(st, g, num, both=True):
    for name in ("k", "v") if both else ("k",):
        if st["kv"] == "e4m3":
            st[name + "_pool"], st[name + "_scale"] = _quantised_pool(g, num, st["Hkv"], st["d"], name == "k")
        else:
            st[name + "_pool"] = _kv_values(g, (num, st["Hkv"], BS, st["d"]), name == "k").to(_dt(st["kv"]))


def _next_pos(starts, lens):
    """Position behind each request's last key."""
    last = (lens - 1).clamp(min=0)
    return (starts.long().gather(1, (last // BS)[:, None])[:, 0] + last % BS + 1).int()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    B, Hkv = case["B"], case["Hkv"]
    if case["op"] == "select":
        mb = -(-case["lmax"] // BS)
        lens = _rand_int(g, case["lmin"], case["lmax"], (B,))
        lens[0] = case["lmax"]
        s = 2.0 * torch.randn(B, Hkv, mb, generator=g, device="cuda")   # mean scores of blocks
        if case["coarse"]:
            s = s.bfloat16().float()
        past = torch.arange(mb, device="cuda") * BS >= lens[:, None]
        st.update(scores=s.masked_fill(past[:, None], -math.inf), seq_lens=lens.int())
        return st
    d, dt = case["d"], _dt(case["dtype"])
    if case["op"] == "means":
        n = _rand_int(g, case["nmin"], case["nmax"], (B,))
        n[0] = case["nmax"]
        start = _rand_int(g, 0, case["smax"], (B,))
        mb = -(-(case["smax"] + case["nmax"]) // BS)
        tables, _, num, _ = _tables(g, B, mb, start + n, 1, 0)
        _pools(st, g, num, both=False)
        st["rope_f32"] = _rope_tables(BS, d, 1e4)[0]
        st.update(cu=torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), n.cumsum(0)]).int(),
                  kv_start=start.int(), block_tables=tables,
                  means=(0.3 * _kv_values(g, (num, Hkv, d), True)).to(dt))   # those of the other blocks
        return st
    if case["op"] == "prefix":
        P, mb = case["P"], case["pmax"] + -(-case["omax"] // BS)
        cut = torch.randperm(B - 1, generator=g, device="cuda")[:P - 1].sort().values + 1
        cu = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), B)])
        blocks = _rand_int(g, case["pmin"], case["pmax"], (P,))
        blocks[0] = case["pmax"]
        of = torch.repeat_interleave(torch.arange(P, device="cuda"), cu[1:] - cu[:-1])
        extra = _rand_int(g, case["omin"], case["omax"], (B,))
        extra[0] = case["omax"]
        lens = blocks[of] * BS + extra
        if case["pad"]:
            lens[(B + 1) // 2:][::3] = 0   # rows that hold no request
        b = torch.arange(mb, device="cuda")
        own_ids = P * case["pmax"] + torch.arange(B, device="cuda")[:, None] * mb + b
        ids = torch.where(b < blocks[of][:, None], of[:, None] * case["pmax"] + b, own_ids)
        used, inverse = torch.unique(ids[b * BS < lens[:, None]], return_inverse=True)   # blocks that some table holds
        num = max(1, int(used.numel()))
        tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
        tables[b * BS < lens[:, None]] = torch.randperm(num, generator=g, device="cuda")[inverse].int()
        gaps = (_rand_int(g, 0, 7, (P, mb)) * (b % 32 == 0)).cumsum(1)
        starts = (b * BS + gaps[of])
        st["kv"] = "bf16"
        _pools(st, g, num)
        st.update(block_tables=tables, block_starts=torch.where(tables >= 0, starts, 0).int(), seq_lens=lens.int(),
                  q_pos=_next_pos(starts, lens), cu=cu.int(), prefix_blocks=blocks.int(),
                  max_requests=int((cu[1:] - cu[:-1]).max()), max_prefix=int(blocks.max()))
        max_pos = int(starts.max()) + 2 * BS
    else:
        lens = _rand_int(g, case["lmin"], case["lmax"], (B,))
        lens[0] = case["lmax"]
        mb = -(-case["lmax"] // BS)
        tables, starts, num, pos = _tables(g, B, mb, lens, case["span"], case["pool_spans"])
        max_pos = int(pos.max()) + 2 * BS
        st.update(block_tables=tables, block_starts=starts, seq_lens=lens.int(), q_pos=_next_pos(starts, lens))
        if case["op"] == "scores":
            st["means"] = (0.3 * _kv_values(g, (num, Hkv, d), True)).to(dt)
        else:
            _pools(st, g, num)
            # some blocks matter to a kv head more than others; the first and the last are always among them
            s = torch.randn(B, Hkv, mb, generator=g, device="cuda")
            n = (lens + BS - 1) // BS
            b = torch.arange(mb, device="cuda")
            s = s.masked_fill((b == 0) | (b == n[:, None, None] - 1), math.inf)
            s = s.masked_fill(b >= n[:, None, None], -math.inf)
            k = min(case["budget"], mb)
            best = s.topk(k, dim=2).indices
            sel = torch.where(best < n[:, None, None], best, mb).sort(2).values
            st["selected"] = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
            st["selected"][..., :k] = torch.where(sel < mb, sel, -1).int()
    st["rope_f32"], st["rope_f16"], st["rope_b16"] = _rope_tables(max_pos, d, case["base"])
    st["q"] = torch.randn(B, case["Hq"], d, generator=g, device="cuda").to(dt)
    return st


# ---------------------------------------------------------------------------------------------- the operators

def _rotate(x, pos, f32):
    """x [..., d] rotated at pos [...] (half rotation) with the 32-bit table."""
    h = x.shape[-1] // 2
    t = f32[pos.long()]
    c, s = t[..., :h], t[..., h:]
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(m), m, 0.0))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _held(st, name, at, head=None):
    """Keys or values of the blocks `at` (of one kv head each, if given) in 32 bits."""
    pool, scale = st[name + "_pool"], st.get(name + "_scale")
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8)[at] if head is None else pool.view(torch.uint8)[at, head]
        return x.view(pool.dtype).float() * (scale[at] if head is None else scale[at, head])[..., None, None]
    return (pool[at] if head is None else pool[at, head]).float()


def _plain_means(st):
    cu, start, d = st["cu"].long(), st["kv_start"].long(), st["d"]
    end = start + cu[1:] - cu[:-1]
    b = (start // BS)[:, None] + torch.arange((st["nmax"] + BS - 2) // BS + 1, device="cuda")
    touched = (b * BS < end[:, None]) & (end > start)[:, None]
    phys = st["block_tables"].long().gather(1, b.clamp(max=st["block_tables"].shape[1] - 1))[touched]
    count = (end[:, None] - b * BS).clamp(max=BS)[touched]
    k = _held(st, "k", phys)                                                     # [n, Hkv, 16, d]
    slot = torch.arange(BS, device="cuda")
    k = _rotate(k, slot.expand(k.shape[:3]), st["rope_f32"])
    k = k.masked_fill((slot >= count[:, None])[:, None, :, None], 0.0)
    st["means"][phys] = (k.sum(2) / count[:, None, None]).to(st["means"].dtype)
    return {"means": st["means"]}


def _plain_scores(st):
    B, Hkv, d, mb = st["B"], st["Hkv"], st["d"], st["block_tables"].shape[1]
    m = st["means"][st["block_tables"].long().clamp(min=0)].float().transpose(1, 2)   # [B, Hkv, mb, d]
    m = _rotate(m, st["block_starts"][:, None].expand(B, Hkv, mb), st["rope_f32"])
    q = _rotate(st["q"].float(), st["q_pos"][:, None].expand(B, st["Hq"]), st["rope_f32"]).view(B, Hkv, -1, d)
    s = torch.matmul(q, m.transpose(2, 3)).amax(2) / math.sqrt(d)
    past = torch.arange(mb, device="cuda") * BS >= st["seq_lens"][:, None, None]
    return {"scores": s.masked_fill(past, -math.inf)}


def _plain_select(st):
    n = ((st["seq_lens"].long() + BS - 1) // BS)[:, None, None]
    mb = st["scores"].shape[2]
    b = torch.arange(mb, device="cuda")
    held = (b < st["first"]) | (b >= n - st["last"])
    rank = torch.where(b < n, torch.where(held, math.inf, st["scores"]), -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices       # ties: the lowest index first
    best = order[..., :st["budget"]]
    best = torch.where(best < n, best, mb).sort(2).values
    out = torch.full((*st["scores"].shape[:2], st["budget"]), -1, dtype=torch.int32, device="cuda")
    out[..., :best.shape[2]] = torch.where(best < mb, best, -1).int()
    return {"selected": out}


def _plain_selected(st):
    B, Hkv, d, S = st["B"], st["Hkv"], st["d"], st["budget"]
    sel = st["selected"].long()
    at = sel.clamp(min=0)
    rows = torch.arange(B, device="cuda")[:, None, None]
    phys, start = st["block_tables"].long()[rows, at].clamp(min=0), st["block_starts"].long()[rows, at]
    head = torch.arange(Hkv, device="cuda")[:, None]
    slot = torch.arange(BS, device="cuda")
    k = _rotate(_held(st, "k", phys, head), start[..., None] + slot, st["rope_f32"]).view(B, Hkv, S * BS, d)
    v = _held(st, "v", phys, head).view(B, Hkv, S * BS, d)
    q = _rotate(st["q"].float(), st["q_pos"][:, None].expand(B, st["Hq"]), st["rope_f32"]).view(B, Hkv, -1, d)
    use = (sel >= 0)[..., None] & (at[..., None] * BS + slot < st["seq_lens"][:, None, None, None])
    s = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    p = _softmax(s.masked_fill(~use.view(B, Hkv, 1, S * BS), -math.inf))
    return {"out": torch.matmul(p, v).view(B, st["Hq"], d).to(_dt(st["dtype"]))}


def _plain_prefix(st):
    """The prefixes' keys are gathered once a group, and all its queries multiply them."""
    B, Hq, Hkv, d, P = st["B"], st["Hq"], st["Hkv"], st["d"], st["P"]
    G, cu, blocks, lens = Hq // Hkv, st["cu"].long(), st["prefix_blocks"].long(), st["seq_lens"].long()
    tables, starts, mb = st["block_tables"].long(), st["block_starts"].long(), st["block_tables"].shape[1]
    slot = torch.arange(BS, device="cuda")
    nb, most = st["max_prefix"], st["max_requests"]
    n = cu[1:] - cu[:-1]
    q = _rotate(st["q"].float(), st["q_pos"][:, None].expand(B, Hq), st["rope_f32"]).view(B, Hkv, G, d)
    # prefixes: the table row of a group's request that is long enough
    row = cu[:-1, None] + torch.arange(most, device="cuda")
    inside = torch.arange(most, device="cuda") < n[:, None]
    row = torch.where(inside, row, 0)
    lead = row.gather(1, (inside & (lens[row] >= blocks[:, None] * BS)).float().argmax(1, keepdim=True))[:, 0]
    pk = _held(st, "k", tables[lead, :nb].clamp(min=0)).transpose(1, 2)          # [P, Hkv, nb, 16, d]
    pos = (starts[lead, :nb, None] + slot)[:, None].expand(P, Hkv, nb, BS)
    pk = _rotate(pk, pos, st["rope_f32"]).reshape(P, Hkv, nb * BS, d)
    pv = _held(st, "v", tables[lead, :nb].clamp(min=0)).transpose(1, 2).reshape(P, Hkv, nb * BS, d)
    pq = q[row].transpose(1, 2).reshape(P, Hkv, most * G, d)
    s1 = (torch.matmul(pq, pk.transpose(2, 3)) / math.sqrt(d)).view(P, Hkv, most, G, nb * BS).transpose(1, 2)[inside]
    of = torch.repeat_interleave(torch.arange(P, device="cuda"), n)
    limit = torch.minimum(blocks[of] * BS, lens)[:, None, None, None]
    s1 = s1.masked_fill(torch.arange(nb * BS, device="cuda") >= limit, -math.inf)
    # each request's own blocks
    no = -(-st["omax"] // BS)
    b = blocks[of][:, None] + torch.arange(no, device="cuda")
    at = b.clamp(max=mb - 1)
    ot = tables.gather(1, at).clamp(min=0)
    ok = _held(st, "k", ot).transpose(1, 2)
    ok = _rotate(ok, (starts.gather(1, at)[..., None] + slot)[:, None].expand(B, Hkv, no, BS), st["rope_f32"])
    ov = _held(st, "v", ot).transpose(1, 2).reshape(B, Hkv, no * BS, d)
    s2 = torch.matmul(q, ok.reshape(B, Hkv, no * BS, d).transpose(2, 3)) / math.sqrt(d)
    past = (b[..., None] * BS + slot).view(B, no * BS) >= lens[:, None]
    p = _softmax(torch.cat([s1, s2.masked_fill(past[:, None, None], -math.inf)], 3))
    p1 = p.new_zeros(P, most, Hkv, G, nb * BS)
    p1[inside] = p[..., :nb * BS]
    o1 = torch.matmul(p1.transpose(1, 2).reshape(P, Hkv, most * G, nb * BS), pv)
    o1 = o1.view(P, Hkv, most, G, d).transpose(1, 2)[inside]
    return {"out": (o1 + torch.matmul(p[..., nb * BS:], ov)).reshape(B, Hq, d).to(torch.bfloat16)}


_PLAIN = {"means": _plain_means, "scores": _plain_scores, "select": _plain_select, "selected": _plain_selected,
          "prefix": _plain_prefix}


def _own_run(st):
    import position_independent_kv_paged_gb300 as mp
    op = st["op"]
    if op == "select":
        return {"selected": mp.block_select(st["scores"], st["seq_lens"], st["budget"], keep_first=st["first"],
                                            keep_last=st["last"])}
    rope = mp.RopeTable(st["rope_f32"], st.get("rope_f16"), st.get("rope_b16"))
    if op == "means":
        if st["kv"] == "e4m3":
            mp.kv_block_means_q8(st["cu"], st["kv_start"], st["block_tables"], st["k_pool"], st["k_scale"], rope,
                                 st["means"], max_new_len=st["nmax"])
        else:
            mp.kv_block_means(st["cu"], st["kv_start"], st["block_tables"], st["k_pool"], rope, st["means"],
                              max_new_len=st["nmax"])
        return {"means": st["means"]}
    if op == "scores":
        return {"scores": mp.block_scores(st["q"], st["means"], st["block_tables"], st["block_starts"],
                                          st["seq_lens"], st["q_pos"], rope)}
    args = (st["block_tables"], st["block_starts"], st["seq_lens"], st["q_pos"], rope)
    mb = st["block_tables"].shape[1]
    if op == "selected":
        if "workspace" not in st:   # kept from call to call, as a serving loop keeps it
            n = mp.attn_decode_selected_workspace_size(st["B"], st["Hq"], st["Hkv"], st["d"], st["budget"])
            st["workspace"] = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
        if st["kv"] == "e4m3":
            out, _ = mp.attn_decode_selected_q8(st["q"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"],
                                                *args, st["selected"], workspace=st["workspace"])
        else:
            out, _ = mp.attn_decode_selected(st["q"], st["k_pool"], st["v_pool"], *args, st["selected"],
                                             workspace=st["workspace"])
        return {"out": out}
    if "workspace" not in st:
        n = mp.attn_decode_prefix_workspace_size(st["B"], st["Hq"], st["Hkv"], st["d"], mb, st["P"],
                                                 st["max_requests"], st["max_prefix"])
        st["workspace"] = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
    out, _ = mp.attn_decode_prefix(st["q"], st["k_pool"], st["v_pool"], *args, st["cu"], st["prefix_blocks"],
                                   max_requests=st["max_requests"], max_prefix_blocks=st["max_prefix"],
                                   workspace=st["workspace"])
    return {"out": out}


def run(st):
    if own:
        return _own_run(st)
    return _PLAIN[st["op"]](st)


# ---------------------------------------------------------------------------------------------- work

def _elem(name):
    return {"f32": 4, "bf16": 2, "e4m3": 1}[name]


def _distinct(case, blocks):
    """Blocks of the pool that `blocks` table entries of the batch touch, as expected from the draw."""
    if not case["pool_spans"]:
        return blocks
    p = 1.0 / np.arange(1, case["pool_spans"] + 1) ** 1.1
    p /= p.sum()
    return min(blocks, float((1 - (1 - p) ** (blocks / case["span"])).sum() * case["span"]))


def work(case):
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    if op == "select":
        n = (case["lmin"] + case["lmax"]) / 2 / BS
        return {"bytes": 4 * B * Hkv * (n + case["budget"]) + 4 * B, "flops": B * Hkv * n}
    d, elem = case["d"], _elem(case["dtype"])
    if op == "means":
        rows = B * ((case["nmin"] + case["nmax"]) / 2 + (BS - 1) / 2) * Hkv * d   # the first block's earlier rows too
        return {"bytes": rows * _elem(case["kv"]) + max(rows / BS, B * Hkv * d) * elem, "flops": 4 * rows}
    Hq = case["Hq"]
    if op == "prefix":
        pre, each = case["P"] * (case["pmin"] + case["pmax"]) / 2 * BS, (case["omin"] + case["omax"]) / 2
        return {"bytes": (pre + B * each) * Hkv * d * 2 * elem + 2 * B * Hq * d * elem,
                "flops": 4 * B * Hq * d * (pre / case["P"] + each)}
    n = (case["lmin"] + case["lmax"]) / 2 / BS
    if op == "scores":
        b = _distinct(case, B * n) * Hkv * d * elem + B * n * 8 + 4 * B * Hkv * (-(-case["lmax"] // BS))
        return {"bytes": b + B * Hq * d * elem, "flops": B * n * Hkv * d * (3 + 2 * Hq // Hkv)}
    k = min(case["budget"], n)   # blocks a kv head reads
    b = min(B * k * Hkv, _distinct(case, B * n) * Hkv) * BS * d * 2 * _elem(case["kv"])
    return {"bytes": b + 4 * B * Hkv * k + 2 * B * Hq * d * elem, "flops": 4 * B * k * BS * Hq * d}


# ---------------------------------------------------------------------------------------------- 64 bits

def _turn(x, pos, base):
    """x [n, heads, d] in 64 bits, as complex numbers times exp(i angle), angle = pos base^(-2 i / d)."""
    h = x.shape[-1] // 2
    i = torch.arange(h, device="cuda", dtype=torch.float64)
    a = pos.double()[:, None] * torch.pow(torch.tensor(base, dtype=torch.float64, device="cuda"), -i / h)
    one = torch.ones((), dtype=torch.float64, device="cuda")
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(one, a)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _rows(st, name, blk, slot):
    """Keys or values (block, slot) of every kv head in 64 bits, [n, Hkv, d]."""
    pool = st[name + "_pool"]
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8)[blk, :, slot].view(pool.dtype).double()
        return x * st[name + "_scale"].double()[blk][..., None]
    return pool[blk, :, slot].double()


def _exact_means(st, case):
    out = st["means"].double()
    cu, start = st["cu"].tolist(), st["kv_start"].tolist()
    r, j, last = [], [], []
    for i in range(case["B"]):
        first, end = start[i], start[i] + cu[i + 1] - cu[i]
        if end > first:
            r += [i] * (-(-end // BS) - first // BS)
            j += range(first // BS, -(-end // BS))
            last += [end] * (-(-end // BS) - first // BS)
    if not r:
        return {"means": out}
    r, j, last = (torch.tensor(x, device="cuda") for x in (r, j, last))
    blk = st["block_tables"].long()[r, j]
    total = torch.zeros(len(r), case["Hkv"], case["d"], dtype=torch.float64, device="cuda")
    for s in range(BS):
        x = _turn(_rows(st, "k", blk, torch.full_like(blk, s)), torch.full_like(blk, s), 1e4)
        total += torch.where((j * BS + s < last)[:, None, None], x, 0.0)
    out[blk] = total / (last - j * BS).clamp(max=BS)[:, None, None]
    return {"means": out}


def _exact_scores(st, case):
    B, Hkv, d, mb = case["B"], case["Hkv"], case["d"], st["block_tables"].shape[1]
    out = torch.full((B, Hkv, mb), -math.inf, dtype=torch.float64, device="cuda")
    for r, L in enumerate(st["seq_lens"].tolist()):
        n = -(-L // BS)
        if n:
            m = _turn(st["means"][st["block_tables"][r, :n].long()].double(), st["block_starts"][r, :n], case["base"])
            q = _turn(st["q"][r:r + 1].double(), st["q_pos"][r:r + 1], case["base"])[0].view(Hkv, -1, d)
            out[r, :, :n] = torch.einsum("hgd,bhd->hgb", q, m).amax(1) * d ** -0.5
    return {"scores": out}


def _exact_select(st, case):
    s = st["scores"].cpu().numpy()
    out = np.full((*s.shape[:2], case["budget"]), -1, np.int32)
    for r, L in enumerate(st["seq_lens"].tolist()):
        n = -(-L // BS)
        b = np.arange(n)
        always = (b < case["first"]) | (b >= n - case["last"])
        for h in range(s.shape[1]):
            best = np.lexsort((b, -s[r, h, :n], ~always))[:case["budget"]]
            out[r, h, :len(best)] = np.sort(best)
    return {"selected": out}


def _attend(q, k, v):
    """q [Hkv, G, d], k and v [n, Hkv, d]"""
    p = torch.softmax(torch.einsum("hgd,khd->hgk", q, k) * q.shape[-1] ** -0.5, -1)
    return torch.einsum("hgk,khd->hgd", p, v).reshape(-1, q.shape[-1])


def _exact_attention(st, case):
    Hkv, d = case["Hkv"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for r, L in enumerate(st["seq_lens"].tolist()):
        if not L:
            continue
        q = _turn(st["q"][r:r + 1].double(), st["q_pos"][r:r + 1], case["base"])[0].view(Hkv, -1, d)
        if case["op"] == "prefix":
            j = torch.arange(L, device="cuda")
            blk, first = st["block_tables"][r].long()[j // BS], st["block_starts"][r].long()[j // BS]
            out[r] = _attend(q, _turn(_rows(st, "k", blk, j % BS), first + j % BS, case["base"]),
                             _rows(st, "v", blk, j % BS))
            continue
        for h in range(Hkv):
            sel = st["selected"][r, h].long()
            j = (sel[sel >= 0][:, None] * BS + torch.arange(BS, device="cuda")).view(-1)
            j = j[j < L]
            blk, first = st["block_tables"][r].long()[j // BS], st["block_starts"][r].long()[j // BS]
            one = {n: x[:, h:h + 1] if n[1:] in ("_pool", "_scale") else x for n, x in st.items()}
            k = _turn(_rows(one, "k", blk, j % BS), first + j % BS, case["base"])
            out[r].view(Hkv, -1, d)[h] = _attend(q[h:h + 1], k, _rows(one, "v", blk, j % BS))
    return {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "means":
        return _exact_means(st, case)
    if case["op"] == "scores":
        return _exact_scores(st, case)
    if case["op"] == "select":
        return _exact_select(st, case)
    return _exact_attention(st, case)
