"""Decode calls of more (request, kv head) pairs than the 64 KB of counters hold, on a workspace that other calls use."""

import pytest

from list_util import make_batch
from test_prefix_gpu import env, groups  # noqa: F401  (env: a fixture)

pytestmark = pytest.mark.gpu


def calls(torch, mp, t, rope):
    """(workspace bytes, call(workspace) -> out) of every decode call that cuts pairs, over one batch."""
    B, Hq, d = t["q"].shape
    Hkv, mb, dev = t["Hkv"], t["block_tables"].shape[1], t["q"].device
    a = (t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)
    sel = torch.arange(mb, dtype=torch.int32, device=dev).expand(B, Hkv, mb).contiguous()
    cu = torch.tensor([0, B], dtype=torch.int32, device=dev)
    none = torch.zeros(1, dtype=torch.int32, device=dev)
    bw = torch.zeros(B, Hkv, mb, dtype=torch.bfloat16, device=dev)
    return {
        "attn_decode": (mp.decode_workspace_size(B, Hq, Hkv, d, mb),
                        lambda ws: mp.attn_decode(*a, workspace=ws)[0]),
        "weights": (mp.attn_decode_weights_workspace_size(B, Hq, Hkv, d, mb),
                    lambda ws: mp.attn_decode_weights(*a, bw, workspace=ws)[0]),
        "selected": (mp.attn_decode_selected_workspace_size(B, Hq, Hkv, d, mb),
                     lambda ws: mp.attn_decode_selected(*a, sel, workspace=ws)[0]),
        "prefix": (mp.attn_decode_prefix_workspace_size(B, Hq, Hkv, d, mb, 1, B, 0),
                   lambda ws: mp.attn_decode_prefix(*a, cu, none, max_requests=B, max_prefix_blocks=0, workspace=ws)[0]),
    }


@pytest.mark.parametrize("Hkv", [8, 9])
def test_one_workspace_for_more_than_16384_pairs(env, Hkv):
    """Requests whose counters lie past 64 KB have their lists cut: the same bits on a workspace of zeros, after calls of
    few requests have left their partial results there, and after their own kind."""
    torch, mp, dev = env
    B = 16384 // Hkv + 40
    lens = [5 + r % 20 for r in range(B)]
    for r in (B - 1, B - 7, B - 20, 3):
        lens[r] = 16 * 1200 + r % 16
    big = make_batch(torch, dev, lens, Hkv, Hkv, 64, "bf16", Hkv)
    small = make_batch(torch, dev, [9000, 12000, 800, 7000], 4 * Hkv, Hkv, 64, "bf16", 3)
    rope = mp.rope_table(max(big["max_pos"], small["max_pos"]), 64, big["base"], device=dev)
    many, few = (calls(torch, mp, t, rope) for t in (big, small))
    ws = torch.zeros(max(n for c in (many, few) for n, _ in c.values()), dtype=torch.uint8, device=dev)
    assert B * Hkv > 16384
    for name, (n, call) in many.items():
        want = call(torch.zeros(n, dtype=torch.uint8, device=dev))
        want_few = {}
        for other, (m, dirty) in few.items():
            want_few[other] = dirty(torch.zeros(m, dtype=torch.uint8, device=dev))
            got = dirty(ws)
            assert torch.equal(got, want_few[other]), other
            ws[65536:].fill_(0x11)   # as partial results of any call would
            assert torch.equal(call(ws), want), (name, other)
            assert torch.equal(call(ws), want), (name, "again")
            assert torch.equal(dirty(ws), want_few[other]), (other, "after", name)
            assert not ws[:65536].any()
    assert mp.device_error() == 0


def first(t, n):
    """The first n requests of a batch."""
    rows = ("q", "block_tables", "block_starts", "seq_lens", "q_pos")
    return {k: v[:n].contiguous() if k in rows else v for k, v in t.items()}


def test_a_workspace_of_the_largest_batch_serves_smaller_ones(env):
    """Batches that shrink request by request, as their plans change: a CTA a pair, the prefix kernel's waves."""
    torch, mp, dev = env
    t = make_batch(torch, dev, [3 + r % 30 for r in range(8193)], 8, 8, 64, "bf16", 5)
    rope = mp.rope_table(t["max_pos"], 64, t["base"], device=dev)
    ws = torch.zeros(mp.attn_decode_selected_workspace_size(8193, 8, 8, 64, 40), dtype=torch.uint8, device=dev)
    for n in (8193, 8192, 8100, 75, 1):
        s = first(t, n)
        sel = torch.arange(40, dtype=torch.int32, device=dev).expand(n, 8, 40).contiguous()
        a = (s["q"], s["k_pool"], s["v_pool"], s["block_tables"], s["block_starts"], s["seq_lens"], s["q_pos"], rope, sel)
        assert torch.equal(mp.attn_decode_selected(*a, workspace=ws)[0], mp.attn_decode_selected(*a)[0]), n
    del t, s, a
    t = groups(torch, dev, [3200 + r % 90 for r in range(176)], [0, 176], [200], 128, 8, 128, 5)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    mb = t["block_tables"].shape[1]
    ws = torch.zeros(mp.attn_decode_prefix_workspace_size(176, 128, 8, 128, mb, 1, 176, 200), dtype=torch.uint8, device=dev)
    for n in (176, 175, 160, 159, 100, 33, 9, 2, 1):
        s = first(t, n)
        cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
        a = (s["q"], s["k_pool"], s["v_pool"], s["block_tables"], s["block_starts"], s["seq_lens"], s["q_pos"], rope, cu,
             t["blocks"])
        kw = dict(max_requests=n, max_prefix_blocks=200)
        assert torch.equal(mp.attn_decode_prefix(*a, workspace=ws, **kw)[0], mp.attn_decode_prefix(*a, **kw)[0]), n
    assert mp.device_error() == 0


@pytest.mark.parametrize("Hkv,d", [(8, 64), (7, 128)])
def test_many_pairs_behind_a_prefix_captured(env, Hkv, d):
    """More pairs than counters, that share a prefix, with lists behind it that are cut: captured on a workspace that other
    calls write to, replayed, and eager, each with the bits of a workspace of its own."""
    torch, mp, dev = env
    B, nb = 16384 // Hkv + 30, 40
    own = [1 + r % 2 for r in range(B)]
    for r in (B - 1, B - 5, B - 9, 2):
        own[r] = 1500
    long = make_batch(torch, dev, [16 * n - r % 16 for r, n in enumerate(own)], 2 * Hkv, Hkv, d, "bf16", d)
    front = torch.arange(nb, dtype=torch.int32, device=dev)   # blocks of the longest list, shared by all
    tables = torch.cat([long["block_tables"][2, front.long()].expand(B, nb), long["block_tables"]], 1).contiguous()
    starts = torch.cat([(16 * front).expand(B, nb), long["block_starts"] + 16 * nb], 1).contiguous()
    lens, pos = long["seq_lens"] + 16 * nb, long["q_pos"] + 16 * nb
    rope = mp.rope_table(long["max_pos"] + 16 * nb, d, long["base"], device=dev)
    cu, blocks = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, B], [nb]))
    n = mp.attn_decode_prefix_workspace_size(B, 2 * Hkv, Hkv, d, tables.shape[1], 1, B, nb)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)

    def call(**kw):
        return mp.attn_decode_prefix(long["q"], long["k_pool"], long["v_pool"], tables, starts, lens, pos, rope, cu, blocks,
                                     max_requests=B, max_prefix_blocks=nb, **kw)[0]
    want, out = call(), torch.full_like(long["q"], 7.0)
    whole = mp.attn_decode(long["q"], long["k_pool"], long["v_pool"], tables, starts, lens, pos, rope)[0]
    assert (want - whole).double().norm() <= 5e-3 * whole.double().norm()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, workspace=ws)
    for _ in range(2):
        ws[65536:].fill_(0x11)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not ws[:65536].any()
        ws[65536:].fill_(0x11)
        assert torch.equal(call(workspace=ws), want)
    assert mp.device_error() == 0
