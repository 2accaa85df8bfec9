"""Prefill while other kernels fill the device: its warps are held up where an idle device never holds them."""

import pytest

from list_util import make_batch

pytestmark = pytest.mark.gpu


def test_prefill_beside_other_kernels_ends_and_repeats_bit_for_bit():
    """The last products' wait: a softmax warp that comes to it late (its code evicted by kernels beside it) finds the
    barrier of every P V product two phases on, where that barrier's parity says "not yet" for good.  500 prefills of a
    few key tiles with decode kernels of other shapes on two other streams."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    dev = torch.device("cuda:0")
    mp.device_error(clear=True)
    lens = [4000, 900, 333, 2500]
    t = make_batch(torch, dev, lens, 16, 2, 128, "bf16", 3)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    g = torch.Generator(device=dev).manual_seed(4)
    ql = 60
    cu = torch.arange(0, ql * 4 + 1, ql, dtype=torch.int32, device=dev)
    q = torch.randn(ql * 4, 16, 128, generator=g, device=dev).bfloat16()
    j = torch.cat([torch.arange(n - ql, n, device=dev) for n in lens])
    row = torch.arange(4, device=dev).repeat_interleave(ql)
    pos = (t["block_starts"].long()[row, j // 16] + j % 16).int()

    def prefill(out):
        mp.attn_prefill(q, cu, pos, t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"], rope, ql,
                        out=out)
    want = torch.empty_like(q)
    prefill(want)
    torch.cuda.synchronize()
    load = [make_batch(torch, dev, [700 + 13 * i for i in range(64)], *h, kv, 5)
            for h, kv in (((8, 2, 64), "e4m3"), ((28, 4, 128), "bf16"))]
    tables = [mp.rope_table(b["max_pos"], b["q"].shape[2], b["base"], device=dev) for b in load]
    side = [torch.cuda.Stream() for _ in load]

    def beside(i):
        b = load[i]
        a = (b["block_tables"], b["block_starts"], b["seq_lens"], b["q_pos"], tables[i])
        if b["kv"] == "e4m3":
            mp.attn_decode_q8(b["q"], b["k_pool"], b["v_pool"], b["k_scale"], b["v_scale"], *a, stream=side[i])
        else:
            mp.attn_decode(b["q"], b["k_pool"], b["v_pool"], *a, stream=side[i])
    outs = [torch.full_like(q, float("nan")) for _ in range(25)]
    for step in range(20):
        for out in outs:
            out.fill_(float("nan"))
            for i in range(2):
                beside(i)
            prefill(out)
        torch.cuda.synchronize()
        assert mp.device_error() == 0, step
        assert all(torch.equal(out, want) for out in outs), step
