"""Decode and mixed calls on a side stream while the current one is busy: their workspace is theirs."""

import pytest

from list_util import make_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["decode", "prerotated", "mixed"])
def test_workspace_is_cleared_on_the_stream_of_the_call(call):
    """The counters that a call clears for itself are zero when its kernel starts, not when the current stream gets to
    it: memory that held something else before, and a current stream that is 50 ms behind."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    dev = torch.device("cuda:0")
    t = make_batch(torch, dev, [5000, 17, 9000], 16, 2, 128, "bf16", 5)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    a = (t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"])
    p = dict(q=t["q"][:1], cu_q_lens=torch.tensor([0, 1], dtype=torch.int32, device=dev), q_pos=t["q_pos"][:1],
             block_tables=t["block_tables"][:1], block_starts=t["block_starts"][:1], kv_lens=t["seq_lens"][:1],
             max_q_len=1)
    dec = {k: t[k] for k in ("q", "block_tables", "block_starts", "seq_lens", "q_pos")}

    def run(**kw):
        if call == "decode":
            return mp.attn_decode(*a, rope, **kw)[0]
        if call == "prerotated":
            return mp.attn_decode_prerotated(*a, **kw)[0]
        return mp.attn_mixed(p, dict(dec), t["k_pool"], t["v_pool"], rope, **kw)[2]
    want = run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = mp.decode_workspace_size(3, 16, 2, 128, t["block_tables"].shape[1])
    assert n > 0
    for _ in range(3):
        torch.cuda.empty_cache()
        for s in (torch.cuda.current_stream(), side):
            with torch.cuda.stream(s):
                junk = torch.full((n,), 0x11, dtype=torch.uint8, device=dev)   # the next workspace of that stream
                del junk
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)   # about 50 ms
        got = run(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert mp.device_error() == 0
