"""Decode over selected blocks and behind prefixes where a few lists are much longer than the others and there are about as
many (request, kv head) pairs as CTAs."""

import numpy as np
import pytest

from select_util import batch
from test_prefix_gpu import check as check_prefix, env, i32, run as run_prefix  # noqa: F401  (env: a fixture)
from test_select_gpu import check, run

pytestmark = pytest.mark.gpu


def every_block(torch, t, Hkv):
    S = t["block_tables"].shape[1]
    return torch.arange(S, dtype=torch.int32, device=t["q"].device).expand(len(t["q"]), Hkv, S).contiguous()


# pairs just below the CTAs at once (456 at head dim 128, 608 at 64; 304 above 8 heads a kv head), few CTAs to spare and
# many, and odd kv heads of which each has a CTA
@pytest.mark.parametrize("kv,Hq,Hkv,d,B,long", [
    ("bf16", 8, 8, 128, 56, (5000,)), ("e4m3", 16, 8, 128, 56, (5000,)), ("bf16", 8, 8, 64, 75, (5000, 4000)),
    ("e4m3", 3, 1, 64, 600, (9000,)), ("bf16", 16, 1, 128, 300, (3000,)), ("bf16", 4, 2, 128, 150, (2000, 6000, 700)),
    ("bf16", 1, 1, 128, 1000, (9000, 30)), ("e4m3", 3, 3, 64, 450, (7000,))])
def test_few_long_lists_among_short_ones(env, kv, Hq, Hkv, d, B, long):
    """The same bits twice on one workspace, whose counters end at zero, and float64's result."""
    torch, mp, dev = env
    lens = [100 + 37 * r % 400 for r in range(B)]
    for i, n in enumerate(long):
        lens[(B - 1) * i // max(1, len(long) - 1)] = n
    t = batch(torch, dev, lens, Hq, Hkv, d, kv, B + d)
    sel = every_block(torch, t, Hkv)
    ws = torch.zeros(mp.attn_decode_selected_workspace_size(B, Hq, Hkv, d, sel.shape[2]), dtype=torch.uint8, device=dev)
    got = [run(env, t, sel, workspace=ws) for _ in range(2)]
    assert not ws[:65536].any()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    check(env, t, sel, got[0])
    if kv == "bf16":   # the same lists as the keys behind a prefix of no block
        t.update(cu=i32(torch, dev, [0, B]), blocks=i32(torch, dev, [0]))
        check_prefix(env, t, run_prefix(env, t))
    assert mp.device_error() == 0


def test_a_long_list_does_not_wait_for_one_cta(env):
    """8192 blocks among 55 requests of 64 take no more than 4 times as long as the same keys spread evenly (with one
    CTA for each of the long lists, 10 times)."""
    torch, mp, dev = env

    def time(lens):
        t = batch(torch, dev, [16 * n for n in lens], 32, 8, 128, "bf16", 3)
        sel, rope = every_block(torch, t, 8), mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
        ws = torch.zeros(mp.attn_decode_selected_workspace_size(56, 32, 8, 128, sel.shape[2]), dtype=torch.uint8, device=dev)
        best = []
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            mp.attn_decode_selected(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"],
                                    t["q_pos"], rope, sel, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        return float(np.min(best))
    assert time([8192] + [64] * 55) <= 4 * time([209] * 56)
