"""Capturing the 8-bit cache's calls into a graph runs nothing; replaying it runs them."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def bits(torch, x):
    """A copy of a tensor's bytes: NaN equals itself."""
    return x.contiguous().view(torch.uint8).clone()


def test_capture_changes_no_bit_and_replay_equals_the_calls():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    B, Hq, Hkv, d, mb, nb = 3, 8, 2, 128, 6, 20

    def i32(a):
        return torch.tensor(a, dtype=torch.int32, device=dev)

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev).bfloat16()
    n = [70, 33, 16]
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    fixed = dict(k=randn(cu[-1], Hkv, d), v=randn(cu[-1], Hkv, d), q=randn(cu[-1], Hq, d), q1=randn(B, Hq, d), cu=i32(cu),
                 start=i32([0] * B), q_pos=i32([i for m in n for i in range(m)]), pos=i32(n),
                 order=torch.randperm(nb, generator=g, device=dev)[:B * mb].view(B, mb).int(),
                 rope=mp.rope_table(256, d, 1e4, device=dev))
    e4m3 = torch.float8_e4m3fn

    def fresh():
        return dict(kp=torch.full((nb, Hkv, 16, d), 0x7f, dtype=torch.uint8, device=dev).view(e4m3),
                    vp=torch.full((nb, Hkv, 16, d), 0xff, dtype=torch.uint8, device=dev).view(e4m3),
                    ks=torch.full((nb, Hkv), float("nan"), device=dev), vs=torch.full((nb, Hkv), float("nan"), device=dev),
                    tables=fixed["order"].clone(), starts=i32([[16 * b for b in range(mb)]] * B), lens=i32(n),
                    scores=torch.full((B, mb), 0.5, device=dev),
                    bw=torch.full((B, Hkv, mb), float("nan"), device=dev).bfloat16(),
                    out=torch.full((cu[-1], Hq, d), float("nan"), device=dev).bfloat16(),
                    o1=torch.full((B, Hq, d), float("nan"), device=dev).bfloat16(),
                    lse=torch.full((B, Hq), float("nan"), device=dev),
                    ws=torch.zeros(mp.attn_decode_q8_workspace_size(B, Hq, Hkv, d, mb), dtype=torch.uint8, device=dev),
                    wp=torch.zeros(mp.attn_prefill_q8_workspace_size(B, Hq, Hkv, d, max(n), mb), dtype=torch.uint8,
                                   device=dev))

    def step(s):
        f = fixed
        cache = (s["kp"], s["vp"], s["ks"], s["vs"])
        mp.kv_append_q8(f["k"], f["v"], f["cu"], f["start"], s["tables"], *cache, max_new_len=max(n))
        mp.attn_prefill_q8(f["q"], f["cu"], f["q_pos"], *cache, s["tables"], s["starts"], s["lens"], f["rope"], max(n),
                           out=s["out"], workspace=s["wp"])
        mp.attn_decode_q8(f["q1"], *cache, s["tables"], s["starts"], s["lens"], f["pos"], f["rope"], out=s["o1"],
                          lse=s["lse"], block_weights=s["bw"], workspace=s["ws"])
        mp.kv_evict(s["scores"], s["tables"], s["starts"], s["lens"], 2, block_weights=s["bw"], decay=0.9, inplace=True)
    want = fresh()
    step(want)
    s = fresh()
    before = {k: bits(torch, x) for k, x in s.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    torch.cuda.synchronize()
    for k, x in s.items():
        assert torch.equal(bits(torch, x), before[k]), f"capture wrote {k}"
    graph.replay()
    torch.cuda.synchronize()
    for k, x in s.items():
        if k not in ("ws", "wp"):
            assert torch.equal(bits(torch, x), bits(torch, want[k])), k
    assert not torch.equal(bits(torch, s["ks"]), before["ks"]) and (s["lens"] == i32([16 + 6, 16 + 1, 16])).all()
    assert mp.device_error() == 0
