"""The decode over one list of blocks (8-bit cache; bf16 cache with block weights): how the list is shared out, the
range of its operands, and its workspace."""

import numpy as np
import pytest

from cache8_util import Case, check_attention, check_weights, score_error
import workloads as W
from list_util import call, f64, make_batch, reference, workspace_size

pytestmark = pytest.mark.gpu

P_HALF = {"e4m3": 2.0 ** -11, "bf16": 2.0 ** -8}   # rounding of P
COUNTERS = 65536                                     # bytes of the completion counters


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    mp.load()
    mp.device_error(clear=True)
    return torch, mp, torch.device("cuda:0")


def check(torch, t, out, lse, bw, what="", ref=None):
    ref = ref or reference(torch, t)
    d, lens = t["q"].shape[2], t["seq_lens"].tolist()
    check_attention(f64(out), ref, "bf16", d, max(lens), what, p_half=P_HALF[t["kv"]])
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(np.isneginf(f64(lse)), ~fin), what
    # the denominator's terms carry the scores' errors and 2^-11 covers ex2 and the sums
    assert np.all(np.abs(f64(lse)[fin] - ref["lse"][fin]) <= (score_error(ref, "bf16", d) + 2.0 ** -11 + 1e-5)[fin]), what
    if bw is not None:
        check_weights(f64(bw), ref, "bf16", d, lens, 7.0, what)


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,d,top", [(40, 8, 2, 128, 17000), (64, 8, 4, 64, 6000), (97, 14, 2, 128, 4000),
                                            (128, 32, 2, 64, 5000)])
def test_up_to_128_requests_that_fill_the_grid(env, kv, B, Hq, Hkv, d, top):
    """Ragged requests, some without a key, in equal ranges of the list: every CTA finds its pair, whichever warp holds
    it, call after call; the counters are zero again after each."""
    torch, mp, dev = env
    rng = np.random.default_rng(B)
    lens = [int(x) for x in np.where(rng.random(B) < 0.2, 0, rng.integers(1, top, B))]
    lens[-1] = top
    t = make_batch(torch, dev, lens, Hq, Hkv, d, kv, B)
    # parts of up to 64 blocks, one a CTA, would not fit the grid: equal ranges
    grid = torch.cuda.get_device_properties(dev).multi_processor_count * (2 if Hq > 8 * Hkv else 4 if d == 64 else 3)
    assert sum(-(-n // 16) for n in lens) * Hkv // 64 + sum(n > 0 for n in lens) * Hkv > grid
    rope = mp.rope_table(t["max_pos"], d, t["base"], device=dev)
    ws = torch.zeros(workspace_size(mp, t), dtype=torch.uint8, device=dev)
    mb, first = t["block_tables"].shape[1], None
    for i in range(25):
        out = torch.full_like(t["q"], float("nan"))
        lse = torch.full((B, Hq), float("nan"), device=dev)
        bw = torch.full((B, Hkv, mb), 7.0, dtype=torch.bfloat16, device=dev)
        call(mp, torch, t, rope, out, lse, bw, ws)
        assert not ws[:COUNTERS].any(), i
        if first is None:
            first = (out, lse, bw)
            check(torch, t, out, lse, bw)
        assert all(torch.equal(a, b) for a, b in zip(first, (out, lse, bw))), i
    assert mp.device_error() == 0


def run_case(env, c):
    """(out, lse, weights) of a cache8_util.Case over the e4m3 cache."""
    torch, mp, dev = env
    t = c.device(torch, dev)
    B, mb = c.tables.shape
    out = torch.full_like(t["q"], float("nan"))
    lse = torch.full((B, c.Hq), float("nan"), device=dev)
    bw = torch.full((B, c.Hkv, mb), 7.0, dtype=t["q"].dtype, device=dev)
    mp.attn_decode_q8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["block_tables"], t["block_starts"],
                      t["seq_lens"], t["q_pos"], mp.rope_table(c.max_pos, c.d, c.base, device=dev), out=out, lse=lse,
                      block_weights=bw)
    torch.cuda.synchronize()
    return out, lse, bw


def check_case(c, got, what=""):
    """Errors against float64; outputs of any size: the part of the bound that is absolute is far below them."""
    out, lse, bw = got
    ref = c.reference()
    check_attention(f64(out), ref, c.dtype, c.d, max(c.lens), what)
    assert np.all(np.abs(f64(lse) - ref["lse"]) <= score_error(ref, c.dtype, c.d) + 2.0 ** -11 + 1e-5), what
    check_weights(f64(bw), ref, c.dtype, c.d, c.lens, 7.0, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 2, 128), (16, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("log", [-22, -34, -60])
def test_blocks_of_zero_values_among_small_scales(env, dtype, Hq, Hkv, d, log):
    """A value scale of zero takes no precision from blocks whose scales are small: bytes near 2^2 times 2^-22 to 2^-60."""
    c = Case(70, (400, 90, 16), Hq, Hkv, d, dtype, share=False)
    c.scale[1] = np.where(np.isnan(c.scale[1]), np.nan, 2.0 ** log)
    for r, n in enumerate((25, 6, 0)):
        c.scale[1][c.tables[r, :n:3]] = 0.0   # every warp (each takes every fourth or eighth block) has both kinds
    got = run_case(env, c)
    assert np.all(f64(got[0])[2] != 0)
    check_case(c, got, f"{dtype} {log}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128), (16, 1, 64)])
@pytest.mark.parametrize("log", [-99, -105, -118, -130, 60])
def test_value_scales_of_any_exponent(env, dtype, Hq, Hkv, d, log):
    """The caller's own scales reach down to fp32's subnormals, where the outputs still are numbers of their type."""
    c = Case(71, (3000, 90, 16), Hq, Hkv, d, dtype, share=False)
    c.scale[1] = np.where(np.isnan(c.scale[1]), np.nan, 2.0 ** log)
    out = f64(run_case(env, c)[0])
    ref = c.reference()
    eps = float(np.median(score_error(ref, dtype, d)))
    # the output's rounding (relative to the largest where it is subnormal) and the scores' typical error
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
    for r in range(3):
        assert np.linalg.norm(out[r] - ref["out"][r]) <= (half + 2 * eps) * np.linalg.norm(ref["out"][r])


def test_one_workspace_for_every_decode_call(env):
    """A zeroed workspace serves attn_decode, its prerotated form, attn_mixed and the calls of one list in any order:
    each result is that of the same call on a fresh workspace, and the counters stay zero."""
    torch, mp, dev = env
    few = make_batch(torch, dev, [5000, 17, 9000], 16, 2, 128, "bf16", 5)          # few pairs, many splits
    many = [make_batch(torch, dev, [900 + 7 * i for i in range(90)], 8, 2, 128, kv, 6) for kv in ("bf16", "e4m3")]
    ropes = {id(t): mp.rope_table(t["max_pos"], 128, t["base"], device=dev) for t in (few, *many)}

    def plain(t, ws, prerotated=False):
        a = (t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"])
        f = mp.attn_decode_prerotated if prerotated else mp.attn_decode
        return f(*a, *(() if prerotated else (ropes[id(t)],)), workspace=ws)[:1]

    def listed(t, ws):
        B, Hq, _ = t["q"].shape
        out, bw = torch.empty_like(t["q"]), torch.zeros(B, t["Hkv"], t["block_tables"].shape[1], dtype=torch.bfloat16,
                                                        device=dev)
        call(mp, torch, t, ropes[id(t)], out, None, bw, ws)
        return out, bw

    def mixed(t, ws):
        i32 = dict(dtype=torch.int32, device=dev)
        p = dict(q=t["q"][:1], cu_q_lens=torch.tensor([0, 1], **i32), q_pos=t["q_pos"][:1],
                 block_tables=t["block_tables"][:1], block_starts=t["block_starts"][:1], kv_lens=t["seq_lens"][:1],
                 max_q_len=1)
        dd = {k: t[k] for k in ("q", "block_tables", "block_starts", "seq_lens", "q_pos")}
        return mp.attn_mixed(p, dd, t["k_pool"], t["v_pool"], ropes[id(t)], workspace=ws)[::2]
    calls = [lambda ws: plain(few, ws), lambda ws: listed(many[0], ws), lambda ws: plain(few, ws, True),
             lambda ws: listed(many[1], ws), lambda ws: mixed(few, ws), lambda ws: plain(many[0], ws),
             lambda ws: listed(few, ws)]
    n = max(max(workspace_size(mp, t), mp.decode_workspace_size(t["q"].shape[0], t["q"].shape[1], 2, 128,
                                                                t["block_tables"].shape[1])) for t in (few, *many))
    alone = [f(torch.zeros(n, dtype=torch.uint8, device=dev)) for f in calls]
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    for i in (0, 1, 2, 3, 4, 5, 6, 5, 4, 3, 2, 1, 0, 6, 3, 0, 3):
        got = calls[i](ws)
        assert all(torch.equal(a, b) for a, b in zip(got, alone[i])), i
        assert not ws[:COUNTERS].any(), i
    assert mp.device_error() == 0


def decode_weights(env, t):
    torch, mp, dev = env
    B, Hq, d = t["q"].shape
    out = torch.full_like(t["q"], float("nan"))
    lse = torch.full((B, Hq), float("nan"), device=dev)
    bw = torch.full((B, t["Hkv"], t["block_tables"].shape[1]), 7.0, dtype=torch.bfloat16, device=dev)
    call(mp, torch, t, mp.rope_table(t["max_pos"], d, t["base"], device=dev), out, lse, bw, None)
    torch.cuda.synchronize()
    return out, lse, bw


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 1, 128), (32, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("log", [17, 100, 117, -12, -20, -45, -110])
def test_bf16_keys_of_any_size(env, Hq, Hkv, d, log):
    """Keys far outside fp16's range against queries that bring the scores back, in one kv head; the others' keys as
    they come.  Powers of two, so the operands are the same numbers."""
    torch, mp, dev = env
    t = make_batch(torch, dev, [700, 33, 1, 200], Hq, Hkv, d, "bf16", 80)
    G = Hq // Hkv
    t["k_pool"][:, 0] *= 2.0 ** log
    t["q"][:, :G] *= 2.0 ** -log
    check(torch, t, *decode_weights(env, t), f"2^{log}")


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 1, 128), (32, 2, 128)])
def test_bf16_keys_of_sizes_that_differ_within_a_block(env, Hq, Hkv, d):
    """Rows between 2^-30 and 2^-14 of one block, rows of zeros, quarters of zeros, and pairs near 6e4 whose rotation
    leaves fp16; slots past the lengths hold huge values and infinities."""
    torch, mp, dev = env
    lens = [700, 33, 1, 200]
    t = make_batch(torch, dev, lens, Hq, Hkv, d, "bf16", 81)
    g = torch.Generator(device=dev).manual_seed(3)
    e = torch.randint(-30, -13, t["k_pool"].shape[:3], generator=g, device=dev)
    t["k_pool"] *= torch.exp2(e)[..., None].bfloat16()
    t["k_pool"][::3, :, 5] = 0
    t["k_pool"][::2, :, :, :d // 8] = 0
    t["q"] *= 2.0 ** 16
    for r, n in enumerate(lens):
        if n % 16:
            t["k_pool"][int(t["block_tables"][r, n // 16]), :, n % 16:] = float("inf") if r & 1 else 3e38
    check(torch, t, *decode_weights(env, t), "small")
    t = make_batch(torch, dev, lens, Hq, Hkv, d, "bf16", 82)
    t["k_pool"] = (t["k_pool"].float() * 16000).clamp(-6.4e4, 6.4e4).bfloat16()
    t["q"] *= 2.0 ** -14
    check(torch, t, *decode_weights(env, t), "large")
    assert mp.device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64), (16, 1, 64)])
def test_blocks_that_start_before_the_table(env, kv, Hq, Hkv, d):
    """Slots before position 0 are masked; where the query is so far on that no table row holds the angle to the
    block's start, the whole block is.  Flagged either way."""
    torch, mp, dev = env
    for near in (True, False):
        t = make_batch(torch, dev, [200, 64], Hq, Hkv, d, kv, 95)
        t["block_starts"][0, 3] = -5
        mp.device_error(clear=True)
        t["q_pos"][0] = t["max_pos"] - (6 if near else 1)   # distance to the block's start: max_pos - 1 or + 4
        B, mb = t["block_tables"].shape
        out, lse = torch.empty_like(t["q"]), torch.empty(B, Hq, device=dev)
        bw = torch.full((B, Hkv, mb), 7.0, dtype=torch.bfloat16, device=dev)
        call(mp, torch, t, mp.rope_table(t["max_pos"], d, t["base"], device=dev), out, lse, bw, None)
        torch.cuda.synchronize()
        assert mp.device_error(clear=True) == 2
        if not near:
            t["block_tables"][0, 3] = -1    # for the reference
        check(torch, t, out, lse, bw, str(near))
        assert near or (bw[0, :, 3] == 0).all()
