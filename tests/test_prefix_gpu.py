"""Decode of batches whose requests share prefixes on the GPU against float64."""

import numpy as np
import pytest

from cache8_util import check_attention, score_error
from list_util import f64
from select_util import batch, reference

pytestmark = pytest.mark.gpu


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


def i32(torch, dev, a):
    return torch.tensor(np.asarray(a).tolist(), dtype=torch.int32, device=dev)


def groups(torch, dev, lens, cu, blocks, Hq, Hkv, d, seed):
    """A batch of those lengths in which requests cu[p] .. cu[p + 1] - 1 share their first blocks[p] blocks."""
    t = batch(torch, dev, lens, Hq, Hkv, d, "bf16", seed)
    for p, nb in enumerate(blocks):
        rows = [r for r in range(cu[p], cu[p + 1]) if lens[r] >= 16 * nb]
        for r in rows[1:]:
            for x in ("block_tables", "block_starts"):
                t[x][r, :nb] = t[x][rows[0], :nb]
            # the rest follows at this request's own gaps
            t["block_starts"][r, nb:] += 64
    last = (t["seq_lens"] - 1).clamp(min=0)
    t["q_pos"] = (t["block_starts"].long().gather(1, (last // 16).long()[:, None])[:, 0] + last % 16 + 1).int()
    t["max_pos"] = int(t["block_starts"].max()) + 80
    t.update(cu=i32(torch, dev, cu), blocks=i32(torch, dev, blocks))
    return t


WIDE = 10 ** 6   # a bound of the prefixes with which these small batches share (the exact one says that it does not pay)


def run(env, t, rope=None, **kw):
    torch, mp, dev = env
    kw.setdefault("max_prefix_blocks", WIDE)
    B, Hq, d = t["q"].shape
    rope = rope or mp.rope_table(t["max_pos"], d, t["base"], device=dev)
    lse = torch.full((B, Hq), float("nan"), device=dev)
    out = torch.full_like(t["q"], float("nan"))
    got = mp.attn_decode_prefix(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"],
                                t["q_pos"], rope, t["cu"], t["blocks"], out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    torch.cuda.synchronize()
    return out, lse


def all_keys(torch, t):
    return lambda r, g: torch.arange(int(t["seq_lens"][r]), device=t["q"].device)


def check(env, t, got, what="", scale=None):
    torch = env[0]
    out, lse = got
    ref = reference(torch, t, all_keys(torch, t), scale)
    d = t["q"].shape[2]
    check_attention(f64(out), ref, "bf16", d, int(t["seq_lens"].max()), what, p_half=2.0 ** -8)
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(np.isneginf(f64(lse)), ~fin), what
    tol = score_error(ref, "bf16", d) + 2.0 ** -11 + 1e-5
    assert np.all(np.abs(f64(lse)[fin] - ref["lse"][fin]) <= tol[fin]), what


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 8, 64), (15, 3, 64), (32, 2, 64), (8, 2, 128), (3, 3, 128),
                                      (14, 2, 128), (16, 2, 128), (9, 1, 128), (32, 2, 128)])
def test_one_prefix(env, Hq, Hkv, d):
    """Ragged requests behind one prefix; one ends exactly with it."""
    torch, mp, dev = env
    for nb in (1, 5, 13, 40):
        lens = [16 * nb + x for x in (1, 0, 37, 500, 16, 3, 64, 250, 99)]
        t = groups(torch, dev, lens, [0, 9], [nb], Hq, Hkv, d, Hq * d + nb)
        check(env, t, run(env, t), f"{Hq}/{Hkv} d{d} {nb}")
    assert mp.device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (14, 2, 128), (32, 2, 128)])
def test_groups_of_any_kind(env, Hq, Hkv, d):
    """Several prefixes of different lengths, a group of one, an empty group, a prefix of no block, requests in front of,
    between... and behind the groups, rows without a key, rows shorter than their prefix."""
    torch, mp, dev = env
    lens = [70, 300, 0, 500, 340, 31, 64, 64, 900, 901, 17, 0, 230, 1200, 1]
    t = groups(torch, dev, lens, [1, 6, 6, 8, 10, 11, 12], [18, 3, 4, 55, 1, 2], Hq, Hkv, d, 5)
    check(env, t, run(env, t), f"{Hq}/{Hkv} d{d}")
    t["cu"], t["blocks"] = i32(torch, dev, [0]), i32(torch, dev, [])       # no prefix at all
    check(env, t, run(env, t), "none")
    t["cu"], t["blocks"] = i32(torch, dev, [0, len(lens)]), i32(torch, dev, [0])
    check(env, t, run(env, t), "no block")
    assert mp.device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,d,B,nb", [(8, 2, 128, 150, 200), (16, 1, 128, 40, 700), (8, 2, 64, 150, 200),
                                           (28, 4, 128, 64, 97), (16, 1, 64, 33, 333), (4, 4, 128, 300, 30),
                                           (4, 4, 128, 300, 10), (8, 4, 64, 320, 6)])
def test_many_requests_and_long_prefixes(env, Hq, Hkv, d, B, nb):
    """More rows than a tile pair, prefixes of many tiles cut into parts: the same bits call after call on one
    workspace, whose counters end at zero; planning bounds larger than what comes change nothing."""
    torch, mp, dev = env
    rng = np.random.default_rng(B)
    lens = [16 * nb + int(x) for x in rng.integers(0, 120, B)]
    lens[B // 2] = 0
    t = groups(torch, dev, lens, [0, B], [nb], Hq, Hkv, d, B)
    mb = t["block_tables"].shape[1]
    n = max(mp.attn_decode_prefix_workspace_size(B, Hq, Hkv, d, mb, 1, B + x, y) for x, y in ((0, nb), (50, nb + WIDE)))
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    first = None
    check(env, t, run(env, t, workspace=ws, max_requests=B, max_prefix_blocks=nb), "exact bounds")
    for i in range(6):
        got = run(env, t, workspace=ws, max_requests=B, max_prefix_blocks=nb + WIDE)
        assert not ws[:65536].any(), i
        if first is None:
            first = got
            check(env, t, got)
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1]), i
    check(env, t, run(env, t, workspace=ws, max_requests=B + 50, max_prefix_blocks=nb + WIDE), "wide bounds")
    assert mp.device_error() == 0


def test_matches_the_decode_that_shares_nothing(env):
    """The same batch through attn_decode: both within the bf16 tolerances of the same reference."""
    torch, mp, dev = env
    lens = [1600 + 50 * i for i in range(20)]
    t = groups(torch, dev, lens, [0, 12, 20], [100, 70], 8, 2, 128, 3)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    a = (t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)
    want = f64(mp.attn_decode(*a)[0])
    got = f64(run(env, t, rope)[0])
    assert np.abs(got - want).max() <= 2e-2 and np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)


def test_what_masked_slots_hold_does_not_show(env):
    """NaN and infinities behind the lengths, in blocks of no request, and under bad ids and positions (flagged)."""
    torch, mp, dev = env
    for d in (64, 128):
        lens = [330, 400, 333, 0, 500]
        t = groups(torch, dev, lens, [0, 5], [20], 8, 2, d, 9)
        bad = torch.ones(t["k_pool"].shape[0], dtype=torch.bool, device=dev)
        bad[t["block_tables"][t["block_tables"] >= 0].long()] = False
        for x, v in (("k_pool", float("inf")), ("v_pool", float("nan"))):
            t[x][bad] = v
            for r, n in enumerate(lens):
                if n % 16:
                    t[x][int(t["block_tables"][r, n // 16]), :, n % 16:] = v
        check(env, t, run(env, t), f"d{d}")
        assert mp.device_error() == 0
        t["block_tables"][:, 3] = -7                                  # in the prefix, in every row
        t["block_tables"][1, 22] = t["k_pool"].shape[0]
        got = run(env, t)
        assert mp.device_error(clear=True) == 1
        check(env, t, got, f"ids d{d}")
        t["block_starts"][:, 5] = t["max_pos"] + 3
        got = run(env, t)
        assert mp.device_error(clear=True) == 1 | 2
        check(env, t, got, f"positions d{d}")


def test_nan_passes_on_to_the_rows_that_attend_to_it(env):
    torch, mp, dev = env
    for d in (64, 128):
        t = groups(torch, dev, [170, 200, 190, 60], [0, 3], [10], 4, 2, d, 13)
        t["v_pool"][int(t["block_tables"][0, 4]), 1, 3, 5] = float("nan")     # in the prefix
        t["v_pool"][int(t["block_tables"][1, 11]), 0, 0, 7] = float("nan")    # request 1's own
        out = f64(run(env, t)[0])
        nan = np.isnan(out)
        assert np.all(nan[:3, 2:, 5]) and np.all(nan[1, :2, 7])
        nan[:3, 2:, 5] = False
        nan[1, :2, 7] = False
        assert not nan.any()


def test_bad_group_data_is_flagged(env):
    """Groups outside the batch and prefixes longer than the tables set the length bit; nothing is read out of range,
    and requests that such a group does not hold are computed."""
    torch, mp, dev = env
    t = groups(torch, dev, [400, 420, 440, 460], [0, 2, 4], [10, 12], 8, 2, 128, 17)
    want = run(env, t)[0]
    for cu, blocks in (([0, 2, 9], [10, 12]), ([0, 2, 4], [10, 10 ** 6]), ([0, 2, 1], [10, 12]), ([0, 2, 4], [10, -3])):
        t["cu"], t["blocks"] = i32(torch, dev, cu), i32(torch, dev, blocks)
        got = run(env, t, max_requests=2)[0]
        assert mp.device_error(clear=True) == 4, (cu, blocks)
        assert torch.equal(got[:2], want[:2])


@pytest.mark.parametrize("d", [64, 128])
def test_groups_beyond_the_planning_bounds(env, d):
    """More requests or longer prefixes than the call was told: flagged, and the requests share nothing."""
    torch, mp, dev = env
    t = groups(torch, dev, [700, 720, 740, 660, 500, 450], [0, 3, 6], [30, 20], 8, 2, d, 31)
    for bounds, bad in ((dict(max_requests=3, max_prefix_blocks=29), True), (dict(max_requests=2, max_prefix_blocks=30), True),
                        (dict(max_requests=3, max_prefix_blocks=1), True), (dict(max_requests=0, max_prefix_blocks=0), True),
                        (dict(max_requests=1000, max_prefix_blocks=1000), False), (dict(max_requests=2), True),
                        (dict(max_requests=3), False), (dict(max_requests=1), True)):
        got = run(env, t, **bounds)
        assert mp.device_error(clear=True) == (4 if bad else 0), bounds
        check(env, t, got, f"d{d} {bounds}")


@pytest.mark.parametrize("d", [64, 128])
def test_one_group_beyond_the_bounds_another_within(env, d):
    """The first group's prefix is longer than the call was told: flagged, its requests read their own keys; the second
    group shares (the bounds say that it pays)."""
    torch, mp, dev = env
    t = groups(torch, dev, [16 * 60 + 3 * i for i in range(100)], [0, 50, 100], [58, 40], 16, 8, d, 37)
    got = run(env, t, max_requests=50, max_prefix_blocks=50)
    assert mp.device_error(clear=True) == 4
    check(env, t, got, f"d{d}")


def test_more_groups_and_requests_than_are_staged(env):
    """Hundreds of groups, thousands of requests, some without a key."""
    torch, mp, dev = env
    rng = np.random.default_rng(12)
    for d, B, P in ((64, 2100, 700), (128, 600, 300)):
        cu = [0] + sorted(int(x) for x in rng.integers(0, B + 1, P))
        blocks = [int(x) for x in rng.integers(0, 6, P)]
        lens = [0] * B
        for p in range(P):
            for r in range(cu[p], cu[p + 1]):
                lens[r] = int(rng.integers(0, 16)) * int(rng.integers(0, 2)) + 16 * (blocks[p] - int(rng.random() < 0.1))
        lens = [max(0, x) for x in lens]
        t = groups(torch, dev, lens, cu, blocks, 2, 1, d, B)
        check(env, t, run(env, t), f"{B} requests")
    assert mp.device_error() == 0


def test_calls_on_two_streams_at_once(env):
    """Calls of both head dims on two streams, each with its workspace: the bits of the calls alone."""
    torch, mp, dev = env
    cases = [groups(torch, dev, [16 * nb + 30 * i for i in range(n)], [0, n], [nb], 8, 2, d, nb)
             for nb, n, d in ((90, 40, 128), (60, 30, 64))]
    ropes = [mp.rope_table(t["max_pos"], t["q"].shape[2], t["base"], device=dev) for t in cases]
    streams = [torch.cuda.Stream() for _ in cases]

    def call(i, **kw):
        t = cases[i]
        return mp.attn_decode_prefix(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"],
                                     t["seq_lens"], t["q_pos"], ropes[i], t["cu"], t["blocks"], max_requests=40,
                                     max_prefix_blocks=WIDE, **kw)[0]
    want = [call(i).clone() for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(call(i, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i]), i
    assert mp.device_error() == 0


def test_captured_and_on_a_side_stream(env):
    """Capture runs nothing, replay equals the call, two captured graphs share a workspace one after the other, and a
    call on a side stream allocates and clears its own while the current one is behind."""
    torch, mp, dev = env
    cases = [groups(torch, dev, [16 * nb + 40 * i for i in range(9)], [0, 9], [nb], 8, 2, d, nb)
             for nb, d in ((60, 128), (25, 64))]
    ropes = [mp.rope_table(t["max_pos"], t["q"].shape[2], t["base"], device=dev) for t in cases]
    want = [run(env, t, rope)[0] for t, rope in zip(cases, ropes)]
    n = max(mp.attn_decode_prefix_workspace_size(9, 8, 2, t["q"].shape[2], t["block_tables"].shape[1], 1, 9, WIDE)
            for t in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    outs = [torch.full_like(t["q"], 7.0) for t in cases]

    def call(i, **kw):
        t = cases[i]
        return mp.attn_decode_prefix(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"],
                                     t["seq_lens"], t["q_pos"], ropes[i], t["cu"], t["blocks"], max_requests=9,
                                     max_prefix_blocks=WIDE, **kw)[0]
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, out=outs[i], workspace=ws)
        torch.cuda.synchronize()
        assert (outs[i] == 7.0).all()
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], call(i)) and not ws[:65536].any()
        assert np.linalg.norm(f64(outs[i] - want[i])) <= 5e-3 * np.linalg.norm(f64(want[i]))
    side = torch.cuda.Stream()
    for i in range(2):
        once = call(i).clone()
        for _ in range(2):
            torch.cuda.empty_cache()
            for s in (torch.cuda.current_stream(), side):
                with torch.cuda.stream(s):
                    junk = torch.full((n,), 0x11, dtype=torch.uint8, device=dev)
                    del junk
            torch.cuda.synchronize()
            torch.cuda._sleep(100_000_000)   # about 50 ms
            got = call(i, stream=side)
            side.synchronize()
            assert torch.equal(got, once)
            torch.cuda.synchronize()
    assert mp.device_error() == 0


def test_many_requests_captured(env):
    """A batch of many requests (its join runs as a kernel of its own) and a small one, captured over one workspace and
    replayed in turn, with other batches in the same buffers between: requests that end, lose their prefix, or whose
    group grows; the same bits as eager calls."""
    torch, mp, dev = env
    rng = np.random.default_rng(8)
    for d, Hkv in ((128, 4), (64, 8)):
        lens = [16 * 30 + int(x) for x in rng.integers(0, 200, 150)] + [0, 0] + [int(x) for x in rng.integers(1, 90, 148)]
        big = groups(torch, dev, lens, [0, 100, 150], [30, 11], 2 * Hkv, Hkv, d, d)
        small = groups(torch, dev, [700, 690, 31, 800], [0, 4], [40], 2 * Hkv, Hkv, d, d + 1)
        rope = mp.rope_table(max(big["max_pos"], small["max_pos"]), d, big["base"], device=dev)
        bounds = dict(max_requests=160, max_prefix_blocks=45)
        n = max(mp.attn_decode_prefix_workspace_size(len(t["seq_lens"]), 2 * Hkv, Hkv, d, t["block_tables"].shape[1],
                                                     len(t["blocks"]), 160, 45) for t in (big, small))
        ws = torch.zeros(n, dtype=torch.uint8, device=dev)

        def call(t, **kw):
            return mp.attn_decode_prefix(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"],
                                         t["seq_lens"], t["q_pos"], rope, t["cu"], t["blocks"], **bounds, **kw)[0]
        graphs, outs = [], [torch.full_like(t["q"], 7.0) for t in (big, small)]
        for t, out in zip((big, small), outs):
            call(t, workspace=ws)
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                call(t, out=out, workspace=ws)
        for step in range(4):
            if step == 1:
                big["seq_lens"][3] = 0
                big["seq_lens"][7] = 16 * 30 - 5       # shorter than the prefix
                big["q_pos"][7] = big["block_starts"][7, 29] + 11
            if step == 2:
                big["blocks"].copy_(i32(torch, dev, [0, 11]))
            if step == 3:
                big["blocks"].copy_(i32(torch, dev, [11, 11]))
                big["cu"].copy_(i32(torch, dev, [0, 99, 99]))
            for i in (0, 1, 0):
                outs[i].fill_(7.0)
                graphs[i].replay()
            torch.cuda.synchronize()
            assert not ws[:65536].any()
            for t, out in zip((big, small), outs):
                lse = torch.empty(t["q"].shape[:2], device=dev)
                assert torch.equal(out, call(t, lse=lse)), (d, step)
                check(env, t, (out, lse), f"d{d} step {step}")
    assert mp.device_error() == 0


def test_with_a_scale(env):
    torch, mp, dev = env
    for d in (64, 128):
        t = groups(torch, dev, [300, 310, 290], [0, 3], [17], 4, 2, d, 23)
        check(env, t, run(env, t, scale=0.3), scale=0.3)
