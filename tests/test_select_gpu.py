"""Block summaries, block scores, block selection and decode over selected blocks on the GPU against float64."""

import numpy as np
import pytest

from cache8_util import HALF, check_attention, score_error
from list_util import f64
from oracle import select as osel
from select_util import batch, keys_of, pools, reference

pytestmark = pytest.mark.gpu

LENS = (523, 0, 1, 16, 47, 2050, 17, 800)
HEADS = [(4, 2, 64), (8, 8, 64), (15, 3, 64), (32, 2, 64), (8, 2, 128), (3, 3, 128), (14, 2, 128), (16, 2, 128),
         (9, 1, 128), (32, 2, 128)]
P_HALF = {"f32": None, "e4m3": 2.0 ** -11, "bf16": 2.0 ** -8}   # rounding of P


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


# ---------------------------------------------------------------- summaries

@pytest.mark.parametrize("kv,dtype", [("f32", "f32"), ("bf16", "bf16"), ("e4m3", "f32"), ("e4m3", "bf16")])
@pytest.mark.parametrize("Hkv,d", [(1, 64), (5, 64), (2, 128), (12, 128)])
def test_means(env, kv, dtype, Hkv, d):
    """Chunks that begin and end inside blocks, single keys, none; slots behind the last key hold NaN."""
    torch, mp, dev = env
    t = batch(torch, dev, [80, 33, 64, 17, 16, 200], Hkv, Hkv, d, kv, 3 * d + Hkv)
    start, count = [5, 32, 15, 0, 16, 100], [75, 1, 33, 17, 0, 61]
    nan = 0x7f if kv == "e4m3" else float("nan")
    for r, (s, n) in enumerate(zip(start, count)):
        if (s + n) % 16:
            p = t["k_pool"].view(torch.uint8) if kv == "e4m3" else t["k_pool"]
            p[int(t["block_tables"][r, (s + n) // 16]), :, (s + n) % 16:] = nan
    cu = np.concatenate([[0], np.cumsum(count)])
    rope = mp.rope_table(16, d, t["base"], device=dev)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    means = torch.full((t["k_pool"].shape[0], Hkv, d), 7.0, dtype=dt, device=dev)
    args = (i32(torch, dev, cu), i32(torch, dev, start), t["block_tables"])
    if kv == "e4m3":
        mp.kv_block_means_q8(*args, t["k_pool"], t["k_scale"], rope, means)
    else:
        mp.kv_block_means(*args, t["k_pool"], rope, means)
    k = f64(t["k_pool"]) * f64(t["k_scale"])[..., None, None]
    tables = t["block_tables"].cpu().numpy()
    want = osel.block_means(k, np.full(means.shape, 7.0), cu, start, tables, t["base"])
    # a rotated element: table, two products and a sum, 4 half steps of |x| + |y|; 16 sums, scale and mean; one rounding
    a = np.nan_to_num(np.abs(k)).max(2)
    size = a + np.roll(a, d // 2, axis=-1)
    tol = 24 * 2.0 ** -24 * size + HALF[dtype] * np.abs(want)
    got = f64(means)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol)
    untouched = np.all(want == 7.0, axis=(1, 2))
    assert untouched.any() and np.all(got[untouched] == 7.0)
    assert mp.device_error() == 0


@pytest.mark.parametrize("kv,dtype,Hkv,d", [("f32", "f32", 3, 64), ("bf16", "bf16", 3, 128), ("e4m3", "bf16", 5, 64),
                                            ("e4m3", "f32", 1, 128)])
def test_means_of_many_blocks(env, kv, dtype, Hkv, d):
    """Enough blocks that a warp takes two kv heads (an odd number of them too): the same bits as block by block."""
    torch, mp, dev = env
    n = 16 * (2700 // Hkv)
    t = batch(torch, dev, [n + 21, 40], Hkv, Hkv, d, kv, 7 * d + Hkv)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rope = mp.rope_table(16, d, t["base"], device=dev)
    fn = mp.kv_block_means_q8 if kv == "e4m3" else mp.kv_block_means
    pool = (t["k_pool"], t["k_scale"]) if kv == "e4m3" else (t["k_pool"],)
    got, want = (torch.full((t["k_pool"].shape[0], Hkv, d), 7.0, dtype=dt, device=dev) for _ in range(2))
    fn(i32(torch, dev, [0, n, n + 40]), i32(torch, dev, [21, 0]), t["block_tables"], *pool, rope, got)
    for at in range(21, n + 21, 1600):
        m = min(1600, n + 21 - at)
        a = (i32(torch, dev, [0, m, m + (at == 21) * 40]), i32(torch, dev, [at, 0]), t["block_tables"])
        fn(*a, *pool, rope, want)
    assert torch.equal(got, want)
    k = f64(t["k_pool"]) * f64(t["k_scale"])[..., None, None]
    ref = osel.block_means(k, np.full(got.shape, 7.0), [0, n, n + 40], [21, 0], t["block_tables"].cpu().numpy(), t["base"])
    a = np.abs(k).max(2)
    tol = 24 * 2.0 ** -24 * (a + np.roll(a, d // 2, axis=-1)) + HALF[dtype] * np.abs(ref)
    assert np.all(np.abs(f64(got) - ref) <= tol) and mp.device_error() == 0


def test_means_skip_what_the_append_skips(env):
    torch, mp, dev = env
    nb, Hkv, d = 6, 2, 64
    k = torch.randn(nb, Hkv, 16, d, device=dev)
    k[2, 1, 3, 5] = float("nan")
    rope = mp.rope_table(16, d, 1e4, device=dev)
    tables = i32(torch, dev, [[0, nb, 1], [2, -1, 3], [4, 5, 4], [5, 5, 5]])
    means = torch.full((nb, Hkv, d), 7.0, device=dev)

    def call(cu, start, **kw):
        mp.kv_block_means(i32(torch, dev, cu), i32(torch, dev, start), tables, k, rope, means, **kw)
        return mp.device_error(clear=True)
    assert call([0, 0, 0, 0, 0], [0, 0, 0, 0]) == 0
    assert (means == 7.0).all()
    assert call([0, 40, 80, 80, 80], [0, 0, 0, 0]) == 1            # ids 6 and -1
    assert (means[[4, 5]] == 7.0).all() and torch.isfinite(means[[0, 1, 3]]).all()
    nan = torch.isnan(means[2])
    assert nan[1, 5] and nan[1, 5 + d // 2] and int(nan.sum()) == 2   # the pair of a NaN element
    before = means.clone()
    assert call([0, 1, 1, 1, 1], [-3, 0, 0, 0]) == 4               # a negative start
    assert call([0, 0, 0, 30, 30], [0, 0, 40, 0], max_new_len=30) == 4   # beyond the table
    assert torch.equal(means[[0, 1, 3, 5]], before[[0, 1, 3, 5]]) and torch.isfinite(means[4]).all()


def test_means_follow_appends_of_any_cut(env):
    """However the keys arrive, a block's summary is that of its keys, bit for bit."""
    torch, mp, dev = env
    g = torch.Generator(device=dev).manual_seed(5)
    nb, Hkv, d, n = 4, 3, 128, 61
    x = torch.randn(n, Hkv, d, generator=g, device=dev).bfloat16()
    tables, rope = i32(torch, dev, [[2, 0, 3, 1]]), mp.rope_table(64, d, 1e4, device=dev)
    got = []
    for cuts in ([61], [1] * 61, [7, 20, 3, 31]):
        kp, vp = (torch.zeros(nb, Hkv, 16, d, dtype=torch.bfloat16, device=dev) for _ in "kv")
        means, at = torch.zeros(nb, Hkv, d, dtype=torch.bfloat16, device=dev), 0
        for c in cuts:
            a = (i32(torch, dev, [0, c]), i32(torch, dev, [at]), tables)
            mp.kv_append(x[at:at + c], x[at:at + c], *a, kp, vp, max_new_len=c)
            mp.kv_block_means(*a, kp, rope, means, max_new_len=c)
            at += c
        got.append(means)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2]) and got[0].any()
    assert mp.device_error() == 0


# ---------------------------------------------------------------- scores

def check_scores(got, ref, size, d, what=""):
    """fp32: two rotations, d products and sums (score_error's terms)."""
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    fin = np.isfinite(ref)
    tol = (6 * 2 ** 0.5 + d + 8) * 2.0 ** -24 * size + 1e-30
    assert np.all(np.abs(got - ref)[fin] <= tol[fin]), what


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_scores(env, dtype, Hq, Hkv, d):
    torch, mp, dev = env
    t = batch(torch, dev, LENS, Hq, Hkv, d, dtype, Hq + d)
    dt = t["q"].dtype
    means = (0.3 * torch.randn(t["k_pool"].shape[0], Hkv, d, device=dev)).to(dt)
    rope = mp.rope_table(t["max_pos"], d, t["base"], device=dev)
    out = torch.full((len(LENS), Hkv, t["block_tables"].shape[1]), 7.0, device=dev)
    args = (t["q"], means, t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)
    for scale in (0.0, 3.0):
        got = mp.block_scores(*args, scale=scale, out=out)
        assert got is out
        ref, size = osel.block_scores(f64(t["q"]), f64(means), t["block_tables"].cpu().numpy(),
                                      t["block_starts"].cpu().numpy(), LENS, t["q_pos"].tolist(), t["base"], scale)
        check_scores(f64(got), ref, size, d, f"{dtype} {Hq}/{Hkv} d{d}")
    assert torch.equal(mp.block_scores(*args, scale=3.0), out)
    assert mp.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_of_bad_entries(env, dtype):
    torch, mp, dev = env
    t = batch(torch, dev, [150, 70], 6, 2, 128, dtype, 11)
    nb = t["k_pool"].shape[0]
    means = torch.randn(nb, 2, 128, device=dev).to(t["q"].dtype)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    t["block_tables"][0, 3], t["block_tables"][0, 5] = nb, -9
    t["block_starts"][1, 1], t["block_starts"][1, 2] = -1, t["max_pos"]
    means[t["block_tables"][0, 7].long(), 1, 3] = float("nan")
    t["q"][1, 4, 0] = float("nan")                    # one head of kv head 1
    args = (t["q"], means, t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)
    got = f64(mp.block_scores(*args))
    assert mp.device_error(clear=True) == 1 | 2
    with np.errstate(invalid="ignore"):
        ref, size = osel.block_scores(f64(t["q"]), f64(means), t["block_tables"].cpu().numpy(),
                                      t["block_starts"].cpu().numpy(), [150, 70], t["q_pos"].tolist(), t["base"],
                                      max_pos=t["max_pos"])
    assert np.isnan(ref[0, 1, 7]) and np.isnan(ref[1, 1, 0]) and np.isneginf(ref[0, :, 3]).all()
    check_scores(got, ref, size, 128)
    t["seq_lens"][0], t["seq_lens"][1], t["q_pos"][1] = -5, 16 * 100, 10 ** 6
    got = mp.block_scores(*args)
    assert mp.device_error(clear=True) & 6 == 6 and torch.isneginf(got[0]).all()


# ---------------------------------------------------------------- selection

@pytest.mark.parametrize("mb,B,Hkv", [(1, 3, 2), (40, 5, 3), (512, 4, 2), (513, 3, 1), (2048, 3, 2), (2500, 2, 2),
                                      (8193, 2, 1), (33000, 2, 1), (70001, 1, 2)])
def test_select(env, mb, B, Hkv):
    """Ragged lengths, ties, NaN, infinities and zeros of both signs; budgets from one block to more than there are."""
    torch, mp, dev = env
    rng = np.random.default_rng(mb)
    for trial in range(6):
        s = rng.standard_normal((B, Hkv, mb)).astype(np.float32) * 4
        if trial % 2:
            s = np.round(s)                           # many ties, zeros
        s[rng.random(s.shape) < 0.05] = np.nan
        s[rng.random(s.shape) < 0.02] = np.inf
        s[rng.random(s.shape) < 0.02] = -np.inf
        s = np.where((s == 0) & (rng.random(s.shape) < 0.5), np.float32(-0.0), s)
        if trial == 4:
            s[:] = 1.5
        if trial == 5:
            s[:] = np.nan
        lens = rng.integers(0, 16 * mb + 1, B)
        lens[0] = 16 * mb
        budget = int(rng.integers(1, max(2, int(mb * 1.1))))
        first = int(rng.integers(0, min(budget, 6) + 1))
        last = int(rng.integers(0, min(budget - first, 9) + 1))
        out = torch.full((B, Hkv, budget), 77, dtype=torch.int32, device=dev)
        got = mp.block_select(torch.from_numpy(s).to(dev), i32(torch, dev, lens), budget, first, last, out=out)
        want = osel.block_select(s, lens, budget, first, last)
        assert got is out and np.array_equal(out.cpu().numpy(), want), (trial, budget, first, last)
        assert torch.equal(mp.block_select(torch.from_numpy(s).to(dev), i32(torch, dev, lens), budget, first, last), out)
    assert mp.device_error() == 0


def test_select_clamps_lengths(env):
    torch, mp, dev = env
    s = torch.arange(8.0, device=dev).expand(2, 1, 8).contiguous()
    got = mp.block_select(s, i32(torch, dev, [-4, 16 * 9]), 3, 1, 1)
    assert mp.device_error(clear=True) == 4
    assert got.tolist() == [[[-1, -1, -1]], [[0, 6, 7]]]


# ---------------------------------------------------------------- attention over selected blocks

def random_selection(rng, lens, Hkv, S, order="ascending"):
    sel = np.full((len(lens), Hkv, S), -1, np.int32)
    for r, n in enumerate(lens):
        nb = -(-int(n) // 16)
        for g in range(Hkv):
            k = min(nb, S)
            c = rng.permutation(nb)[:k]
            sel[r, g, :k] = np.sort(c) if order == "ascending" else c
    return sel


def run(env, t, sel, **kw):
    torch, mp, dev = env
    B, Hq, d = t["q"].shape
    rope = kw.pop("rope", None) or mp.rope_table(t["max_pos"], d, t["base"], device=dev)
    lse = torch.full((B, Hq), float("nan"), device=dev)
    f = mp.attn_decode_selected_q8 if t["kv"] == "e4m3" else mp.attn_decode_selected
    out, l2 = f(t["q"], *pools(t), t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope, sel, lse=lse, **kw)
    assert l2 is lse
    torch.cuda.synchronize()
    return out, lse


def check(env, t, sel, got, what="", scale=None):
    torch = env[0]
    out, lse = got
    ref = reference(torch, t, keys_of(torch, t, sel), scale)
    d = t["q"].shape[2]
    dtype = "f32" if t["q"].dtype == torch.float32 else "bf16"
    check_attention(f64(out), ref, dtype, d, sel.shape[2] * 16, what, p_half=P_HALF[t["kv"]] if dtype == "bf16" else None)
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(np.isneginf(f64(lse)), ~fin), what
    tol = score_error(ref, dtype, d) + 2.0 ** -11 + 1e-5
    assert np.all(np.abs(f64(lse)[fin] - ref["lse"][fin]) <= tol[fin]), what
    return ref


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_selected(env, kv, Hq, Hkv, d):
    torch, mp, dev = env
    t = batch(torch, dev, LENS, Hq, Hkv, d, kv, Hq * d + 1)
    rng = np.random.default_rng(Hq)
    for S in (1, 7, 60, 200):                        # 200: more than any request has
        sel = i32(torch, dev, random_selection(rng, LENS, Hkv, S))
        check(env, t, sel, run(env, t, sel), f"{kv} {Hq}/{Hkv} d{d} S{S}")
    assert mp.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (32, 2)])
def test_selected_f32_queries_over_e4m3(env, d, Hq, Hkv):
    torch, mp, dev = env
    t = batch(torch, dev, LENS, Hq, Hkv, d, "e4m3", 21)
    t["q"] = t["q"].float()
    sel = i32(torch, dev, random_selection(np.random.default_rng(0), LENS, Hkv, 9))
    check(env, t, sel, run(env, t, sel))


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_every_block_selected_is_the_whole_decode(env, kv):
    torch, mp, dev = env
    t = batch(torch, dev, LENS, 8, 2, 128, kv, 31)
    mb = t["block_tables"].shape[1]
    sel = torch.arange(mb, device=dev, dtype=torch.int32).expand(len(LENS), 2, mb).contiguous()
    out, lse = run(env, t, sel)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    bw = torch.zeros(len(LENS), 2, mb, dtype=t["q"].dtype, device=dev)
    a = (t["q"], *pools(t), t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)
    want = mp.attn_decode_q8(*a, block_weights=bw)[0] if kv == "e4m3" else mp.attn_decode_weights(*a, bw)[0]
    if kv != "bf16":
        assert torch.equal(out, want)
        return
    # the whole decode rounds a weight to bf16 where this call takes it as a sum of two bf16 values: half a step (2^-8) of
    # each p |v|, and both round the output, by half a step each
    ref = reference(torch, t, keys_of(torch, t, sel))
    tol = 2.0 ** -8 * ref["mass"] + 2 * 2.0 ** -8 * np.abs(ref["out"]) * (1 + 2.0 ** -5) + 1e-6
    assert np.all(np.abs(f64(out) - f64(want)) <= tol)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_unused_bad_unordered_and_repeated_entries(env, kv):
    """-1 anywhere in a list, numbers outside the request's blocks (flagged), any order, a block twice, no key at all;
    the slots that no length covers hold NaN."""
    torch, mp, dev = env
    lens = (330, 100, 50, 7)
    t = batch(torch, dev, lens, 8, 2, 128, kv, 41)
    nan = 0x7f if kv == "e4m3" else float("nan")
    for r, n in enumerate(lens):
        for x in "kv":
            p = t[x + "_pool"].view(torch.uint8) if kv == "e4m3" else t[x + "_pool"]
            p[int(t["block_tables"][r, n // 16]), :, n % 16:] = nan
    sel = np.full((4, 2, 12), -1, np.int32)
    sel[0, 0] = [20, 3, -1, 7, -1, 0, 11, 19, 1, -1, 2, 4]
    sel[0, 1, :3] = [5, 5, 20]                       # block 5 counts twice
    sel[1, 0, :4] = [6, -1, 2, 0]
    sel[1, 1] = -1                                   # nothing at all
    sel[2, 0, :2] = [3, 2]
    sel[2, 1, :2] = [1, 3]
    sel[3] = 0                                       # one block: the first entry is read
    s = i32(torch, dev, sel)
    ref = check(env, t, s, run(env, t, s), kv)
    assert np.all(np.isneginf(ref["lse"][1, 4:])) and mp.device_error() == 0
    sel[0, 0, 1], sel[2, 1, 0], sel[1, 0, 0] = 21, -2, 2 ** 31 - 1
    s = i32(torch, dev, sel)
    got = run(env, t, s)
    assert mp.device_error(clear=True) == 1
    check(env, t, s, got, kv + " bad")
    t["block_tables"][0, 3] = -5                     # selected, or not, by one of the heads
    t["block_tables"][0, 11] = t["k_pool"].shape[0]
    got = run(env, t, s)
    assert mp.device_error(clear=True) == 1
    check(env, t, s, got, kv + " ids")


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_nan_passes_on_where_it_is_selected(env, kv):
    torch, mp, dev = env
    t = batch(torch, dev, (100, 100), 4, 2, 128, kv, 51)
    for x, at in (("k", (0, 2, 0, 5, 9)), ("v", (1, 3, 1, 1, 64))):
        r, b, g, slot, e = at
        p = t[x + "_pool"].view(torch.uint8) if kv == "e4m3" else t[x + "_pool"]
        p[int(t["block_tables"][r, b]), g, slot, e] = 0x7f if kv == "e4m3" else float("nan")
    sel = np.tile(np.array([0, 2, 3, 6], np.int32), (2, 2, 1))
    out = f64(run(env, t, i32(torch, dev, sel))[0])
    assert np.all(np.isnan(out[0, :2])) and np.all(np.isfinite(out[0, 2:]))
    assert np.all(np.isnan(out[1, 2:, 64])) and np.all(np.isfinite(out[1, :2]))
    sel = np.tile(np.array([0, 1, 4, 5], np.int32), (2, 2, 1))
    assert np.all(np.isfinite(f64(run(env, t, i32(torch, dev, sel))[0])))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Hq,Hkv,d,S", [(1, 8, 2, 128, 700), (200, 8, 2, 128, 90), (150, 32, 2, 64, 70), (3, 64, 8, 128, 513)])
def test_lists_that_fill_the_grid_or_one_pair(env, kv, B, Hq, Hkv, d, S):
    """Lists longer than a staged piece, pairs cut between CTAs, many pairs: the same bits call after call on one
    workspace, whose counters end at zero."""
    torch, mp, dev = env
    rng = np.random.default_rng(B)
    top = 16 * S + 200
    lens = [int(x) for x in rng.integers(1, top, B)]
    lens[0] = top
    t = batch(torch, dev, lens, Hq, Hkv, d, kv, B)
    sel = i32(torch, dev, random_selection(rng, lens, Hkv, S, "any"))
    ws = torch.zeros(mp.attn_decode_selected_workspace_size(B, Hq, Hkv, d, S), dtype=torch.uint8, device=dev)
    first = None
    for i in range(10):
        got = run(env, t, sel, workspace=ws)
        assert not ws[:65536].any(), i
        if first is None:
            first = got
            check(env, t, sel, got)
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1]), i
    assert mp.device_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 4, 128), (3, 3, 64), (24, 2, 128)])
def test_many_lists_of_mixed_lengths(env, kv, Hq, Hkv, d):
    """Several times more (request, kv head) pairs than CTAs, nearly all of a few blocks, some of none, three long
    enough to be cut: the same bits twice on one workspace, whose counters end at zero."""
    torch, mp, dev = env
    rng = np.random.default_rng(Hq)
    B = 1300 // Hkv
    lens = [int(x) for x in rng.integers(0, 70, B)]
    lens[5], lens[B // 2], lens[B - 1] = 9000, 7001, 12000
    t = batch(torch, dev, lens, Hq, Hkv, d, kv, d + Hq)
    S = 640
    sel = np.full((B, Hkv, S), -1, np.int32)
    for r, n in enumerate(lens):
        for g in range(Hkv):
            blocks = rng.permutation(-(-n // 16))[:S]
            sel[r, g, :len(blocks)] = blocks
    ws = torch.zeros(mp.attn_decode_selected_workspace_size(B, Hq, Hkv, d, S), dtype=torch.uint8, device=dev)
    got = [run(env, t, i32(torch, dev, sel), workspace=ws) for _ in range(2)]
    assert not ws[:65536].any()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    check(env, t, i32(torch, dev, sel), got[0])
    assert mp.device_error() == 0


def test_more_lists_than_get_a_cta_each(env):
    """70000 (request, kv head) pairs of up to three blocks: every CTA walks a range of them."""
    torch, mp, dev = env
    B, Hkv, d, S = 8750, 8, 64, 3
    g = torch.Generator(device=dev).manual_seed(3)
    nb, mb, base = 512, 4, 1e4
    t = dict(kv="bf16", Hkv=Hkv, base=base, max_pos=4096,
             q=torch.randn(B, 8, d, generator=g, device=dev).bfloat16(),
             block_tables=torch.randint(0, nb, (B, mb), generator=g, device=dev, dtype=torch.int32),
             block_starts=torch.randint(0, 4000, (B, mb), generator=g, device=dev, dtype=torch.int32),
             seq_lens=torch.randint(0, 16 * mb + 1, (B,), generator=g, device=dev, dtype=torch.int32),
             q_pos=torch.randint(0, 4096, (B,), generator=g, device=dev, dtype=torch.int32))
    for x in ("k_pool", "v_pool"):
        t[x] = torch.randn(nb, Hkv, 16, d, generator=g, device=dev).bfloat16()
    sel = torch.argsort(torch.rand(B, Hkv, mb, generator=g, device=dev), -1)[..., :S].int().contiguous()
    sel[sel >= ((t["seq_lens"] + 15) // 16)[:, None, None]] = -1
    out, lse = run(env, t, sel)
    rows = torch.randperm(B, generator=g, device=dev)[:300]
    part = {k: (v[rows] if k in ("q", "block_tables", "block_starts", "seq_lens", "q_pos") else v) for k, v in t.items()}
    check(env, part, sel[rows], (out[rows], lse[rows]))
    assert mp.device_error() == 0


def test_selected_with_a_scale(env):
    torch, mp, dev = env
    for kv in ("f32", "bf16"):
        t = batch(torch, dev, (300, 20), 4, 2, 64, kv, 61)
        sel = i32(torch, dev, random_selection(np.random.default_rng(1), (300, 20), 2, 5))
        check(env, t, sel, run(env, t, sel, scale=0.4), scale=0.4)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_serving_loop_of_all_of_them(env, kv):
    """Prompts appended in chunks, then decode steps: append, summaries, scores, selection, attention, captured once
    and replayed; each step equals the calls made one by one, and its attention that of the float64 reference over the
    blocks that the float64 scores select (budget 6 of up to 14 blocks)."""
    torch, mp, dev = env
    g = torch.Generator(device=dev).manual_seed(7)
    B, Hq, Hkv, d, mb, budget, steps = 3, 8, 2, 128, 14, 6, 20
    nb = B * mb
    rope = mp.rope_table(512, d, 1e4, device=dev)
    tables = torch.randperm(nb, generator=g, device=dev).view(B, mb).int()
    starts = (torch.arange(mb, device=dev) * 17 + torch.tensor([[0], [40], [7]], device=dev)).int()

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev).bfloat16()
    n0 = [190, 33, 96]
    cu = i32(torch, dev, np.concatenate([[0], np.cumsum(n0)]))
    prompt = randn(sum(n0), Hkv, d), randn(sum(n0), Hkv, d)
    new = [(randn(B, Hkv, d), randn(B, Hkv, d), randn(B, Hq, d)) for _ in range(steps)]

    def fresh():
        s = dict(means=torch.zeros(nb, Hkv, d, dtype=torch.bfloat16, device=dev), lens=i32(torch, dev, n0),
                 k=torch.empty(B, Hkv, d, dtype=torch.bfloat16, device=dev), one=i32(torch, dev, range(B + 1)),
                 scores=torch.empty(B, Hkv, mb, device=dev), out=torch.empty(B, Hq, d, dtype=torch.bfloat16, device=dev),
                 sel=torch.empty(B, Hkv, budget, dtype=torch.int32, device=dev),
                 ws=torch.zeros(mp.attn_decode_selected_workspace_size(B, Hq, Hkv, d, budget), dtype=torch.uint8, device=dev))
        s["v"], s["q"] = torch.empty_like(s["k"]), torch.empty_like(s["out"])
        shape = (nb, Hkv, 16, d)
        if kv == "e4m3":
            s["cache"] = tuple(torch.full(shape, 0x7f, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in "kv") + \
                tuple(torch.full((nb, Hkv), float("nan"), device=dev) for _ in "kv")
        else:
            s["cache"] = tuple(torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev) for _ in "kv")
        append(s, *prompt, cu, i32(torch, dev, [0] * B), max(n0))
        return s

    def append(s, k, v, cu, start, most):
        if kv == "e4m3":
            mp.kv_append_q8(k, v, cu, start, tables, *s["cache"], max_new_len=most)
            mp.kv_block_means_q8(cu, start, tables, s["cache"][0], s["cache"][2], rope, s["means"], max_new_len=most)
        else:
            mp.kv_append(k, v, cu, start, tables, *s["cache"], max_new_len=most)
            mp.kv_block_means(cu, start, tables, s["cache"][0], rope, s["means"], max_new_len=most)

    def step(s):
        append(s, s["k"], s["v"], s["one"], s["lens"], 1)
        at = starts.gather(1, (s["lens"] // 16).long()[:, None])[:, 0] + s["lens"] % 16
        s["pos"] = at.int()
        s["lens"] += 1
        mp.block_scores(s["q"], s["means"], tables, starts, s["lens"], s["pos"], rope, out=s["scores"])
        mp.block_select(s["scores"], s["lens"], budget, keep_first=1, keep_last=2, out=s["sel"])
        f = mp.attn_decode_selected_q8 if kv == "e4m3" else mp.attn_decode_selected
        f(s["q"], *s["cache"], tables, starts, s["lens"], s["pos"], rope, s["sel"], out=s["out"], workspace=s["ws"])

    def feed(s, i):
        for name, x in zip("kvq", new[i]):
            s[name].copy_(x)
    plain, s = fresh(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        feed(s, 0)
        step(s)          # warm-up of the temporaries
    torch.cuda.current_stream().wait_stream(side)
    s2 = fresh()
    for name in s2:      # back to the start, in the same buffers
        for x, y in zip(s[name] if name == "cache" else (s[name],), s2[name] if name == "cache" else (s2[name],)):
            x.view(torch.uint8).copy_(y.view(torch.uint8)) if x.dim() else x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    t = dict(kv=kv, base=1e4, Hkv=Hkv, block_tables=tables, block_starts=starts, max_pos=512)
    for i in range(steps):
        feed(plain, i)
        step(plain)
        feed(s, i)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "sel", "scores", "means", "lens"):
            assert torch.equal(s[name].view(torch.uint8), plain[name].view(torch.uint8)), (i, name)
        t.update(q=plain["q"], seq_lens=plain["lens"], q_pos=plain["pos"], k_pool=plain["cache"][0], v_pool=plain["cache"][1])
        if kv == "e4m3":
            t.update(k_scale=plain["cache"][2], v_scale=plain["cache"][3])
        if i % 7 == 0:
            k = np.nan_to_num(f64(t["k_pool"].float()) * (f64(t["k_scale"])[..., None, None] if kv == "e4m3" else 1.0))
            cu0 = np.concatenate([[0], np.cumsum(plain["lens"].tolist())])
            means = osel.block_means(k, np.zeros((nb, Hkv, d)), cu0, [0] * B, tables.tolist(), 1e4)
            used = np.abs(means).sum((1, 2)) > 0
            half = HALF["bf16"] * np.abs(means) + 2e-5
            assert np.all((np.abs(f64(plain["means"]) - means) <= half)[used])
            check(env, t, plain["sel"], (plain["out"], _lse(env, t, plain["sel"], rope)), f"step {i}")
            exact = osel.block_select(f64(plain["scores"]), plain["lens"].tolist(), budget, 1, 2)
            assert np.array_equal(plain["sel"].cpu().numpy(), exact)
    assert mp.device_error() == 0


def _lse(env, t, sel, rope):
    return run(env, t, sel, rope=rope)[1]


@pytest.mark.parametrize("call", ["means", "scores", "select", "selected"])
def test_calls_on_a_side_stream(env, call):
    """What a call allocates, clears and reads belongs to its stream, while the current one is 50 ms behind."""
    torch, mp, dev = env
    lens = [5000, 17, 9000]
    t = batch(torch, dev, lens, 16, 2, 128, "bf16", 71)
    rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
    nb, mb = t["k_pool"].shape[0], t["block_tables"].shape[1]
    means = torch.randn(nb, 2, 128, device=dev).bfloat16()
    scores = torch.randn(3, 2, mb, device=dev)
    sel = i32(torch, dev, random_selection(np.random.default_rng(2), lens, 2, 50))
    cu, start = i32(torch, dev, [0, 40, 41, 141]), i32(torch, dev, [100, 3, 17])
    tabs = (t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)

    def go(**kw):
        if call == "means":
            m = means.clone() if not kw else before
            mp.kv_block_means(cu, start, t["block_tables"], t["k_pool"], rope, m, **kw)
            return m
        if call == "scores":
            return mp.block_scores(t["q"], means, *tabs, **kw)
        if call == "select":
            return mp.block_select(scores, t["seq_lens"], 30, **kw)
        return mp.attn_decode_selected(t["q"], t["k_pool"], t["v_pool"], *tabs, sel, **kw)[0]
    want, before = go().clone(), means.clone()
    n = mp.attn_decode_selected_workspace_size(3, 16, 2, 128, 50)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.empty_cache()
        for s in (torch.cuda.current_stream(), side):
            with torch.cuda.stream(s):
                junk = torch.full((n,), 0x11, dtype=torch.uint8, device=dev)   # the next workspace of that stream
                del junk
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)   # about 50 ms
        got = go(stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()
    assert mp.device_error() == 0
