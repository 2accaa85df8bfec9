"""The 8-bit cache's calls and the block-weight decode at the ends of their ranges."""

import numpy as np
import pytest

from cache8_util import Case, check_attention, check_weights
from list_util import call, f64, make_batch, reference

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


def decode(env, t, **kw):
    torch, mp, dev = env
    B, Hq, d = t["q"].shape
    out = torch.full_like(t["q"], float("nan"))
    lse = torch.full((B, Hq), float("nan"), device=dev)
    bw = torch.full((B, t["Hkv"], t["block_tables"].shape[1]), 7.0, dtype=t["q"].dtype, device=dev)
    call(mp, torch, t, mp.rope_table(t["max_pos"], d, t["base"], device=dev), out, lse, bw, None, **kw)
    torch.cuda.synchronize()
    return out, lse, bw


def as_f32(torch, t):
    """The same batch in full precision: f32 query, and over the bf16 cache f32 pools."""
    r = dict(t, q=t["q"].float())
    if t["kv"] == "bf16":
        r.update(k_pool=t["k_pool"].float(), v_pool=t["v_pool"].float())
    return r


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
@pytest.mark.parametrize("f32", [False, True])
def test_pools_past_32_bit_offsets(env, kv, f32):
    """Blocks near the end of pools of more than 2^32 bytes give what they give in a small pool."""
    torch, mp, dev = env
    t = make_batch(torch, dev, [700, 33, 1, 200], 8, 8, 128, kv, 7)
    if f32:
        t = as_f32(torch, t)
    want = decode(env, t)
    n, size = t["k_pool"].shape[0], 300_000
    big = dict(t)
    for x in "kv":
        p = torch.empty(size, *t["k_pool"].shape[1:], dtype=t["k_pool"].dtype, device=dev)
        assert p.nbytes > 2 ** 32
        p.view(torch.uint8)[size - n:] = t[x + "_pool"].view(torch.uint8)
        s = torch.full((size, 8), float("nan"), device=dev)
        s[size - n:] = t[x + "_scale"]
        big[x + "_pool"], big[x + "_scale"] = p, s
    big["block_tables"] = torch.where(t["block_tables"] >= 0, t["block_tables"] + (size - n), -1)
    got = decode(env, big)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if kv == "e4m3" and not f32:
        cu = torch.tensor([0, 300, 333, 334, 434], dtype=torch.int32, device=dev)
        g = torch.Generator(device=dev).manual_seed(1)
        q = torch.randn(434, 8, 128, generator=g, device=dev).bfloat16()
        pos = torch.arange(434, dtype=torch.int32, device=dev)
        rope = mp.rope_table(t["max_pos"], 128, t["base"], device=dev)
        outs = [mp.attn_prefill_q8(q, cu, pos, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["block_tables"],
                                   s["block_starts"], s["seq_lens"], rope, 300)[0] for s in (t, big)]
        assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()
        new = [torch.randn(434, 8, 128, generator=g, device=dev) for _ in range(2)]
        start = torch.tensor([3, 0, 0, 90], dtype=torch.int32, device=dev)
        for s in (t, big):
            mp.kv_append_q8(*new, cu, start, s["block_tables"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                            max_new_len=300)
        torch.cuda.synchronize()
        for x in "kv":
            assert torch.equal(big[x + "_pool"].view(torch.uint8)[size - n:], t[x + "_pool"].view(torch.uint8))
            assert torch.equal(big[x + "_scale"][size - n:], t[x + "_scale"])
    assert mp.device_error() == 0


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
@pytest.mark.parametrize("f32", [False, True])
def test_lengths_outside_the_table_are_clamped_and_flagged(env, kv, f32):
    torch, mp, dev = env
    t = make_batch(torch, dev, [160, 33, 5, 160], 8, 2, 128, kv, 8)
    if f32:
        t = as_f32(torch, t)
    want = decode(env, dict(t, seq_lens=torch.tensor([160, 0, 5, 160], dtype=torch.int32, device=dev)))
    assert mp.device_error(clear=True) == 0
    got = decode(env, dict(t, seq_lens=torch.tensor([161, -3, 5, 2 ** 31 - 1], dtype=torch.int32, device=dev)))
    assert mp.device_error(clear=True) == 4
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64)])
def test_prefill_lengths_outside_the_table(env, Hq, Hkv, d):
    """A context longer than its table is clamped to it, one that is negative or shorter than its chunk gives rows without
    keys; the other requests are right."""
    torch, mp, dev = env
    c = Case(93, (80, 64, 48, 33), Hq, Hkv, d, "bf16", q_lens=(30, 64, 10, 1), share=False)
    t = c.device(torch, dev)
    rope = mp.rope_table(c.max_pos, d, c.base, device=dev)

    def run(lens):
        mp.device_error(clear=True)
        n = torch.tensor(lens, dtype=torch.int32, device=dev)
        out = mp.attn_prefill_q8(t["q"], t["cu"], t["q_pos"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"],
                                 t["block_tables"], t["block_starts"], n, rope, 64)[0]
        torch.cuda.synchronize()
        return out, mp.device_error(clear=True)
    good, err = run([80, 64, 48, 33])
    assert err == 0
    check_attention(f64(good), c.reference(causal=True), "bf16", d, 80, p_half=2.0 ** -8)
    out, err = run([10 ** 9, 64, -5, 33])
    assert err == 4
    assert torch.equal(out[:30], good[:30])       # clamped to the table's 80 keys
    assert torch.equal(out[30:94], good[30:94]) and torch.equal(out[104:], good[104:])
    assert (out[94:104] == 0).all()


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("scale", [0.01, 0.7])
def test_scale_of_the_caller(env, kv, f32, scale):
    torch, mp, dev = env
    t = make_batch(torch, dev, [300, 33], 8, 2, 64, kv, 9)
    ref = reference(torch, dict(t, q=t["q"].double() * (scale * 8)))    # over 1 / sqrt(64)
    out, lse, bw = decode(env, as_f32(torch, t) if f32 else t, scale=scale)
    dtype = "f32" if f32 else "bf16"
    check_attention(f64(out), ref, dtype, 64, 300, p_half=None if f32 or kv == "e4m3" else 2.0 ** -8)
    check_weights(f64(bw), ref, dtype, 64, [300, 33], 7.0)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("max_pos", [5, 16, 20])
def test_tables_of_few_positions(env, f32, max_pos):
    """A rotary table shorter than two blocks: keys past it are masked and flagged."""
    torch, mp, dev = env
    for kv in ("e4m3", "bf16"):
        t = make_batch(torch, dev, [33, 3], 4, 2, 64, kv, 10)
        t["max_pos"] = max_pos
        t["q_pos"] = torch.tensor([max_pos - 1, 2], dtype=torch.int32, device=dev)
        t["block_starts"][0, :3] = torch.tensor([0, 2, max_pos], dtype=torch.int32, device=dev)
        t["block_starts"][1, 0] = 0
        mp.device_error(clear=True)
        out, lse, bw = decode(env, as_f32(torch, t) if f32 else t)
        assert mp.device_error(clear=True) == 2
        ref = reference(torch, t)
        dtype = "f32" if f32 else "bf16"
        check_attention(f64(out), ref, dtype, 64, 33, p_half=None if f32 or kv == "e4m3" else 2.0 ** -8)
        check_weights(f64(bw), ref, dtype, 64, [33, 3], 7.0)


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
@pytest.mark.parametrize("f32", [False, True])
def test_many_short_requests(env, kv, f32):
    """More pairs than the device holds CTAs: none is split."""
    torch, mp, dev = env
    lens = [(37 * i) % 100 for i in range(400)]
    t = make_batch(torch, dev, lens, 8, 2, 64, kv, 11)
    out, lse, bw = decode(env, as_f32(torch, t) if f32 else t)
    ref = reference(torch, t)
    dtype = "f32" if f32 else "bf16"
    check_attention(f64(out), ref, dtype, 64, 100, p_half=None if f32 or kv == "e4m3" else 2.0 ** -8)
    check_weights(f64(bw), ref, dtype, 64, lens, 7.0)
    assert mp.device_error() == 0


@pytest.mark.parametrize("inplace", [False, True])
def test_evict_tables_too_wide_for_shared_memory(env, inplace):
    """Above 49152 blocks the selection reads the scores back from memory."""
    torch, mp, dev = env
    rng = np.random.default_rng(12)
    B, mb = 3, 60_000
    lens = np.array([mb * 16 - 5, 50_001 * 16, 49_000 * 16])
    tables, starts = rng.integers(0, 1 << 20, (B, mb)), rng.integers(0, 1 << 20, (B, mb))
    scores = rng.choice(np.float32([0.5, 1.0, 2.0, np.nan]), (B, mb)) * rng.choice(np.float32([1.0, 3.0]), (B, mb))
    # weights from few values, so that many scores are equal
    w = torch.from_numpy(rng.choice(np.float32([0.0, 0.25, 1.5]), (B, 2, mb))).to(dev).bfloat16()
    for budget, first, last in ((30_000, 1, 1), (59_999, 4, 7), (11, 4, 7)):
        a = [torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in
             (scores, tables.astype(np.int32), starts.astype(np.int32), lens.astype(np.int32))]
        got = mp.kv_evict(*a, budget, keep_first=first, keep_last=last, block_weights=w, decay=0.75, inplace=inplace)
        torch.cuda.synchronize()
        got = {k: v.cpu().numpy() for k, v in got._asdict().items()}
        for r in range(B):
            n = -(-int(lens[r]) // 16)
            s = (scores[r, :n].astype(np.float64) * 0.75 + f64(w)[r, :, :n].sum(0)).astype(np.float32)
            keep = np.ones(n, bool)
            if n > budget:
                cand = np.arange(first, n - last)
                rank = np.where(np.isnan(s[cand]), -np.inf, s[cand])
                order = cand[np.lexsort((cand, -rank))]          # best first, of equal ones the lower index
                keep[order[budget - first - last:]] = False
            m = int(keep.sum())
            for name, x, fill in (("scores", s, 0), ("block_tables", tables[r, :n], -1), ("block_starts", starts[r, :n], 0)):
                assert np.array_equal(got[name][r, :m], x[keep], equal_nan=name == "scores"), (name, r, budget)
                assert (got[name][r, m:] == fill).all()
            assert np.array_equal(got["evicted"][r, :n - m], tables[r, :n][~keep]) and (got["evicted"][r, n - m:] == -1).all()
            assert got["n_evicted"][r] == n - m and got["seq_lens"][r] == lens[r] - 16 * (n - m)
    assert mp.device_error() == 0
