"""The 8-bit cache, block weights and eviction on the GPU against the float64 oracle."""

import numpy as np
import pytest

from oracle import cache8 as c8
import oracle
import workloads as W
from cache8_util import Case, check_attention, check_weights
from gpu_util import upload_decode

pytestmark = pytest.mark.gpu

LENS = (523, 0, 1, 16, 47, 2050, 17, 800)


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


def f64(t):
    return t.double().cpu().numpy()


def decode(env, c, weights=True, rope=None, **kw):
    torch, mp, dev = env
    t = c.device(torch, dev)
    rope = rope or mp.rope_table(c.max_pos, c.d, c.base, device=dev)
    B, mb = c.tables.shape
    bw = torch.full((B, c.Hkv, mb), 7.0, dtype=t["q"].dtype, device=dev) if weights else None
    lse = torch.full((B, c.Hq), float("nan"), device=dev)
    out, _ = mp.attn_decode_q8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["block_tables"],
                               t["block_starts"], t["seq_lens"], t["q_pos"], rope, lse=lse, block_weights=bw, **kw)
    torch.cuda.synchronize()
    return f64(out), f64(lse), f64(bw) if weights else None


def check_decode(env, c, got, what="", **kw):
    out, lse, bw = got
    ref = c.reference(**kw)
    check_attention(out, ref, c.dtype, c.d, max(c.lens), what)
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(np.isfinite(lse), fin)
    from cache8_util import score_error
    eps = score_error(ref, c.dtype, c.d)
    assert np.all(np.abs(lse - ref["lse"])[fin] <= (eps + 2.0 ** -11 + 1e-5)[fin]), what
    if bw is not None:
        check_weights(bw, ref, c.dtype, c.d, c.lens, 7.0, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 8, 64), (15, 3, 64), (32, 2, 64), (8, 2, 128), (3, 3, 128),
                                      (14, 2, 128), (16, 2, 128), (9, 1, 128), (32, 2, 128)])
def test_decode_matches_the_oracle(env, dtype, Hq, Hkv, d):
    c = Case(Hq * d, LENS, Hq, Hkv, d, dtype)
    check_decode(env, c, decode(env, c), f"{dtype} {Hq}/{Hkv} d{d}")
    assert env[1].device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [dict(pow2=False), dict(spread=2.0), dict(pow2=False, spread=2.0)])
def test_decode_with_scales_of_any_size(env, dtype, kw):
    """Scales that are no powers of two, and that differ by up to 2^24 from block to block."""
    c = Case(3, (700, 33, 5), 8, 2, 128, dtype, **kw)
    if "spread" in kw:   # keys of the same size, values of very different ones
        c.scale[0] = np.where(np.isnan(c.scale[0]), np.nan, 2.0 ** -8)
    check_decode(env, c, decode(env, c), str(kw))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_with_zero_scales_and_zero_queries(env, dtype):
    c = Case(4, (130, 40), 4, 1, 64, dtype)
    c.scale[1][c.tables[0, :3]] = 0.0          # blocks of zeros
    c.scale[0][c.tables[0, 2:5]] = 0.0
    c.scale[1][c.tables[1, :3]] = 0.0          # a request whose values are all zero
    c.q[0, 1] = 0.0
    c.q_store[0, 1] = 0
    got = decode(env, c)
    check_decode(env, c, got)
    assert np.all(got[0][1] == 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_with_queries_of_any_size(env, dtype):
    """Queries far outside fp16's range against keys that bring the scores back."""
    c = Case(5, (200, 17), 4, 2, 128, dtype)
    for f, h in ((2.0 ** 40, 0), (2.0 ** -40, 1)):
        c.q[:, 2 * h:2 * h + 2] *= f
        c.scale[0][:, h] /= f
    c.q_store = c.q.astype(np.float32) if dtype == "f32" else W.to_bf16_bits(c.q.astype(np.float32))
    check_decode(env, c, decode(env, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_masks_bad_blocks_and_positions(env, dtype):
    """Bad ids and keys past the table are masked, whatever the slots hold; a request may lose every key."""
    torch, mp, dev = env
    c = Case(6, (150, 70, 33), 8, 2, 128, dtype, share=False)
    nb = len(c.pool[0])
    c.tables[0, 3] = nb
    c.tables[0, 5] = -1
    c.tables[2, :3] = -7                        # a row with nothing left
    c.max_pos = int(c.starts[1, 4]) + 3         # request 1's last block reaches past the table after 3 keys
    c.starts[0] = np.where(c.starts[0] + 15 < c.max_pos, c.starts[0], 0)
    c.q_pos[:] = np.minimum(c.q_pos, c.max_pos - 1)
    for p in c.pool:
        p[c.tables[1, 4], :, 3:] = 0x7f
    got = decode(env, c)
    assert mp.device_error(clear=True) == 1 | 2
    check_decode(env, c, got)
    assert np.all(got[0][2] == 0) and np.all(np.isneginf(got[1][2])) and np.all(got[2][2, :, :3] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_passes_nan_on(env, dtype):
    """A NaN key or value that a query attends to makes that head group's output NaN and no other."""
    c = Case(7, (100, 100, 100), 4, 2, 128, dtype, share=False)
    c.pool[0][c.tables[0, 2], 0, 5, 9] = 0x7f
    c.pool[1][c.tables[1, 3], 1, 1, 64] = 0xff
    out, _, _ = decode(env, c, weights=False)
    assert np.all(np.isnan(out[0, :2])) and np.all(np.isfinite(out[0, 2:]))
    assert np.all(np.isnan(out[1, 2:, 64])) and np.all(np.isfinite(out[1, :2]))
    assert np.all(np.isfinite(out[2]))


def test_decode_sharp_and_flat_scores(env):
    """A dominating key (the rest far below it) and all-equal scores: no weight is lost, block sums add up to G."""
    for q_scale in (0.0, 30.0):
        c = Case(8, (4096, 600), 8, 2, 128, "bf16")
        c.q *= q_scale
        c.q_store = W.to_bf16_bits(c.q.astype(np.float32))
        c.q = W.bf16_bits_to_f32(c.q_store).astype(np.float64)
        out, lse, bw = decode(env, c)
        ref = c.reference()
        if q_scale == 0.0:
            check_attention(out, ref, "bf16", 128, 4096)
            assert np.all(np.abs(bw[0] - 4 / 256) <= 4 / 256 * 2.0 ** -7)
        assert np.all(np.abs(bw[0].sum(-1) - 4.0) <= 4 * 2.0 ** -7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_workspace_for_calls_of_other_shapes(env, dtype):
    """Shapes with and without splits and weights take turns on one workspace, zeroed once."""
    torch, mp, dev = env
    cases = [Case(9, (3000, 50), 8, 2, 128, dtype), Case(10, (20,) * 40, 4, 2, 64, dtype),
             Case(11, (9000,), 16, 1, 128, dtype)]
    n = max(mp.attn_decode_q8_workspace_size(len(c.lens), c.Hq, c.Hkv, c.d, c.tables.shape[1]) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    for i in (0, 1, 2, 1, 0, 2):
        check_decode(env, cases[i], decode(env, cases[i], workspace=ws, weights=i != 1))


def torch_reference(torch, t, base, Hkv):
    """The reference of cache8.attention for one row per request, in float64 on the GPU (for sizes numpy is slow at)."""
    q, B = t["q"].double(), t["q"].shape[0]
    Hq, d = q.shape[1:]
    G, mb = Hq // Hkv, t["block_tables"].shape[1]
    res = {k: np.zeros((B, Hq, d)) for k in ("out", "spread", "mass")}
    res.update(lse=np.full((B, Hq), -np.inf), smax=np.zeros((B, Hq)), weights=np.zeros((B, Hkv, mb)))

    def turn(x, pos):   # [..., n, d] rotated at pos [n]
        i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
        a = pos.double()[:, None] * base ** (-2 * i / d)
        x1, x2 = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)
    for r in range(B):
        n = int(t["seq_lens"][r])
        if not n:
            continue
        j = torch.arange(n, device=q.device)
        blk = t["block_tables"][r].long()[j // 16]
        pos = t["block_starts"][r].long()[j // 16] + j % 16
        qr = turn(q[r], t["q_pos"][r].expand(Hq))
        for g in range(Hkv):
            k, v = (t[x + "_pool"].view(torch.uint8)[blk, g, j % 16].view(torch.float8_e4m3fn).double() *
                    t[x + "_scale"].double()[blk, g][:, None] for x in "kv")
            k = turn(k, pos)
            h = slice(g * G, (g + 1) * G)
            s = qr[h] @ k.T / d ** 0.5
            p = torch.softmax(s, 1)
            o = p @ v
            res["out"][r, h], res["lse"][r, h] = f64(o), f64(torch.logsumexp(s, 1))
            res["mass"][r, h] = f64(p @ v.abs())
            for i in range(G):
                res["spread"][r, g * G + i] = f64(p[i] @ (v - o[i]).abs())
            res["smax"][r, h] = f64(qr[h].norm(dim=1) * k.norm(dim=1).max() / d ** 0.5)
            w = torch.zeros(-(-n // 16) * 16, dtype=torch.float64, device=q.device)
            w[:n] = p.sum(0)
            res["weights"][r, g, :w.numel() // 16] = f64(w.view(-1, 16).sum(1))
    return res


@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ([0, 3, 40, 0, 17, 1, 64] * 45, 4, 2, 64),           # more requests than a CTA has threads, many of them empty
    ([40000], 8, 1, 128),                                 # one pair shared by many CTAs
    ([70001, 5, 90000], 20, 2, 64),                       # groups of 10
    ([33000, 0, 60000, 16, 52017, 49999], 28, 28, 128),   # ranges longer than one staging of metadata
    ([33000, 0, 60000, 16, 52017, 49999], 56, 8, 128),
])
def test_decode_at_sizes_that_cut_pairs_and_ranges(env, lens, Hq, Hkv, d):
    torch, mp, dev = env
    g = torch.Generator(device=dev).manual_seed(len(lens) + Hq)
    B, mb = len(lens), -(-max(lens) // 16)
    n = torch.tensor(lens, device=dev)
    nb = int(((n + 15) // 16).sum()) + 1
    order = torch.randperm(nb, generator=g, device=dev)
    used = torch.arange(mb, device=dev) * 16 < n[:, None]
    tables = torch.full((B, mb), -1, dtype=torch.int32, device=dev)
    tables[used] = order[:int(used.sum())].int()
    gaps = torch.randint(0, 3, (B, mb), generator=g, device=dev).cumsum(1)
    starts = torch.where(used, torch.arange(mb, device=dev) * 16 + gaps, 0).int()
    t = {}
    for x in "kv":
        y = torch.randn(nb, Hkv, 16, d, generator=g, device=dev)
        s = torch.exp2(torch.ceil(torch.log2(y.abs().amax((2, 3)) / 448)))
        t[x + "_scale"], t[x + "_pool"] = s, (y / s[..., None, None]).to(torch.float8_e4m3fn)
    last = (n - 1).clamp(min=0)
    t.update(q=torch.randn(B, Hq, d, generator=g, device=dev).bfloat16(), block_tables=tables, block_starts=starts,
             seq_lens=n.int(), q_pos=(starts.long().gather(1, (last // 16)[:, None])[:, 0] + last % 16 + 1).int())
    rope = mp.rope_table(int(starts.max()) + 40, d, 1e4, device=dev)
    ref = torch_reference(torch, t, 1e4, Hkv)
    ws = torch.zeros(mp.attn_decode_q8_workspace_size(B, Hq, Hkv, d, mb), dtype=torch.uint8, device=dev)
    outs = []
    for weights in (True, False, True):
        bw = torch.full((B, Hkv, mb), 7.0, dtype=torch.bfloat16, device=dev) if weights else None
        lse = torch.empty(B, Hq, device=dev)
        out, _ = mp.attn_decode_q8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], tables, starts,
                                   t["seq_lens"], t["q_pos"], rope, lse=lse, block_weights=bw, workspace=ws)
        torch.cuda.synchronize()
        check_attention(f64(out), ref, "bf16", d, max(lens))
        fin = np.isfinite(ref["lse"])
        assert np.array_equal(np.isfinite(f64(lse)), fin)
        assert np.abs(f64(lse)[fin] - ref["lse"][fin]).max() <= 1e-2
        if weights:
            check_weights(f64(bw), ref, "bf16", d, lens, 7.0)
        outs.append((out, lse, bw))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))   # the parts merge in a fixed order
    assert mp.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B", [1, 300])
def test_a_batch_without_any_key(env, dtype, B):
    """Zero lengths throughout: out 0, lse -inf, the weights left as they were."""
    torch, mp, dev = env
    ty = dict(f32=torch.float32, bf16=torch.bfloat16)[dtype]
    Hq, Hkv, d, mb = 8, 2, 64, 3
    q = torch.ones(B, Hq, d, dtype=ty, device=dev)
    pool = torch.ones(4, Hkv, 16, d, device=dev)
    sc = torch.ones(4, Hkv, device=dev)
    tables, starts = (torch.zeros(B, mb, dtype=torch.int32, device=dev) for _ in range(2))
    lens, pos = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(2))
    rope = mp.rope_table(64, d, 1e4, device=dev)
    for q8 in (True, False):
        bw = torch.full((B, Hkv, mb), 7.0, dtype=ty, device=dev)
        out, lse = torch.full_like(q, 5.0), torch.full((B, Hq), 5.0, device=dev)
        if q8:
            p8 = pool.to(torch.float8_e4m3fn)
            mp.attn_decode_q8(q, p8, p8, sc, sc, tables, starts, lens, pos, rope, out=out, lse=lse, block_weights=bw)
        else:
            mp.attn_decode_weights(q, pool.to(ty), pool.to(ty), tables, starts, lens, pos, rope, bw, out=out, lse=lse)
        torch.cuda.synchronize()
        assert (out == 0).all() and (lse == -float("inf")).all() and (bw == 7.0).all()
    assert mp.device_error() == 0


def test_two_graphs_on_one_workspace(env):
    """Two captured calls of different shapes share a workspace and are replayed in turn."""
    torch, mp, dev = env
    cases = [Case(60, (2500, 300), 8, 2, 128, "bf16"), Case(61, (40,) * 30 + (900,), 4, 4, 64, "bf16")]
    ws = torch.zeros(max(mp.attn_decode_q8_workspace_size(len(c.lens), c.Hq, c.Hkv, c.d, c.tables.shape[1])
                         for c in cases), dtype=torch.uint8, device=dev)
    runs = []
    for c in cases:
        t = c.device(torch, dev)
        rope = mp.rope_table(c.max_pos, c.d, c.base, device=dev)
        out = torch.empty_like(t["q"])
        bw = torch.zeros(len(c.lens), c.Hkv, c.tables.shape[1], dtype=torch.bfloat16, device=dev)

        def call(t=t, rope=rope, out=out, bw=bw):
            mp.attn_decode_q8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["block_tables"],
                              t["block_starts"], t["seq_lens"], t["q_pos"], rope, out=out, block_weights=bw,
                              workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((c, g, out, bw, t))
    for _ in range(3):
        for c, g, out, bw, _t in runs:
            out.zero_()
            bw.zero_()
            g.replay()
    torch.cuda.synchronize()
    for c, g, out, bw, _t in runs:
        ref = c.reference()
        check_attention(f64(out), ref, "bf16", c.d, max(c.lens))
        check_weights(f64(bw), ref, "bf16", c.d, c.lens, 0.0)


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("f32", 8, 2, 64), ("bf16", 4, 2, 64), ("bf16", 32, 2, 64),
                                            ("bf16", 8, 1, 128), ("bf16", 28, 4, 128), ("bf16", 16, 1, 128)])
def test_decode_weights_over_the_unquantised_cache(env, dtype, Hq, Hkv, d):
    """out near attn_decode's, out and weights against float64 (scores from fp16 products; P is bf16)."""
    torch, mp, dev = env
    lens = [300, 0, 1, 16, 47, 2050, 17, 800]
    w = W.irregular_decode(21, dtype, seq_lens=lens, Hq=Hq, Hkv=Hkv, d=d)
    t = upload_decode(w, torch, dev)
    rope = mp.rope_table(w.max_pos, d, w.rope_base, device=dev)
    mb = t["block_tables"].shape[1]
    bw = torch.full((len(lens), Hkv, mb), 7.0, dtype=t["q"].dtype, device=dev)
    lse, lse0 = (torch.empty(len(lens), Hq, device=dev) for _ in range(2))
    args = (t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"], t["seq_lens"], t["q_pos"], rope)
    out, _ = mp.attn_decode_weights(*args, bw, lse=lse)
    out0, _ = mp.attn_decode(*args, lse=lse0)
    torch.cuda.synchronize()
    k, v = (oracle.widen(x, dtype) for x in (w.kv.k_pool, w.kv.v_pool))
    ref = c8.attention(oracle.widen(w.decode.q, dtype), np.arange(len(lens) + 1), w.decode.q_pos, k, v,
                       w.decode.block_tables, w.decode.block_starts, lens, w.rope_base)
    check_attention(f64(out), ref, dtype, d, max(lens), p_half=2.0 ** -8 if dtype == "bf16" else None)
    check_weights(f64(bw), ref, dtype, d, lens, 7.0)
    assert float((out.float() - out0.float()).abs().max()) <= (2e-2 if dtype == "bf16" else 1e-5)
    assert mp.device_error() == 0


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("f32", 8, 2, 64), ("bf16", 8, 2, 64), ("bf16", 8, 1, 128),
                                            ("bf16", 16, 1, 128)])
def test_decode_weights_with_nan_in_masked_and_attended_slots(env, dtype, Hq, Hkv, d):
    """Slots past the lengths hold NaN and one request has bad blocks: nothing of them shows; an attended NaN does."""
    torch, mp, dev = env
    lens = [35, 300, 7, 48]
    w = W.irregular_decode(22, dtype, seq_lens=lens, Hq=Hq, Hkv=Hkv, d=d, pool_blocks=40)
    D = w.decode
    blocks = iter(np.random.default_rng(22).permutation(40))   # each block in one place: the generator repeats them
    for r, n in enumerate(lens):
        for b in range(-(-n // 16)):
            D.block_tables[r, b] = next(blocks)
    nan = np.float32(np.nan) if dtype == "f32" else np.uint16(0x7fc0)
    for r, n in enumerate(lens):
        if n % 16:
            for p in (w.kv.k_pool, w.kv.v_pool):
                p[D.block_tables[r, n // 16], :, n % 16:] = nan
    D.block_tables[1, 3] = 10 ** 6
    t = upload_decode(w, torch, dev)
    rope = mp.rope_table(w.max_pos, d, w.rope_base, device=dev)
    mb = t["block_tables"].shape[1]

    def call():
        bw = torch.zeros(len(lens), Hkv, mb, dtype=t["q"].dtype, device=dev)
        out, _ = mp.attn_decode_weights(t["q"], t["k_pool"], t["v_pool"], t["block_tables"], t["block_starts"],
                                        t["seq_lens"], t["q_pos"], rope, bw)
        torch.cuda.synchronize()
        return f64(out), f64(bw)
    mp.device_error(clear=True)
    out, bw = call()
    assert mp.device_error(clear=True) == 1
    k, v = (oracle.widen(x, dtype) for x in (w.kv.k_pool, w.kv.v_pool))
    ref = c8.attention(oracle.widen(D.q, dtype), np.arange(len(lens) + 1), D.q_pos, k, v, D.block_tables,
                       D.block_starts, lens, w.rope_base)
    check_attention(out, ref, dtype, d, max(lens), p_half=2.0 ** -8 if dtype == "bf16" else None)
    check_weights(bw, ref, dtype, d, lens, 0.0)
    t["v_pool"][int(D.block_tables[3, 1]), 0, 4, 5] = float("nan")
    t["k_pool"][int(D.block_tables[0, 0]), Hkv - 1, 2, 1] = float("nan")
    out, bw = call()
    assert mp.device_error(clear=True) == 1
    G = Hq // Hkv
    assert np.all(np.isnan(out[3, :G, 5])) and np.all(np.isfinite(out[3, :, 6]))
    assert np.all(np.isnan(out[0, -G:])) and np.all(np.isnan(bw[0, -1, :3]))


# ------------------------------------------------------------------------------------------------ prefill

@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (12, 2, 64), (8, 2, 128), (7, 1, 128), (16, 1, 128), (3, 3, 128)])
@pytest.mark.parametrize("pow2", [True, False])
def test_prefill_matches_the_oracle(env, Hq, Hkv, d, pow2):
    """Chunks of 1 token to more than a query tile, over caches of 0 to a few hundred keys, tails inside a block.
    P is bf16 there; a scale that is no power of two adds one bf16 rounding to each key and value."""
    torch, mp, dev = env
    lens, ql = (300, 1, 47, 16, 530, 33), (120, 1, 1, 16, 260, 33)
    c = Case(30 + d, lens, Hq, Hkv, d, "bf16", pow2=pow2, q_lens=ql, share=False)
    t = c.device(torch, dev)
    rope = mp.rope_table(c.max_pos, d, c.base, device=dev)
    lse = torch.empty(len(c.q_pos), Hq, device=dev)
    out, _ = mp.attn_prefill_q8(t["q"], t["cu"], t["q_pos"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"],
                                t["block_tables"], t["block_starts"], t["seq_lens"], rope, max(ql), lse=lse)
    torch.cuda.synchronize()
    ref = c.reference(causal=True)
    big = dict(ref, smax=ref["smax"] * (1 if pow2 else 3))
    check_attention(f64(out), big, "bf16", d, max(lens), p_half=2.0 ** -8 * (1 if pow2 else 2))
    assert mp.device_error() == 0


def test_prefill_masks_bad_blocks(env):
    torch, mp, dev = env
    c = Case(41, (200, 64), 8, 2, 128, "bf16", q_lens=(70, 64), share=False)
    c.tables[0, 2] = 10 ** 6
    c.tables[1, 0] = -1                        # the first chunk rows of request 1 see nothing
    t = c.device(torch, dev)
    rope = mp.rope_table(c.max_pos, 128, c.base, device=dev)
    out, _ = mp.attn_prefill_q8(t["q"], t["cu"], t["q_pos"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"],
                                t["block_tables"], t["block_starts"], t["seq_lens"], rope, 70)
    torch.cuda.synchronize()
    assert mp.device_error(clear=True) == 1
    check_attention(f64(out), c.reference(causal=True), "bf16", 128, 200, p_half=2.0 ** -8)
    assert np.all(f64(out)[70:86] == 0)


def test_prefill_refuses_a_small_workspace(env):
    torch, mp, dev = env
    c = Case(42, (40,), 4, 2, 64, "bf16", q_lens=(10,))
    t = c.device(torch, dev)
    rope = mp.rope_table(c.max_pos, 64, c.base, device=dev)
    with pytest.raises(mp.MiniPICError) as e:
        mp.attn_prefill_q8(t["q"], t["cu"], t["q_pos"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"],
                           t["block_tables"], t["block_starts"], t["seq_lens"], rope, 10,
                           workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    assert e.value.status == 3


# ------------------------------------------------------------------------------------------------ append

def append(env, pool, scale, new, cu, start, tables, dtype, max_new=None):
    torch, mp, dev = env

    def dv(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    store = [W.to_bf16_bits(x) if dtype == "bf16" else x.astype(np.float32) for x in new]
    n = [dv(x.view(np.int16)).view(torch.bfloat16) if dtype == "bf16" else dv(x) for x in store]
    p = [dv(x).view(torch.float8_e4m3fn) for x in pool]
    s = [dv(x.astype(np.float32)) for x in scale]
    mp.kv_append_q8(*n, dv(np.array(cu, np.int32)), dv(np.array(start, np.int32)), dv(np.array(tables, np.int32)), *p,
                    *s, max_new_len=max_new)
    torch.cuda.synchronize()
    vals = [W.bf16_bits_to_f32(x) if dtype == "bf16" else x for x in store]
    return [x.view(torch.uint8).cpu().numpy() for x in p], [f64(x) for x in s], vals


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,d", [(1, 64), (3, 128), (8, 128), (5, 64)])
def test_append_equals_the_oracle_bit_for_bit(env, dtype, Hkv, d):
    """Fresh blocks, blocks entered late, scales that grow and that do not, counts of zero, 129 to 300 tokens."""
    rng = np.random.default_rng(Hkv + d)
    n = np.array([1, 0, 17, 300, 16, 129, 3])
    start = np.array([5, 3, 31, 0, 16, 9, 15])
    cu = np.concatenate([[0], np.cumsum(n)])
    mb = int(((start + n + 15) // 16).max())
    tables = rng.permutation(7 * mb + 2)[:7 * mb].reshape(7, mb)
    pool = [rng.integers(0, 256, (7 * mb + 2, Hkv, 16, d)).astype(np.uint8) for _ in range(2)]
    for p in pool:
        p[(p & 0x7f) == 0x7f] = 0x3c
    scale = [np.exp2(rng.integers(-12, 0, (7 * mb + 2, Hkv))).astype(np.float64) for _ in range(2)]
    new = [(rng.standard_normal((cu[-1], Hkv, d)) * np.exp(2 * rng.standard_normal((cu[-1], Hkv, 1)))).astype(np.float32)
           for _ in range(2)]
    got_p, got_s, vals = append(env, pool, scale, new, cu, start, tables, dtype)
    for i in range(2):
        want_p, want_s = c8.append(pool[i], scale[i], vals[i], cu, start, tables)
        assert np.array_equal(got_s[i], want_s)
        assert np.array_equal(got_p[i], want_p)
    assert env[1].device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_extreme_values(env, dtype):
    """Zeros, tiny, huge, infinite and NaN values; another scale than a power of two in the block entered."""
    torch, mp, dev = env
    mp.device_error(clear=True)
    d, Hkv = 64, 6
    x = np.random.default_rng(0).standard_normal((3, Hkv, d)).astype(np.float32)
    x[:, 0] = 0.0
    x[:, 1] *= 2.0 ** -120
    x[:, 2] *= 2.0 ** 125
    x[0, 3, 5], x[1, 3, 6] = np.inf, -np.inf
    x[2, 4, 7] = np.nan
    pool = [np.full((2, Hkv, 16, d), 0x30, np.uint8)] * 2
    scale = [np.full((2, Hkv), 0.013671875 * 1.1).astype(np.float32).astype(np.float64)] * 2
    for start in (0, 4):
        mp.device_error(clear=True)
        got_p, got_s, vals = append(env, pool, scale, [x, x], [0, 3], [start], [[1]], dtype)
        assert mp.device_error(clear=True) == 16   # the infinities
        want_p, want_s = c8.append(pool[0], scale[0], vals[0], [0, 3], [start], [[1]])
        assert np.array_equal(got_s[0], want_s) and np.array_equal(got_s[1], want_s)
        pow2 = np.log2(want_s[1]) == np.round(np.log2(want_s[1]))
        for p in got_p:
            nan = (want_p & 0x7f) == 0x7f
            assert np.array_equal(nan, (p & 0x7f) == 0x7f)
            same = (p == want_p) | nan
            assert np.all(same[:, pow2] if start == 0 else same[1][pow2])
            # x / s is rounded to fp32 first where s is no power of two: at most the neighbouring byte
            assert np.all(np.abs((p & 0x7f).astype(int) - (want_p & 0x7f).astype(int)) <= 1)


def test_append_skips_and_flags_what_does_not_fit(env):
    torch, mp, dev = env
    rng = np.random.default_rng(3)
    pool = [rng.integers(0, 0x70, (6, 2, 16, 64)).astype(np.uint8) for _ in range(2)]
    scale = [np.ones((6, 2))] * 2
    new = [rng.standard_normal((60, 2, 64)).astype(np.float32) for _ in range(2)]
    mp.device_error(clear=True)
    for tables, start, bit in (([[0, 9], [1, 2]], [0, 0], 1), ([[0, -1], [1, 2]], [0, 0], 1),
                               ([[0, 3], [1, 2]], [-3, 0], 4), ([[0, 3], [1, 2]], [5, 0], 4)):
        got_p, got_s, vals = append(env, pool, scale, new, [0, 30, 60], start, tables, "f32")
        assert mp.device_error(clear=True) == bit
        for i in range(2):  # what fits is written as alone
            want_p, want_s = c8.append(pool[i], scale[i], vals[i], [30, 60], [0], [[1, 2]])
            if start[0] >= 0:
                m = min(30, (16 if bit == 1 else 32) - start[0])
                want_p, want_s = c8.append(want_p, want_s, vals[i], [0, m], [start[0]], tables[:1])
            assert np.array_equal(got_p[i], want_p) and np.array_equal(got_s[i], want_s)
    # rows past the new ones
    append(env, pool, scale, [x[:50] for x in new], [0, 30, 60], [0, 0], [[0, 3], [1, 2]], "f32")
    assert mp.device_error(clear=True) == 4


def test_append_past_its_bound_is_written_whole(env):
    """max_new_len only sizes the grid: a request with more tokens than it is still written."""
    rng = np.random.default_rng(4)
    pool, scale = [np.zeros((20, 2, 16, 128), np.uint8)] * 2, [np.ones((20, 2))] * 2
    new = [rng.standard_normal((290, 2, 128)).astype(np.float32) for _ in range(2)]
    tables = rng.permutation(20)[None]
    got_p, got_s, vals = append(env, pool, scale, new, [0, 290], [7], tables, "bf16", max_new=1)
    for i in range(2):
        want_p, want_s = c8.append(pool[i], scale[i], vals[i], [0, 290], [7], tables)
        assert np.array_equal(got_p[i], want_p) and np.array_equal(got_s[i], want_s)


# ------------------------------------------------------------------------------------------------ eviction

def evict(env, scores, tables, starts, lens, budget, first, last, weights=None, decay=1.0, dtype="f32", inplace=False):
    torch, mp, dev = env

    def dv(a, t):
        return torch.from_numpy(np.ascontiguousarray(a, t)).to(dev)
    w = None if weights is None else dv(weights, np.float32).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    a = [dv(scores, np.float32), dv(tables, np.int32), dv(starts, np.int32), dv(lens, np.int32)]
    keep = [x.clone() for x in a]
    r = mp.kv_evict(*a, budget, keep_first=first, keep_last=last, block_weights=w, decay=decay, inplace=inplace)
    torch.cuda.synchronize()
    if not inplace:
        assert all(torch.equal(x, y) or x.isnan().any() for x, y in zip(a, keep))
    return {k: v.cpu().numpy() for k, v in r._asdict().items()}, None if w is None else f64(w)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,mb,Hkv,dtype,decay", [(3, 1, 1, "f32", 1.0), (5, 33, 2, "bf16", 0.5), (4, 1024, 8, "bf16", 1.0),
                                                  (3, 2500, 3, "f32", 0.9), (1, 9000, 1, "bf16", 0.0)])
def test_evict_equals_the_oracle(env, B, mb, Hkv, dtype, decay, inplace):
    rng = np.random.default_rng(mb)
    lens = rng.integers(0, mb * 16 + 1, B)
    lens[0] = mb * 16 - (mb > 1)
    tables, starts = rng.integers(0, 1 << 20, (B, mb)), rng.integers(0, 1 << 20, (B, mb))
    scores = np.exp(2 * rng.standard_normal((B, mb))).astype(np.float32)
    w = np.exp(2 * rng.standard_normal((B, Hkv, mb)))
    for budget, first, last in ((max(2, mb // 3), 1, 1), (mb + 5, 0, 3), (max(7, mb // 2), 3, 4), (2, 0, 1), (5, 2, 3)):
        got, wv = evict(env, scores, tables, starts, lens, budget, first, last, w, decay, dtype, inplace)
        want = c8.evict(scores, tables, starts, lens, budget, first, last, wv, decay)
        for k in want:
            assert np.array_equal(got[k], want[k]), (k, budget, first, last)
    assert env[1].device_error() == 0


def test_evict_ties_and_odd_scores(env):
    """Equal scores leave from the end; signed zeros are equal; negative and infinite scores rank as numbers; NaN leaves
    first."""
    mb = 2100
    rng = np.random.default_rng(5)
    tables = np.arange(mb)[None]
    for scores in (np.ones((1, mb)), rng.choice([0.0, -0.0, 1.0], (1, mb)), -np.exp(rng.standard_normal((1, mb))),
                   rng.choice([np.inf, -np.inf, 3.0, -2.0, np.nan], (1, mb))):
        scores = scores.astype(np.float32)
        for budget in (1, 700, 2099):
            got, _ = evict(env, scores, tables, tables * 16, [mb * 16 - 3], budget, 0, 1)
            want = c8.evict(scores, tables, tables * 16, [mb * 16 - 3], budget, 0, 1)
            for k in want:
                assert np.array_equal(got[k], want[k], equal_nan=k == "scores"), (k, budget)


def test_evict_flags_bad_lengths(env):
    torch, mp, dev = env
    mp.device_error(clear=True)
    t = np.arange(8).reshape(2, 4)
    got, _ = evict(env, np.ones((2, 4)), t, t, [-5, 1000], 2, 0, 1)
    assert mp.device_error(clear=True) == 4
    assert got["n_evicted"].tolist() == [0, 2] and got["seq_lens"].tolist() == [0, 32]


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("graph", [False, True])
def test_a_bounded_8bit_session(env, graph):
    """As a server uses them: prompts appended and prefilled over the 8-bit cache, then decode steps that append a
    token, attend with block weights and evict in place, the position of the next token going on.  With ``graph`` the
    step is captured once and replayed.  Tables equal the oracle's step by step; attention is checked on the cache's
    bytes."""
    torch, mp, dev = env
    rng = np.random.default_rng(12)
    B, Hq, Hkv, d, mb, base, budget = 3, 8, 2, 128, 16, 1e4, 9
    n0 = np.array([150, 37, 16])
    nb = B * mb + 1
    own = rng.permutation(nb)[:B * mb].reshape(B, mb)
    max_pos, steps = 512, 12

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)

    def randn(*s):
        return torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    kp, vp = (torch.full((nb, Hkv, 16, d), 0x7f, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
              for _ in range(2))
    ks, vs = (torch.full((nb, Hkv), float("nan"), device=dev) for _ in range(2))
    tables, starts, scores = i32(own), i32(np.tile(np.arange(mb) * 16, (B, 1))), torch.zeros(B, mb, device=dev)
    rope = mp.rope_table(max_pos, d, base, device=dev)
    cu = np.concatenate([[0], np.cumsum(n0)])
    mp.kv_append_q8(randn(cu[-1], Hkv, d), randn(cu[-1], Hkv, d), i32(cu), i32(np.zeros(B)), tables, kp, vp, ks, vs,
                    max_new_len=int(n0.max()))
    q = randn(cu[-1], Hq, d)
    q_pos = np.concatenate([np.arange(n) for n in n0])
    out, _ = mp.attn_prefill_q8(q, i32(cu), i32(q_pos), kp, vp, ks, vs, tables, starts, i32(n0), rope, int(n0.max()))

    def pools():
        return [c8.values(p.view(torch.uint8).cpu().numpy(), f64(s)) for p, s in ((kp, ks), (vp, vs))]
    ref = c8.attention(f64(q), cu, q_pos, *pools(), own, starts.cpu().numpy(), n0, base, causal=True)
    check_attention(f64(out), ref, "bf16", d, 150, p_half=2.0 ** -8)

    lens, pos = i32(n0), i32(n0)
    one = i32(np.arange(B + 1))
    k1, v1, q1 = (torch.empty(B, h, d, dtype=torch.bfloat16, device=dev) for h in (Hkv, Hkv, Hq))
    ws = torch.zeros(mp.attn_decode_q8_workspace_size(B, Hq, Hkv, d, mb), dtype=torch.uint8, device=dev)
    bw = torch.zeros(B, Hkv, mb, dtype=torch.bfloat16, device=dev)
    o1 = torch.empty_like(q1)
    spare = i32(own)   # every physical block of a request, to put a fresh one behind the kept ones
    taken = {}

    def step():
        mp.kv_append_q8(k1, v1, one, lens, tables, kp, vp, ks, vs, max_new_len=1)
        lens.add_(1)
        mp.attn_decode_q8(q1, kp, vp, ks, vs, tables, starts, lens, pos, rope, out=o1, block_weights=bw, workspace=ws)
        r = mp.kv_evict(scores, tables, starts, lens, budget, keep_first=1, keep_last=2, block_weights=bw, decay=0.9,
                        inplace=True)
        taken["evicted"], taken["n"] = r.evicted, r.n_evicted
        pos.add_(1)

    def host():
        return tables.cpu().numpy().copy(), starts.cpu().numpy().copy(), lens.cpu().numpy().copy()

    def next_block():
        """Host bookkeeping between steps: a request whose last block is full gets a free one at the next position."""
        t, s, n = host()
        for r in range(B):
            if n[r] % 16 == 0:
                k = n[r] // 16
                t[r, k] = next(b for b in own[r] if b not in t[r, :k])
                s[r, k] = int(pos[r])
        tables.copy_(i32(t))
        starts.copy_(i32(s))

    g = None
    for i in range(steps):
        next_block()
        for x in (k1, v1, q1):
            x.copy_(randn(*x.shape))
        t, s, n = host()
        sc, p0 = scores.cpu().numpy(), pos.cpu().numpy()
        if graph and i == 2:
            state = [x.clone() for x in (tables, starts, lens, pos, scores, bw, ws, kp.view(torch.uint8),
                                         vp.view(torch.uint8), ks, vs)]
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            for x, y in zip((tables, starts, lens, pos, scores, bw, ws, kp.view(torch.uint8), vp.view(torch.uint8),
                             ks, vs), state):
                assert torch.equal(x, y) or x.isnan().any()   # capture ran nothing
        g.replay() if g is not None else step()
        torch.cuda.synchronize()
        ref = c8.attention(f64(q1), np.arange(B + 1), p0, *pools(), t, s, n + 1, base)
        check_attention(f64(o1), ref, "bf16", d, 200, f"step {i}")
        w = f64(bw)
        check = c8.evict(sc, t, s, n + 1, budget, 1, 2, w, 0.9)
        for name, x in (("block_tables", tables), ("block_starts", starts), ("seq_lens", lens), ("scores", scores),
                        ("evicted", taken["evicted"]), ("n_evicted", taken["n"])):
            assert np.array_equal(x.cpu().numpy(), check[name]), (i, name)
    assert mp.device_error() == 0


def test_calls_on_another_stream(env):
    """Temporaries of a call on a side stream belong to that stream: two calls at once do not meet."""
    torch, mp, dev = env
    cases = [Case(50 + i, (2000, 700), 8, 2, 128, "bf16") for i in range(2)]
    ts = [c.device(torch, dev) for c in cases]
    ropes = [mp.rope_table(c.max_pos, c.d, c.base, device=dev) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = [mp.attn_decode_q8(t["q"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], t["block_tables"],
                                  t["block_starts"], t["seq_lens"], t["q_pos"], rope, stream=s)[0]
                for t, rope, s in zip(ts, ropes, streams)]
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        check_attention(f64(o), c.reference(), "bf16", 128, 2000)
