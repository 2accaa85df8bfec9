"""Pins of the oracle for the 8-bit cache, block weights and eviction: against
torch's own e4m3 conversion, closed forms and brute force."""

import itertools

import numpy as np
import pytest

import oracle
from oracle import cache8 as c8
import workloads as W


def test_e4m3_values_and_rounding_match_torch():
    torch = pytest.importorskip("torch")
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(c8.VALUES))
    assert np.array_equal(t[~np.isnan(t)], c8.VALUES[~np.isnan(t)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000), c8.VALUES[:126],
                        (c8.VALUES[:125] + c8.VALUES[1:126]) / 2, [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(c8.encode(x), want)
    assert np.array_equal(c8.encode([np.inf, -np.inf, 1e9]), [0x7e, 0xfe, 0x7e])
    assert c8.encode([np.nan])[0] & 0x7f == 0x7f


def test_scale_is_the_least_power_of_two():
    for amax in (448.0, 448.0000001, 1.0, 1.75, 1.7500001, 3e38, 2.0 ** -93, 1e-40, 0.0):
        s = c8.scale_for(np.array([amax, -amax / 2, np.nan, np.inf]))
        assert amax <= 448 * s and np.log2(s) == int(np.log2(s))
        assert s == 2.0 ** -100 or amax > 448 * s / 2


def test_append_keeps_what_the_scale_can_hold():
    """Row by row or at once, values end within the e4m3 rounding of the block's
    scale; earlier rows are re-rounded, never dropped."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((20, 2, 64)) * np.exp(rng.standard_normal((20, 2, 1)))
    tables = np.array([[1, 0]])
    pool, scale = np.full((2, 2, 16, 64), 0x7f, np.uint8), np.full((2, 2), 7.0)
    one = c8.append(pool, scale, x, [0, 20], [0], tables)
    step = (pool, scale)
    for i in range(20):
        step = c8.append(*step, x[i:i + 1], [0, 1], [i], tables)
    assert np.array_equal(one[1], step[1])
    for p, s in (one, step):
        v = c8.values(p, s)
        got = np.concatenate([v[1].transpose(1, 0, 2), v[0][:, :4].transpose(1, 0, 2)])
        sc = np.concatenate([np.repeat(s[1][None], 16, 0), np.repeat(s[0][None], 4, 0)])[..., None]
        # two roundings: half a step each, 2^-4 relative or half of a subnormal step
        assert np.all(np.abs(got - x) <= 2 * np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * sc))


def test_attention_equals_the_decode_oracle_and_weights_are_shares():
    w = W.irregular_decode(5, "f32", seq_lens=[0, 1, 37, 64], Hq=4, Hkv=2, d=64)
    d = w.decode
    k, v = w.kv.k_pool.astype(np.float64), w.kv.v_pool.astype(np.float64)
    r = c8.attention(d.q, np.arange(d.batch + 1), d.q_pos, k, v, d.block_tables, d.block_starts, d.seq_lens, w.rope_base)
    ref, lse = oracle.decode(w)
    assert np.allclose(r["out"], ref, atol=1e-12)
    fin = np.isfinite(lse)
    assert np.array_equal(np.isfinite(r["lse"]), fin) and np.allclose(r["lse"][fin], lse[fin], atol=1e-12)
    assert np.allclose(r["weights"].sum(2)[1:], 2.0) and np.all(r["weights"][0] == 0)
    assert np.allclose(r["weights"][1, :, 1:], 0)


def test_causal_attention_equals_the_prefill_oracle():
    w = W.irregular_prefill(3, "f32", kv_lens=[40, 33], q_lens=[17, 33], Hq=4, Hkv=2, d=64)
    p = w.prefill
    r = c8.attention(p.q, p.cu_q_lens, p.q_pos, w.kv.k_pool.astype(np.float64), w.kv.v_pool.astype(np.float64),
                     p.block_tables, p.block_starts, p.kv_lens, w.rope_base, causal=True)
    ref, _ = oracle.prefill(w)
    assert np.allclose(r["out"], ref, atol=1e-12)


def test_evict_keeps_the_best_set():
    """Brute force: no other set of `budget` blocks that holds the required ones has a larger total."""
    rng = np.random.default_rng(2)
    n, budget, first, last = 9, 5, 1, 2
    scores = rng.random((1, 12)).astype(np.float32)
    w = rng.random((1, 3, 12))
    tables = np.arange(100, 112)[None].astype(np.int32)
    o = c8.evict(scores, tables, tables * 16, [n * 16 - 5], budget, first, last, weights=w, decay=0.5)
    s = (scores[0, :n].astype(np.float64) * 0.5 + w[0, :, :n].sum(0)).astype(np.float32)
    kept = o["block_tables"][0, :budget] - 100
    must = {0, n - 1, n - 2}
    assert must <= set(kept.tolist()) and np.all(np.diff(kept) > 0)
    best = max(sum(s[b] for b in c) for c in itertools.combinations(range(n), budget) if must <= set(c))
    assert np.isclose(sum(s[b] for b in kept), best)
    assert o["seq_lens"][0] == budget * 16 - 5 and o["n_evicted"][0] == 4
    assert sorted(kept.tolist() + (o["evicted"][0, :4] - 100).tolist()) == list(range(n))
    tie = c8.evict(np.ones((1, 6), np.float32), tables[:, :6], tables[:, :6], [96], 4, 0, 1)
    assert tie["block_tables"][0].tolist() == [100, 101, 102, 105, -1, -1]
