"""Pins of the oracle for block summaries, scores and selection: closed forms, explicit scores, brute force."""

import itertools

import numpy as np
import pytest

import oracle
from oracle import select as sel


def test_a_summary_scores_the_mean_of_its_keys_at_any_start():
    """(R_t q) . (R_b m) equals the mean over the block's keys of their scores at start b."""
    rng = np.random.default_rng(0)
    Hkv, G, d, base = 2, 3, 8, 100.0
    k = rng.standard_normal((5, Hkv, 16, d))
    tables, cu, start = np.array([[3, 1, 4], [0, 2, -1]]), [0, 40, 50], [0, 7]
    means = sel.block_means(k, np.zeros((5, Hkv, d)), cu, start, tables, base)
    q, q_pos = rng.standard_normal((2, Hkv * G, d)), [100, 57]
    starts = np.array([[5, 30, 60], [0, 1234, 0]])
    lens = [40, 17]
    s, size = sel.block_scores(q, means, tables, starts, lens, q_pos, base)
    for r, n in enumerate(lens):
        for b in range(-(-n // 16)):
            m = min(16, n - 16 * b)
            kr = oracle.rope_rotate(k[tables[r, b]][:, :m], starts[r, b] + np.arange(m), base)
            qr = oracle.rope_rotate(q[r], np.full(Hkv * G, q_pos[r]), base)
            for g in range(Hkv):
                want = (qr[g * G:(g + 1) * G] @ kr[g].T / np.sqrt(d)).mean(1).max()
                assert abs(s[r, g, b] - want) < 1e-12
                assert abs(want) <= size[r, g, b] + 1e-12
    assert np.all(np.isneginf(s[1, :, 2])) and np.all(np.isfinite(s[0]))


def test_means_touch_the_appended_blocks_only():
    k = np.ones((4, 1, 16, 4))
    k[2, 0, 5:] = np.nan
    before = np.full((4, 1, 4), 9.0)
    got = sel.block_means(k, before, [0, 3, 3], [18, 4], np.array([[0, 2], [1, 3]]), 10.0)
    assert np.all(got[[0, 1, 3]] == 9.0) and np.all(np.isfinite(got[2]))
    pos = oracle.rope_rotate(np.ones((5, 4)), np.arange(5), 10.0).mean(0)
    assert np.allclose(got[2, 0], pos, atol=1e-15)


def test_selection_by_brute_force():
    rng = np.random.default_rng(1)
    for trial in range(300):
        n = int(rng.integers(0, 8))
        s = rng.integers(-2, 3, n).astype(float)
        s[rng.random(n) < 0.2] = np.nan
        budget = int(rng.integers(1, 7))
        first = int(rng.integers(0, budget + 1))
        last = int(rng.integers(0, budget - first + 1))
        got = sel.block_select(np.concatenate([s, np.full(2, 7.0)])[None, None], [16 * n - (3 if n else 0)], budget, first,
                               last)[0, 0]
        chosen = got[got >= 0]
        assert list(chosen) == sorted(chosen) and np.all(got[len(chosen):] == -1) and len(chosen) == min(n, budget)
        if n <= budget:
            continue
        held = {b for b in range(n) if b < first or b >= n - last}
        assert held <= set(chosen)
        value = np.where(np.isnan(s), -1e9, s)
        best = max(value[list(c)].sum() for c in itertools.combinations(range(n), budget) if held <= set(c))
        assert value[chosen].sum() == best
        for out in set(range(n)) - set(chosen):   # of equal scores the lower index
            assert not any(value[c] == value[out] and c > out and c not in held for c in chosen)


def test_nan_ranks_below_every_score():
    s = np.array([[[0.0, np.nan, -np.inf, 1.0, 2.0]]])
    assert list(sel.block_select(s, [80], 4, 0, 0)[0, 0]) == [0, 2, 3, 4]


@pytest.mark.parametrize("wrong", ["slot", "start"])
def test_planted_mistakes_show(wrong):
    """Keys not rotated by their slot, or a summary not rotated by its block's start, change the scores."""
    rng = np.random.default_rng(2)
    k, q = rng.standard_normal((2, 1, 16, 8)), rng.standard_normal((1, 2, 8))
    tables, starts = np.array([[1, 0]]), np.array([[3, 40]])
    right = sel.block_means(k, np.zeros((2, 1, 8)), [0, 32], [0], tables, 50.0)
    s, _ = sel.block_scores(q, right, tables, starts, [32], [70], 50.0)
    means = k.mean(2) if wrong == "slot" else right
    w, _ = sel.block_scores(q, means, tables, starts + (wrong == "start"), [32], [70], 50.0)
    assert np.abs(s - w).max() > 1e-2
