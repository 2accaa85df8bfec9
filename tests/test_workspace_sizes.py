"""Workspace sizes of the decodes over selected blocks and behind shared prefixes: enough for every smaller call."""

import random

import pytest


@pytest.fixture(scope="module")
def mp():
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as m
    m.load()
    return m


def spread(rng, hi):
    return int(round(hi ** rng.random()))


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (16, 8, 64), (16, 1, 128), (64, 8, 128), (128, 8, 128), (9, 9, 64)])
def test_sizes_hold_for_smaller_calls(mp, Hq, Hkv, d):
    """No size grows when a batch, a table, a budget or a bound becomes smaller, one or all of them."""
    rng = random.Random(Hq * d)
    prefix, selected = mp.attn_decode_prefix_workspace_size, mp.attn_decode_selected_workspace_size
    for _ in range(3000):
        big = [spread(rng, 20000), spread(rng, 4000), spread(rng, 300), spread(rng, 20000), spread(rng, 10 ** 6)]
        small = [rng.choice((x, max(1, x - 1), spread(rng, x))) for x in big]
        size = [prefix(b, Hq, Hkv, d, mb, p, r, n) for b, mb, p, r, n in (big, small)]
        assert 0 < size[1] <= size[0], (big, small)
        size = [selected(b, Hq, Hkv, d, mb) for b, mb, *_ in (big, small)]
        assert 0 < size[1] <= size[0], (big, small)


def test_sizes_across_plans(mp):
    """Batches on both sides of where a plan changes: the waves of the prefix kernel, a CTA a pair, f32 splits."""
    prefix, selected = mp.attn_decode_prefix_workspace_size, mp.attn_decode_selected_workspace_size
    for f, batches in ((lambda b: prefix(b, 64, 8, 128, 2100, 1, b, 2048), range(200, 260)),
                       (lambda b: prefix(b, 128, 8, 128, 208, 1, b, 200), range(2, 300)),
                       (lambda b: prefix(b, 16, 8, 64, 108, 1, b, 100), range(2, 3000, 7)),
                       (lambda b: selected(b, 8, 8, 64, 40), range(8100, 8300)),
                       (lambda b: selected(b, 8, 8, 64, 400), range(1, 200))):
        sizes = [f(b) for b in batches]
        assert sizes == sorted(sizes)
