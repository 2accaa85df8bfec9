"""Decode behind shared prefixes on the GPU with data that a server's buffers hold in earnest: what stale rows, bad
groups and other numbers leave, each against float64."""

import pytest

from test_prefix_gpu import check, env, groups, run  # noqa: F401  (env: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (32, 2, 128), (3, 3, 128), (8, 2, 64), (16, 1, 64)])
def test_rows_that_do_not_share_hold_anything(env, Hq, Hkv, d):
    """Empty rows of a padded batch inside the group, with positions outside the table and queries of NaN and infinities:
    zeros and -inf for them, unflagged, and the other rows as ever."""
    torch, mp, dev = env
    lens = [16 * 30 + 7 * i for i in range(45)]
    empty = [0, 1, 9, 17, 30, 31, 32, 44]
    for r in empty:
        lens[r] = 0
    lens[20] = 100    # shorter than the prefix: its own keys, at its own position
    t = groups(torch, dev, lens, [0, 45], [30], Hq, Hkv, d, 41)
    for r, pos in zip(empty, (-1, 2 ** 31 - 1, -2 ** 31, t["max_pos"], t["max_pos"] + 1, -1, 10 ** 9, -12345)):
        t["q_pos"][r] = pos
        t["q"][r] = float("nan") if r % 2 else float("inf")
    check(env, t, run(env, t), f"{Hq}/{Hkv} d{d}")
    assert mp.device_error() == 0
