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


@pytest.mark.parametrize("d", [64, 128])
def test_bad_groups_share_nothing(env, d):
    """Groups whose numbers lie outside the batch or the planning bounds, or whose boundaries descend, and every group
    behind descending ones, are flagged and read their own keys: rows that they hold begin with different blocks."""
    torch, mp, dev = env
    t = groups(torch, dev, [400, 420, 440, 460, 500, 380, 0, 390], [0, 3], [10], 8, 2, d, 43)   # requests 0 .. 2 share
    for cu, blocks in (([0, 3, 9], [10, 12]), ([0, 3, 8], [10, 33]), ([0, 3, 2, 6], [10, 12, 12]), ([-1, 3, 6], [10, 0]),
                       ([3, 0, 8], [10, 12]), ([0, 3, 1, 8, 8], [10, 3, 12, 4]), ([0, 3, -5, 8], [10, 3, 12]),
                       ([0, 3, 2 ** 31 - 1, 8, -2 ** 31, 8], [10, 12, 12, 12, 12]), ([-2 ** 31, 2 ** 31 - 1], [10])):
        t["cu"], t["blocks"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (cu, blocks))
        got = run(env, t, max_requests=6, max_prefix_blocks=10 ** 6)
        assert mp.device_error(clear=True) == 4, (cu, blocks)
        check(env, t, got, f"d{d} {cu}")


@pytest.mark.parametrize("Hq,Hkv,d,B", [(8, 8, 64, 200), (8, 8, 128, 160), (4, 2, 128, 60)])
def test_overlapping_groups(env, Hq, Hkv, d, B):
    """Groups that go over the same requests again and again (flagged), more than are staged among them: no item is left
    without a CTA, whatever an earlier call left in the workspace, with the join in the same kernel or its own."""
    torch, mp, dev = env
    t = groups(torch, dev, [16 * 40 + 5 * i % 130 for i in range(B)], [0, B // 2], [40], Hq, Hkv, d, 47)
    mb = t["block_tables"].shape[1]
    ws = torch.zeros(max(mp.attn_decode_prefix_workspace_size(B, Hq, Hkv, d, mb, n, B, 10 ** 6) for n in (1, 9, 300)),
                     dtype=torch.uint8, device=dev)
    check(env, t, run(env, t, workspace=ws, max_requests=B), "one group")
    assert mp.device_error() == 0
    for n in (9, 300):
        cu = [0] * (n - 7) + [B // 2, 0, B, 0, B, 3, B, 1]
        t["cu"], t["blocks"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (cu, [40] * n))
        got = run(env, t, workspace=ws, max_requests=B)
        assert mp.device_error(clear=True) == 4
        check(env, t, got, f"{n} groups")
        assert not ws[:65536].any()


@pytest.mark.parametrize("Hkv,d,B", [(2, 64, 6), (2, 128, 6), (8, 64, 160), (8, 128, 120)])
def test_a_nan_query_shows(env, Hkv, d, B):
    """A query with a NaN element makes its head's row NaN, lse too, and no other: for a request that ends with its
    prefix, one whose own keys are all masked, and one with keys of its own; with the join in the same kernel or its own."""
    torch, mp, dev = env
    lens = [16 * 40 + 11 * i % 90 for i in range(B)]
    lens[1], lens[3] = 16 * 40, 16 * 41
    t = groups(torch, dev, lens, [0, B], [40], 2 * Hkv, Hkv, d, 53)
    t["block_tables"][3, 40] = -1
    for r in (1, 3, 4):
        t["q"][r, 1, 7] = float("nan")
    out, lse = run(env, t, max_requests=B)
    assert mp.device_error(clear=True) == 1 | 16    # the block id, and a query outside fp16
    nan = torch.zeros_like(lse, dtype=torch.bool)
    nan[[1, 3, 4], 1] = True
    assert torch.equal(lse.isnan(), nan) and torch.equal(out.isnan(), nan[..., None].expand_as(out))


def shared_or_not(t):
    """Bounds under which the kernel for shared prefixes runs, and ones under which nothing is shared."""
    return (True, dict(max_requests=len(t["q"]), max_prefix_blocks=10 ** 6)), \
           (False, dict(max_requests=len(t["q"]), max_prefix_blocks=int(t["blocks"].max())))


@pytest.mark.parametrize("d", [64, 128])
def test_keys_outside_fp16(env, d):
    """A key of a shared prefix outside fp16's range sets the range bit, and only rows of its kv head may be off; where the
    bounds share nothing it is a key like any other."""
    torch, mp, dev = env
    t = groups(torch, dev, [16 * 12 + 9 * i for i in range(7)], [0, 4], [12], 8, 2, d, 59)
    t["k_pool"][int(t["block_tables"][0, 3]), 1, 5, 9] = 2.0 ** 17
    other = dict(t, q=t["q"][:, :4].contiguous(), Hkv=1, k_pool=t["k_pool"][:, :1], v_pool=t["v_pool"][:, :1])
    for shared, bounds in shared_or_not(t):
        out, lse = run(env, t, **bounds)
        assert mp.device_error(clear=True) == (16 if shared else 0)
        check(env, other, (out[:, :4], lse[:, :4]), f"kv head 0, d{d}")
        assert shared or (out.isfinite().all() and lse.isfinite().all())


@pytest.mark.parametrize("d", [64, 128])
def test_blocks_that_start_before_position_0(env, d):
    """In a shared prefix they are masked whole, where the bounds share nothing the slots before position 0 (flagged);
    what the values of the masked slots hold does not show."""
    torch, mp, dev = env
    for start in (-5, -16, -10 ** 6):
        t = groups(torch, dev, [16 * 12 + 9 * i for i in range(7)], [0, 7], [12], 8, 2, d, 61)
        t["block_starts"][:, 4] = start
        t["v_pool"][int(t["block_tables"][0, 4]), :, :min(16, -start)] = float("nan")
        for shared, bounds in shared_or_not(t):
            got = run(env, t, **bounds)
            assert mp.device_error(clear=True) == 2
            want = dict(t, block_starts=t["block_starts"].clone())
            if shared:
                want["block_starts"][:, 4] = -16
            check(env, want, got, f"{start} shared {shared} d{d}")
