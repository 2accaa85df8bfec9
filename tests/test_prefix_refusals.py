"""Group arrays that are not aligned to their elements are refused on the host (no GPU needed)."""

import ctypes

from test_select_abi import decode, kv, lib, mp, rope  # noqa: F401  (lib: a fixture)

REF = ctypes.byref


def test_misaligned_groups(lib):
    for cu, blocks in ((0xC001, 0xD000), (0xC000, 0xD002), (0xC003, 0xD003)):
        g = mp._Prefixes(cu, blocks, 1, 1, 2)
        assert lib.minipic_attn_decode_prefix(1, 4, REF(kv()), REF(rope()), REF(decode(B=0)), REF(g), 0.0, None, 0, None) == 1
    g = mp._Prefixes(0xC004, 0xD00C, 1, 1, 2)
    assert lib.minipic_attn_decode_prefix(1, 4, REF(kv()), REF(rope()), REF(decode(B=0)), REF(g), 0.0, None, 0, None) == 0
