"""Decode and mixed calls over the f32 / bf16 cache: what masked slots hold never shows."""

import numpy as np
import pytest

import workloads as W
from gpu_util import upload_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64), (32, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("call", ["decode", "prerotated", "mixed"])
def test_nan_and_infinity_in_masked_slots(dtype, Hq, Hkv, d, call):
    """Slots past the lengths and blocks whose positions lie outside the table hold NaN or infinities, and some table
    entries are bad: the outputs are those of a pool with zeros there."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if call == "mixed" and dtype == "f32":
        pytest.skip("the mixed call is bf16 only")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    dev = torch.device("cuda:0")
    lens = [300, 47, 2050, 16, 1, 7]
    w = W.irregular_decode(34, dtype, seq_lens=lens, Hq=Hq, Hkv=Hkv, d=d, pool_blocks=200)
    D = w.decode
    blocks = iter(np.random.default_rng(34).permutation(200))   # each block in one place
    for r, n in enumerate(lens):
        for b in range(-(-n // 16)):
            D.block_tables[r, b] = next(blocks)
    dead = [(0, 4), (2, 9), (3, 0)]                              # their starts lie outside the table
    for r, b in dead:
        D.block_starts[r, b] = w.max_pos
    t = upload_decode(w, torch, dev)
    rope = mp.rope_table(w.max_pos, d, w.rope_base, device=dev)
    clean = {k: t[k].clone() for k in ("k_pool", "v_pool")}
    for k, bad in (("k_pool", float("inf")), ("v_pool", float("nan"))):
        for r, n in enumerate(lens):
            if n % 16:
                x = int(D.block_tables[r, n // 16])
                t[k][x, :, n % 16:] = bad
                clean[k][x, :, n % 16:] = 0
        if call != "prerotated":                                  # which has no positions
            for r, b in dead:
                t[k][int(D.block_tables[r, b])] = bad
                clean[k][int(D.block_tables[r, b])] = 0
    bad_id = t["block_tables"].clone()
    bad_id[1, 1], bad_id[2, 50], bad_id[5, 0] = 10 ** 6, -1, -5

    def run(pools, tables):
        a = (t["q"], pools["k_pool"], pools["v_pool"], tables, t["block_starts"], t["seq_lens"], t["q_pos"])
        mp.device_error(clear=True)
        if call == "decode":
            out = mp.attn_decode(*a, rope)[0]
        elif call == "prerotated":
            out = mp.attn_decode_prerotated(*a)[0]
        else:
            p = dict(q=t["q"][3:4], cu_q_lens=torch.tensor([0, 1], dtype=torch.int32, device=dev), q_pos=t["q_pos"][3:4],
                     block_tables=tables[3:4].contiguous(), block_starts=t["block_starts"][3:4].contiguous(),
                     kv_lens=t["seq_lens"][3:4], max_q_len=1)
            dec = dict(zip(("q", "block_tables", "block_starts", "seq_lens", "q_pos"), (a[0],) + a[3:]))
            out = mp.attn_mixed(p, dec, a[1], a[2], rope)[2]
        torch.cuda.synchronize()
        return out, mp.device_error(clear=True)
    for tables in (t["block_tables"], bad_id):
        want, _ = run(clean, tables)
        got, err = run(t, tables)
        assert torch.isfinite(got.float()).all()
        assert torch.equal(got, want)
        assert err == (0 if call == "prerotated" else 2) | (1 if tables is bad_id else 0)
    assert (got[5] == 0).all()
