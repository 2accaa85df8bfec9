"""Block starts of any 32-bit value in the decode and mixed calls: masked and flagged, nothing else changed."""

import pytest

import workloads as W
from gpu_util import upload_decode

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64), (32, 2, 128)])
@pytest.mark.parametrize("mixed", [False, True])
def test_starts_of_any_value(dtype, Hq, Hkv, d, mixed):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if mixed and dtype == "f32":
        pytest.skip("the mixed call is bf16 only")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    dev = torch.device("cuda:0")
    lens = [300, 47, 2050, 16]
    w = W.irregular_decode(33, dtype, seq_lens=lens, Hq=Hq, Hkv=Hkv, d=d)
    t = upload_decode(w, torch, dev)
    rope = mp.rope_table(w.max_pos, d, w.rope_base, device=dev)

    def run(t):
        ws = torch.zeros(mp.decode_workspace_size(len(lens), Hq, Hkv, d, t["block_tables"].shape[1]), dtype=torch.uint8,
                         device=dev)
        dec = {k: t[k] for k in ("q", "block_tables", "block_starts", "seq_lens", "q_pos")}
        if mixed:
            p = dict(q=t["q"][:1], cu_q_lens=torch.tensor([0, 1], dtype=torch.int32, device=dev), q_pos=t["q_pos"][:1],
                     block_tables=t["block_tables"][:1], block_starts=t["block_starts"][:1], kv_lens=t["seq_lens"][:1],
                     max_q_len=1)
            out = mp.attn_mixed(p, dec, t["k_pool"], t["v_pool"], rope, workspace=ws)[2]
        else:
            out = mp.attn_decode(dec["q"], t["k_pool"], t["v_pool"], *list(dec.values())[1:], rope, workspace=ws)[0]
        torch.cuda.synchronize()
        return out
    mp.device_error(clear=True)
    run(t)
    assert mp.device_error(clear=True) == 0
    masked = dict(t, block_tables=t["block_tables"].clone(), block_starts=t["block_starts"].clone())
    for r, b, start in ((0, 3, LOW), (1, 0, HIGH), (2, 5, LOW + 1), (2, 60, HIGH - 7), (2, 100, -16), (3, 0, w.max_pos)):
        masked["block_starts"][r, b] = start
        masked["block_tables"][r, b] = -1
    masked["q_pos"] = t["q_pos"].clone()
    masked["q_pos"][0] = 0                     # its distance to the lowest start is 2^31
    want = run(masked)
    assert mp.device_error(clear=True) & 1
    got = run(dict(masked, block_tables=t["block_tables"]))
    assert mp.device_error(clear=True) == 2
    assert torch.equal(got, want)
    assert (got[3] == 0).all() and torch.isfinite(got.float()).all()
