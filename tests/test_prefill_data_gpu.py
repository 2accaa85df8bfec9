"""The chunked prefill over data outside its ranges: positions outside the rotary table, keys outside fp16."""

import numpy as np
import pytest

from cache8_util import Case, check_attention

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


def prefill(env, c, cache):
    """(out, lse, device error) over the e4m3 pools of a case, or over their values in bf16."""
    torch, mp, dev = env
    t = c.device(torch, dev)
    ql = int(np.diff(c.cu).max())
    lse = torch.full((len(c.q_pos), c.Hq), float("nan"), device=dev)
    out = torch.full_like(t["q"], float("nan"))
    rope = mp.rope_table(c.max_pos, c.d, c.base, device=dev)
    mp.device_error(clear=True)
    rest = (t["block_tables"], t["block_starts"], t["seq_lens"], rope, ql)
    if cache == "e4m3":
        mp.attn_prefill_q8(t["q"], t["cu"], t["q_pos"], t["k_pool"], t["v_pool"], t["k_scale"], t["v_scale"], *rest,
                           lse=lse, out=out)
    else:
        k, v = (torch.from_numpy(np.nan_to_num(x).astype(np.float32)).to(dev).bfloat16() for x in c.values())
        mp.attn_prefill(t["q"], t["cu"], t["q_pos"], k, v, *rest, lse=lse, out=out)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), mp.device_error(clear=True)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64), (16, 1, 128)])
def test_keys_outside_the_table_are_masked_and_flagged(env, cache, Hq, Hkv, d):
    """A block that reaches past the table loses those keys, one that starts outside it is masked whole; the device
    error says so, and nothing is flagged without them."""
    c = Case(90 + d, (200, 64, 47), Hq, Hkv, d, "bf16", q_lens=(70, 64, 3), share=False)
    out, lse, err = prefill(env, c, cache)
    assert err == 0
    check_attention(out, c.reference(causal=True), "bf16", d, 200, "inside", p_half=2.0 ** -8)
    for what in ("reaches past", "starts behind", "starts before", "starts far before"):
        b = Case(90 + d, (200, 64, 47), Hq, Hkv, d, "bf16", q_lens=(70, 64, 3), share=False)
        b.max_pos = c.max_pos
        b.starts[0, 2] = dict(zip(("reaches past", "starts behind", "starts before", "starts far before"),
                                  (c.max_pos - 5, c.max_pos, -3, -2 ** 31)))[what]
        out, lse, err = prefill(env, b, cache)
        assert err == 2, what
        if what != "reaches past":
            b.tables[0, 2] = -1    # for the reference
        ref = b.reference(causal=True)
        check_attention(out, ref, "bf16", d, 200, what, p_half=2.0 ** -8)
        assert np.array_equal(np.isneginf(lse), np.isneginf(ref["lse"]))


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64)])
def test_8bit_keys_outside_fp16_are_flagged(env, Hq, Hkv, d):
    """A key that is beyond 65504 when rotated sets the range bit; the rows of other requests and kv heads are right."""
    c = Case(91, (200, 64), Hq, Hkv, d, "bf16", q_lens=(70, 64), share=False)
    good = c.reference(causal=True)
    c.scale[0][c.tables[0, 1], 0] = 2.0 ** 12
    out, lse, err = prefill(env, c, "e4m3")
    assert err == 16
    G = Hq // Hkv
    part = {k: np.where(np.arange(Hq)[None, :] < G, 0, good[k]) if good[k].ndim == 2 else
            np.where(np.arange(Hq)[None, :, None] < G, 0, good[k]) for k in ("out", "spread", "mass", "smax")}
    check_attention(np.where(np.arange(Hq)[None, :, None] < G, 0, out), part, "bf16", d, 200, p_half=2.0 ** -8)
    check_attention(out[70:], {k: v[70:] for k, v in good.items() if k != "weights"}, "bf16", d, 200, p_half=2.0 ** -8)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64)])
def test_8bit_prefill_passes_nan_on(env, Hq, Hkv, d):
    """A NaN key or value makes the rows of its head group that attend to it NaN; the rows of the chunk before it, whose
    causal mask excludes it, stay right, as do the other heads."""
    c = Case(92, (96, 64), Hq, Hkv, d, "bf16", q_lens=(96, 64), share=False)
    good = c.reference(causal=True)
    c.pool[0][c.tables[0, 2], 0, 3, 5] = 0x7f            # key 35 of request 0
    c.pool[1][c.tables[1, 1], Hkv - 1, 2, 7] = 0xff      # value of key 18 of request 1
    out, lse, err = prefill(env, c, "e4m3")
    G = Hq // Hkv
    assert np.all(np.isnan(out[35:96, :G])) and np.all(np.isnan(out[96 + 18:, -G:]))
    ok = np.ones(out.shape, bool)
    ok[35:96, :G] = ok[96 + 18:, -G:] = False
    zeroed = {k: np.where(ok, v, 0) if v.ndim == 3 else v for k, v in good.items() if k in ("out", "spread", "mass", "smax")}
    check_attention(np.where(ok, out, 0), zeroed, "bf16", d, 96, p_half=2.0 ** -8)
