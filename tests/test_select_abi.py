"""Refusals of the calls over selected blocks and shared prefixes: every case fails
validation on the host, before any launch (no GPU needed)."""

import ctypes

import pytest

import position_independent_kv_paged_gb300 as mp
from position_independent_kv_paged_gb300 import _build

REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mp.load()


# fake, never dereferenced addresses
def kv(nb=4, hkv=2, bs=16, d=128, k=0x1000, v=0x2000):
    return mp._KV(k, v, nb, hkv, bs, d)


def kvq8(nb=4, hkv=2, bs=16, d=128, k=0x1000, v=0x2000, ks=0x2100, vs=0x2200):
    return mp._KVQ8(k, v, ks, vs, nb, hkv, bs, d)


def rope(d=128, f32=0x9000, f16=0xB000, n=1024):
    return mp._Rope(f32, n, d, f16, None)


def decode(B=1, mb=4, q=0x3000, bt=0x4000, st=0x5000, sl=0x6000, qp=0x7000, out=0x8000):
    return mp._Decode(q, bt, st, sl, qp, B, mb, out, None)


def test_means_refusals(lib):
    def ab(B=2, total=5, mx=3, mb=4, cu=0x5000):
        return mp._Append(None, None, cu, 0x6000, 0x7000, B, total, mx, mb)

    def call(dtype=1, p=None, rp=None, b=None, means=0xA000):
        return lib.minipic_kv_block_means(dtype, REF(p or kv()), REF(rp or rope()), REF(b or ab()), means, None)

    def q8(dtype=1, p=None, b=None):
        return lib.minipic_kv_block_means_q8(dtype, REF(p or kvq8()), REF(rope()), REF(b or ab()), 0xA000, None)
    assert call(dtype=2) == 1
    assert call(p=kv(d=80), rp=rope(d=80)) == 2
    assert call(p=kv(bs=8)) == 2
    assert call(p=kv(hkv=0)) == 1
    assert call(p=kv(nb=0)) == 1
    assert call(p=kv(k=0x1008)) == 1
    assert call(p=kv(k=None)) == 1
    assert call(rp=rope(d=64)) == 1
    assert call(rp=rope(f32=None)) == 1
    assert call(rp=rope(n=15)) == 2                            # a table row for every slot
    assert call(means=None) == 1
    assert call(means=0xA008) == 1
    assert call(b=ab(cu=None)) == 1
    assert call(b=ab(B=-1)) == 1
    assert call(b=ab(mx=-1)) == 1
    assert call(b=ab(mb=0)) == 1
    assert call(b=ab(B=70000)) == 1
    for nothing in (ab(B=0), ab(total=0), ab(mx=0)):
        assert call(b=nothing) == 0 and q8(b=nothing) == 0
    assert q8(p=kvq8(ks=None)) == 1
    assert q8(p=kvq8(ks=0x2101)) == 1
    assert q8(dtype=3) == 1
    assert lib.minipic_kv_block_means(1, None, REF(rope()), REF(ab()), 0xA000, None) == 1
    assert lib.minipic_kv_block_means_q8(1, None, REF(rope()), REF(ab()), 0xA000, None) == 1
    assert lib.minipic_kv_block_means(1, REF(kv()), REF(rope()), None, 0xA000, None) == 1
    assert lib.minipic_kv_block_means(1, REF(kv()), None, REF(ab()), 0xA000, None) == 1


def test_scores_refusals(lib):
    def sb(B=1, mb=4, nb=4, hkv=2, d=128, q=0x1000, means=0x2000, out=0x8000, sl=0x5000):
        return mp._Scores(q, means, 0x3000, 0x4000, sl, 0x6000, B, mb, nb, hkv, d, out)

    def call(dtype=1, Hq=4, b=None, rp=None, scale=0.0):
        return lib.minipic_block_scores(dtype, Hq, REF(b or sb()), REF(rp or rope()), scale, None)
    assert call(dtype=2) == 1
    assert call(Hq=3) == 1
    assert call(Hq=34) == 2                                    # group of 17
    assert call(b=sb(d=96), rp=rope(d=96)) == 2
    assert call(b=sb(B=-1)) == 1
    assert call(b=sb(mb=0)) == 1
    assert call(b=sb(nb=-1)) == 1
    assert call(b=sb(q=None)) == 1
    assert call(b=sb(means=None)) == 1
    assert call(b=sb(means=0x2004)) == 1
    assert call(b=sb(out=0x8004)) == 1
    assert call(b=sb(sl=None)) == 1
    assert call(rp=rope(d=64)) == 1
    assert call(scale=float("nan")) == 1
    assert call(b=sb(B=65536)) == 2
    assert call(b=sb(mb=2 ** 27)) == 2
    assert call(b=sb(B=0)) == 0
    assert lib.minipic_block_scores(1, 4, None, REF(rope()), 0.0, None) == 1
    assert lib.minipic_block_scores(1, 4, REF(sb()), None, 0.0, None) == 1


def test_select_refusals(lib):
    def call(B=1, hkv=2, mb=8, budget=4, first=1, last=1, scores=0x1000, sl=0x2000, out=0x3000):
        return lib.minipic_block_select(REF(mp._Select(scores, sl, out, B, hkv, mb, budget, first, last)), None)
    assert call(budget=0) == 1
    assert call(budget=1) == 1                                 # below keep_first + keep_last
    assert call(first=-1) == 1
    assert call(last=-1) == 1
    assert call(first=2 ** 31 - 1, budget=2 ** 31 - 1) == 1
    assert call(hkv=0) == 1
    assert call(B=-1) == 1
    assert call(mb=0) == 1
    assert call(scores=None) == 1
    assert call(scores=0x1002) == 1
    assert call(out=None) == 1
    assert call(sl=None) == 1
    assert call(mb=2 ** 27) == 2
    assert call(B=2 ** 20, hkv=2 ** 12) == 2
    assert call(B=0) == 0
    assert lib.minipic_block_select(None, None) == 1


def test_selected_refusals(lib):
    def call(dtype=1, Hq=4, p=None, rp=None, db=None, sel=0xC000, S=4, ws=None, n=0, scale=0.0):
        return lib.minipic_attn_decode_selected(dtype, Hq, REF(p or kv()), REF(rp or rope()), REF(db or decode()), scale,
                                                sel, S, ws, n, None)

    def q8(p=None, db=None, **kw):
        return lib.minipic_attn_decode_selected_q8(1, 4, REF(p or kvq8()), REF(rope()), REF(db or decode()), 0.0, 0xC000,
                                                   4, None, 0, None)
    assert call(dtype=7) == 1
    assert call(Hq=3) == 1
    assert call(Hq=34) == 2
    assert call(p=kv(d=96)) == 2
    assert call(p=kv(k=0x1008)) == 1
    assert call(rp=rope(d=64)) == 1
    assert call(rp=rope(f16=None)) == 1                        # bf16 rotates with the fp16 rows
    assert call(db=decode(q=0)) == 1
    assert call(db=decode(out=0x8008)) == 1
    assert call(db=decode(mb=0)) == 1
    assert call(scale=float("inf")) == 1
    assert call(sel=None) == 1
    assert call(sel=0xC002) == 1
    assert call(S=0) == 1 and call(S=-4) == 1
    assert call(S=2 ** 27) == 2
    assert call(db=decode(B=65535), S=2 ** 20) == 2            # 32-bit sums of blocks
    assert call(db=decode(B=65536)) == 2
    assert call(db=decode(B=0)) == 0
    assert q8(p=kvq8(ks=None)) == 1
    assert q8(p=kvq8(vs=0x2202)) == 1
    assert q8(db=decode(B=0)) == 0
    f = lib.minipic_attn_decode_selected_q8
    assert f(1, 4, REF(kvq8()), REF(rope()), None, 0.0, 0xC000, 4, None, 0, None) == 1
    assert f(1, 4, None, REF(rope()), REF(decode()), 0.0, 0xC000, 4, None, 0, None) == 1
    assert lib.minipic_attn_decode_selected(1, 4, REF(kv()), REF(rope()), None, 0.0, 0xC000, 4, None, 0, None) == 1
    size = lib.minipic_attn_decode_selected_workspace_size
    assert size(0, 32, 8, 128, 64, 16) == 0 and size(1, 33, 8, 128, 64, 16) == 0 and size(1, 32, 8, 128, 0, 16) == 0
    assert size(64, 32, 8, 128, 64, 16) > 0


def test_prefix_refusals(lib):
    def gr(cu=0xC000, blocks=0xD000, P=1, most=1, longest=2):
        return mp._Prefixes(cu, blocks, P, most, longest)

    def call(dtype=1, Hq=4, p=None, rp=None, db=None, g=None, ws=None, n=0):
        return lib.minipic_attn_decode_prefix(dtype, Hq, REF(p or kv()), REF(rp or rope()), REF(db or decode()),
                                              REF(g or gr()), 0.0, ws, n, None)
    assert call(dtype=0) == 2                                  # f32
    assert call(dtype=9) == 1
    assert call(Hq=3) == 1
    assert call(p=kv(d=96)) == 2
    assert call(p=kv(nb=0)) == 1
    assert call(rp=rope(f16=None)) == 1
    assert call(db=decode(q=0)) == 1
    assert call(db=decode(mb=0)) == 1
    assert call(g=gr(cu=None)) == 1
    assert call(g=gr(blocks=None)) == 1
    assert call(g=gr(P=-1)) == 1
    assert call(g=gr(most=-1)) == 1
    assert call(g=gr(longest=-1)) == 1
    assert call(db=decode(B=65536)) == 2
    assert call(db=decode(B=0)) == 0
    assert lib.minipic_attn_decode_prefix(1, 4, REF(kv()), REF(rope()), REF(decode()), None, 0.0, None, 0, None) == 1
    size = lib.minipic_attn_decode_prefix_workspace_size
    assert size(0, 32, 8, 128, 512, 1, 64, 256, 16) == 0 and size(8, 33, 8, 128, 512, 1, 8, 256, 16) == 0
    assert size(8, 32, 8, 128, 512, 1, 8, 256, 16) > 0 and size(8, 32, 8, 128, 512, 0, 0, 0, 16) > 0


def test_binding_checks_before_the_call(lib, monkeypatch):
    """Host tensors, wrong dtypes, shapes and strides raise before any call."""
    torch = pytest.importorskip("torch")
    i1, i2 = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    bf, tab = torch.bfloat16, torch.zeros(16, 64)
    both, pool = mp.RopeTable(tab, tab.half()), torch.zeros(4, 2, 16, 64, dtype=bf)
    q, sel = torch.zeros(1, 4, 64, dtype=bf), torch.zeros(1, 2, 3, dtype=torch.int32)
    for f in (lambda: mp.kv_block_means(i1, i1, i2, pool, both, torch.zeros(4, 2, 64, dtype=bf)),
              lambda: mp.block_scores(q, torch.zeros(4, 2, 64, dtype=bf), i2, i2, i1, i1, both),
              lambda: mp.block_select(torch.zeros(1, 2, 4), i1, 2),
              lambda: mp.attn_decode_selected(q, pool, pool, i2, i2, i1, i1, both, sel),
              lambda: mp.attn_decode_prefix(q, pool, pool, i2, i2, i1, i1, both, torch.zeros(2, dtype=torch.int32), i1)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()

    class Here(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = []
    monkeypatch.setattr(mp, "_run", lambda stream, call: calls.append(1))

    def z(*s, dtype=torch.float32):
        return torch.zeros(*s).to(dtype).as_subclass(Here)
    i32, f8 = torch.int32, torch.float8_e4m3fn
    table = mp.RopeTable(z(32, 64), z(32, 64, dtype=torch.float16))

    def refused(f, good, *bad):
        for k, x in bad:
            with pytest.raises((ValueError, TypeError)):
                f(**dict(good, **{k: x}))
    app = dict(cu_new_lens=z(4, dtype=i32), kv_start=z(3, dtype=i32), block_tables=z(3, 6, dtype=i32), rope=table,
               max_new_len=3)
    pool, means = z(5, 2, 16, 64, dtype=bf), z(5, 2, 64, dtype=bf)
    refused(mp.kv_block_means, dict(app, k_pool=pool, means=means), ("cu_new_lens", z(3, dtype=i32)),
            ("kv_start", z(3)), ("block_tables", z(2, 6, dtype=i32)), ("k_pool", z(5, 2, 16, 64)),
            ("means", z(5, 2, 32, dtype=bf)), ("means", z(4, 2, 64, dtype=bf)), ("means", z(5, 2, 64, dtype=f8)),
            ("rope", z(32, 128)), ("means", z(2, 5, 64, dtype=bf).transpose(0, 1)))
    refused(mp.kv_block_means_q8, dict(app, k_pool=z(5, 2, 16, 64, dtype=f8), k_scale=z(5, 2), means=means),
            ("k_pool", pool), ("k_scale", z(5, 3)), ("k_scale", z(5, 2, dtype=bf)), ("means", z(5, 3, 64, dtype=bf)))
    tabs = dict(block_tables=z(3, 6, dtype=i32), block_starts=z(3, 6, dtype=i32), seq_lens=z(3, dtype=i32),
                q_pos=z(3, dtype=i32), rope=table)
    refused(mp.block_scores, dict(tabs, q=z(3, 4, 64, dtype=bf), means=means), ("q", z(3, 4, 64)),
            ("q", z(3, 4, 128, dtype=bf)), ("means", z(5, 2, 64)), ("block_starts", z(3, 5, dtype=i32)),
            ("seq_lens", z(4, dtype=i32)), ("q_pos", z(3)), ("rope", z(32, 128)), ("out", z(3, 2, 7)),
            ("out", z(3, 2, 6, dtype=bf)))
    refused(mp.block_select, dict(scores=z(3, 2, 6), seq_lens=z(3, dtype=i32), budget=4),
            ("scores", z(3, 2, 6, dtype=bf)), ("scores", z(3, 6, 2).transpose(1, 2)), ("seq_lens", z(2, dtype=i32)),
            ("out", z(3, 2, 5, dtype=i32)), ("out", z(3, 2, 4)))
    dec = dict(tabs, q=z(3, 4, 64, dtype=bf), k_pool=pool, v_pool=pool, selected=z(3, 2, 3, dtype=i32))
    refused(mp.attn_decode_selected, dec, ("selected", z(3, 1, 3, dtype=i32)), ("selected", z(3, 2, 3)),
            ("selected", z(3, 3, dtype=i32)), ("v_pool", z(5, 2, 16, 64)), ("q", z(3, 4, 64)), ("out", z(3, 4, 64)),
            ("lse", z(3, 2)), ("rope", z(32, 64)))
    q8 = dict(dec, k_pool=z(5, 2, 16, 64, dtype=f8), v_pool=z(5, 2, 16, 64, dtype=f8), k_scale=z(5, 2), v_scale=z(5, 2))
    refused(mp.attn_decode_selected_q8, q8, ("k_scale", z(5, 3)), ("k_pool", pool), ("selected", z(2, 2, 3, dtype=i32)))
    pre = dict(tabs, q=z(3, 4, 64, dtype=bf), k_pool=pool, v_pool=pool, cu_requests=z(3, dtype=i32),
               prefix_blocks=z(2, dtype=i32), max_requests=2, max_prefix_blocks=1)
    refused(mp.attn_decode_prefix, pre, ("cu_requests", z(2, dtype=i32)), ("prefix_blocks", z(2)), ("q", z(3, 4, 64)),
            ("k_pool", z(5, 2, 16, 64)), ("rope", z(32, 64)), ("prefix_blocks", z(2, 1, dtype=i32)))
    assert not calls   # nothing got as far as a launch
