"""Refusals of the 8-bit cache, block-weight and eviction calls: every case
fails validation on the host, before any launch (no GPU needed)."""

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
def kvq8(nb=4, hkv=2, bs=16, d=128, k=0x1000, v=0x2000, ks=0x2100, vs=0x2200):
    return mp._KVQ8(k, v, ks, vs, nb, hkv, bs, d)


def rope(d=128, f16=0xB000, b16=0xC000, n=1024):
    return mp._Rope(0x9000, n, d, f16, b16)


def decode(B=1, mb=4, q=0x3000, bt=0x4000, st=0x5000, sl=0x6000, qp=0x7000, out=0x8000):
    return mp._Decode(q, bt, st, sl, qp, B, mb, out, None)


def call_decode(lib, dtype=1, Hq=4, kv=None, rp=None, db=None, bw=None, ws=None, n=0, scale=0.0):
    return lib.minipic_attn_decode_q8(dtype, Hq, REF(kv or kvq8()), REF(rp or rope()), REF(db or decode()), scale, bw,
                                      ws, n, None)


def test_decode_q8_refusals(lib):
    assert call_decode(lib, dtype=7) == 1
    assert call_decode(lib, Hq=3) == 1
    assert call_decode(lib, Hq=34) == 2                       # group of 17
    assert call_decode(lib, kv=kvq8(d=96)) == 2
    assert call_decode(lib, kv=kvq8(bs=32)) == 2
    assert call_decode(lib, kv=kvq8(k=0x1008)) == 1           # misaligned pool
    assert call_decode(lib, kv=kvq8(ks=None)) == 1            # no scales
    assert call_decode(lib, kv=kvq8(vs=0x2202)) == 1          # misaligned scales
    assert call_decode(lib, rp=rope(d=64)) == 1
    assert call_decode(lib, rp=rope(f16=None)) == 1           # bf16 reads the fp16 rows
    assert call_decode(lib, rp=rope(f16=0xB008)) == 1
    assert call_decode(lib, db=decode(q=0)) == 1
    assert call_decode(lib, db=decode(out=0x8008)) == 1
    assert call_decode(lib, db=decode(mb=0)) == 1
    assert call_decode(lib, db=decode(B=-1)) == 1
    assert call_decode(lib, scale=float("nan")) == 1
    assert call_decode(lib, bw=0x8004) == 1                   # misaligned block weights
    assert call_decode(lib, db=decode(B=65536)) == 2
    assert call_decode(lib, db=decode(B=60000, mb=40000)) == 2   # 32-bit sums of blocks
    assert call_decode(lib, kv=kvq8(nb=2 ** 30)) == 2            # 32-bit tile numbers
    for dtype in (0, 1):
        assert call_decode(lib, dtype=dtype, db=decode(mb=2 ** 27)) == 2   # 32-bit numbers of keys
    assert call_decode(lib, Hq=60000, kv=kvq8(nb=1, hkv=60000), db=decode(B=100, mb=10 ** 6)) == 2
    assert call_decode(lib, db=decode(B=0)) == 0
    f = lib.minipic_attn_decode_q8
    assert f(1, 4, None, REF(rope()), REF(decode()), 0.0, None, None, 0, None) == 1
    assert f(1, 4, REF(kvq8()), None, REF(decode()), 0.0, None, None, 0, None) == 1
    assert f(1, 4, REF(kvq8()), REF(rope()), None, 0.0, None, None, 0, None) == 1


def test_decode_weights_refusals(lib):
    def call(dtype=1, Hq=4, rp=None, db=None, bw=0xD000):
        kv = mp._KV(0x1000, 0x2000, 4, 2, 16, 128)
        return lib.minipic_attn_decode_weights(dtype, Hq, REF(kv), REF(rp or rope()), REF(db or decode()), 0.0, bw,
                                               None, 0, None)
    assert call(dtype=5) == 1
    assert call(Hq=5) == 1
    assert call(bw=None) == 1                                  # the weights are what the call is for
    assert call(bw=0xD008) == 1
    assert call(rp=rope(f16=None)) == 1                        # the fp16 rows
    assert call(rp=rope(f16=0xB008)) == 1
    assert call(db=decode(B=65536)) == 2
    assert call(db=decode(B=0)) == 0


def test_workspace_sizes(lib):
    for f in (lib.minipic_attn_decode_q8_workspace_size, lib.minipic_attn_decode_weights_workspace_size):
        assert f(0, 32, 8, 128, 512, 16) == 0 and f(1, 33, 8, 128, 512, 16) == 0
        assert f(64, 32, 8, 128, 512, 16) >= 64 * 32 * 512 * 4   # a raw sum per query head and block
        assert f(1, 4, 2, 64, 1, 16) > 0
        assert f(65535, 128, 8, 128, 65536, 16) > 2 ** 40        # sizes past 32 bits
    g = lib.minipic_attn_prefill_q8_workspace_size
    assert g(8, 32, 8, 128, 512, 416, 16) >= 8 * 416 * 8 * 16 * 128 * 4
    assert g(8, 32, 8, 128, 0, 416, 16) == 0
    assert g(64, 64, 8, 128, 512, 65536, 16) > 2 ** 36


def test_prefill_q8_refusals(lib):
    def pb(B=1, total=16, mq=16, mb=4, q=0x3000, out=0xA000):
        return mp._Prefill(q, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, B, total, mq, mb, out, None)

    def call(dtype=1, Hq=4, kv=None, rp=None, b=None, ws=None, n=0):
        return lib.minipic_attn_prefill_q8(dtype, Hq, REF(kv or kvq8()), REF(rp or rope()), REF(b or pb()), 0.0, ws, n,
                                           None)
    assert call(dtype=0) == 2                                  # f32
    assert call(dtype=9) == 1
    assert call(Hq=3) == 1
    assert call(kv=kvq8(ks=None)) == 1
    assert call(kv=kvq8(nb=0)) == 1
    assert call(rp=rope(f16=None)) == 1
    assert call(b=pb(q=0)) == 1
    assert call(b=pb(mb=0)) == 1
    assert call(b=pb(B=-2)) == 1
    assert call(b=pb(B=0)) == 0 and call(b=pb(total=0)) == 0
    assert lib.minipic_attn_prefill_q8(1, 4, REF(kvq8()), REF(rope()), None, 0.0, None, 0, None) == 1


def test_append_q8_refusals(lib):
    def ab(B=2, total=5, mx=3, mb=4, k=0x3000):
        return mp._Append(k, 0x4000, 0x5000, 0x6000, 0x7000, B, total, mx, mb)

    def call(dtype=1, kv=None, b=None):
        return lib.minipic_kv_append_q8(dtype, REF(kv or kvq8()), REF(b or ab()), None)
    assert call(dtype=2) == 1
    assert call(kv=kvq8(d=80)) == 2
    assert call(kv=kvq8(bs=8)) == 2
    assert call(kv=kvq8(hkv=0)) == 1
    assert call(kv=kvq8(nb=0)) == 1
    assert call(kv=kvq8(ks=None)) == 1
    assert call(kv=kvq8(vs=0x2201)) == 1
    assert call(kv=kvq8(v=0x2004)) == 1
    assert call(b=ab(k=0)) == 1
    assert call(b=ab(k=0x3008)) == 1
    assert call(b=ab(B=-1)) == 1
    assert call(b=ab(mx=-1)) == 1
    assert call(b=ab(mb=0)) == 1
    assert call(b=ab(B=70000)) == 1
    for nothing in (ab(B=0), ab(total=0), ab(mx=0)):
        assert call(b=nothing) == 0
    assert lib.minipic_kv_append_q8(1, None, REF(ab()), None) == 1


def test_evict_refusals(lib):
    def eb(B=1, mb=8, hkv=2, budget=4, first=1, last=1, decay=1.0, w=0x1000, scores=0x2000, out=0x3000):
        return mp._Evict(w, scores, 0x4000, 0x5000, 0x6000, out, 0x7000, 0x8000, 0x9000, 0xA000, 0xB000, B, mb, hkv,
                         budget, first, last, decay)

    def call(dtype=1, b=None):
        return lib.minipic_kv_evict(dtype, REF(b or eb()), None)
    assert call(dtype=3) == 1
    assert call(b=eb(last=0)) == 1                             # the block being written has to stay
    assert call(b=eb(first=-1)) == 1
    assert call(b=eb(budget=1)) == 1                           # below keep_first + keep_last
    assert call(b=eb(first=2 ** 31 - 1, budget=2 ** 31 - 1)) == 1
    assert call(b=eb(decay=float("inf"))) == 1
    assert call(b=eb(decay=-0.5)) == 1
    assert call(b=eb(hkv=0)) == 1
    assert call(b=eb(B=-1)) == 1
    assert call(b=eb(scores=None)) == 1
    assert call(b=eb(out=None)) == 1
    assert call(b=eb(B=0)) == 0
    assert lib.minipic_kv_evict(1, None, None) == 1


def test_binding_checks_types_and_shapes(lib):
    """Host tensors, wrong dtypes and wrong shapes raise before any call."""
    torch = pytest.importorskip("torch")
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc, i2, i1 = torch.ones(4, 2), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, tab = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(16, 64)
    both, p4 = mp.RopeTable(tab, tab.half()), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mp.attn_decode_q8(q, pool, pool, sc, sc, i2, i2, i1, i1, both)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mp.attn_decode_weights(q, p4, p4, i2, i2, i1, i1, both, torch.zeros(1, 2, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        mp.attn_prefill_q8(q, i1, i1, pool, pool, sc, sc, i2, i2, i1, both, 1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mp.kv_append_q8(q[:, :2], q[:, :2], i1, i1, i2, pool, pool, sc, sc)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mp.kv_evict(torch.zeros(1, 4), i2, i2, i1, 4)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """The box has one GPU: a tensor that says it lives on the second one."""
    torch = pytest.importorskip("torch")

    class Far(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="q is on cuda:1, but the current device is cuda:0"):
        mp._args(("q", torch.zeros(2, 3).as_subclass(Far), torch.float32, (2, 3)))


def test_binding_checks_shapes_before_the_call(lib, monkeypatch):
    torch = pytest.importorskip("torch")

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
    i32, f8, bf = torch.int32, torch.float8_e4m3fn, torch.bfloat16
    good = dict(scores=z(2, 4), block_tables=z(2, 4, dtype=i32), block_starts=z(2, 4, dtype=i32),
                seq_lens=z(2, dtype=i32), budget=2, block_weights=z(2, 3, 4))
    for k, bad in (("scores", z(2, 5)), ("block_tables", z(2, 4)), ("block_starts", z(3, 4, dtype=i32)),
                   ("seq_lens", z(3, dtype=i32)), ("block_weights", z(2, 3, 5)),
                   ("block_weights", z(2, 3, 4, dtype=torch.float16)), ("scores", z(4, 2).t())):
        with pytest.raises((ValueError, TypeError)):
            mp.kv_evict(**dict(good, **{k: bad}))
    pools = dict(k_pool=z(5, 2, 16, 64, dtype=f8), v_pool=z(5, 2, 16, 64, dtype=f8), k_scale=z(5, 2), v_scale=z(5, 2))
    dec = dict(q=z(3, 4, 64, dtype=bf), **pools, block_tables=z(3, 6, dtype=i32), block_starts=z(3, 6, dtype=i32),
               seq_lens=z(3, dtype=i32), q_pos=z(3, dtype=i32),
               rope=mp.RopeTable(z(32, 64), z(32, 64, dtype=torch.float16)), block_weights=z(3, 2, 6, dtype=bf))
    for k, bad in (("q", z(3, 4, 128, dtype=bf)), ("q", z(3, 4, 64, dtype=torch.float16)),
                   ("v_pool", z(5, 2, 16, 128, dtype=f8)), ("k_pool", z(5, 2, 16, 64)), ("k_scale", z(5, 3)),
                   ("v_scale", z(2, 5).t()), ("block_tables", z(2, 6, dtype=i32)), ("block_starts", z(3, 5, dtype=i32)),
                   ("seq_lens", z(4, dtype=i32)), ("q_pos", z(3)), ("rope", z(32, 64)),
                   ("rope", mp.RopeTable(z(32, 128), z(32, 128, dtype=torch.float16))),
                   ("block_weights", z(3, 2, 6)), ("block_weights", z(3, 2, 7, dtype=bf)), ("out", z(3, 4, 64)),
                   ("lse", z(3, 2))):
        with pytest.raises((ValueError, TypeError)):
            mp.attn_decode_q8(**dict(dec, **{k: bad}))
    app = dict(k_new=z(7, 2, 64, dtype=bf), v_new=z(7, 2, 64, dtype=bf), cu_new_lens=z(4, dtype=i32),
               kv_start=z(3, dtype=i32), block_tables=z(3, 6, dtype=i32), **pools, max_new_len=3)
    for k, bad in (("k_new", z(7, 3, 64, dtype=bf)), ("v_new", z(7, 2, 64)), ("cu_new_lens", z(3, dtype=i32)),
                   ("kv_start", z(4, dtype=i32)), ("block_tables", z(2, 6, dtype=i32))):
        with pytest.raises((ValueError, TypeError)):
            mp.kv_append_q8(**dict(app, **{k: bad}))
    pre = dict(q=z(7, 4, 64, dtype=bf), cu_q_lens=z(4, dtype=i32), q_pos=z(7, dtype=i32), **pools,
               block_tables=z(3, 6, dtype=i32), block_starts=z(3, 6, dtype=i32), kv_lens=z(3, dtype=i32),
               rope=dec["rope"], max_q_len=3)
    for k, bad in (("q", z(7, 4, 64)), ("cu_q_lens", z(3, dtype=i32)), ("q_pos", z(6, dtype=i32)),
                   ("kv_lens", z(2, dtype=i32)), ("rope", z(32, 64)), ("out", z(7, 4, 64))):
        with pytest.raises((ValueError, TypeError)):
            mp.attn_prefill_q8(**dict(pre, **{k: bad}))
    assert not calls   # nothing got as far as a launch
