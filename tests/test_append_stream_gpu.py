"""Appends on a side stream whose inputs that stream is still writing."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_counts_are_read_on_the_stream_of_the_call(q8):
    """Without max_new_len the counts are read after the stream's work, not after the current stream's."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from position_independent_kv_paged_gb300 import _build
    _build.build()
    import position_independent_kv_paged_gb300 as mp
    dev = torch.device("cuda:0")
    n, Hkv, d = 20, 2, 64
    k, v = (torch.randn(n, Hkv, d, device=dev) for _ in range(2))
    tables = torch.tensor([[1, 2]], dtype=torch.int32, device=dev)
    start = torch.zeros(1, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()
    pools = []
    for late in (False, True):
        cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
        written = cu.clone()
        kp, vp = (torch.zeros(3, Hkv, 16, d, device=dev) for _ in range(2))
        more = ()
        if q8:
            kp, vp = kp.to(torch.float8_e4m3fn), vp.to(torch.float8_e4m3fn)
            more = tuple(torch.ones(3, Hkv, device=dev) for _ in range(2))
        append = mp.kv_append_q8 if q8 else mp.kv_append
        append(k, v, cu, start, tables, kp.clone(), vp.clone(), *[x.clone() for x in more])   # nothing loads late below
        if late:
            cu.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            if late:
                torch.cuda._sleep(100_000_000)   # about 50 ms
                cu.copy_(written)
        append(k, v, cu, start, tables, kp, vp, *more, stream=side)
        torch.cuda.synchronize()
        pools.append([kp.float(), vp.float(), *more])
    assert pools[0][0][1:].abs().sum() > 0
    assert all(torch.equal(a, b) for a, b in zip(*pools))
    assert mp.device_error() == 0
