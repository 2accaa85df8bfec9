"""How much the decodes over selected blocks and behind prefixes add to their output's own rounding."""

import numpy as np
import pytest

from list_util import f64
from select_util import batch, keys_of, reference
from test_prefix_gpu import all_keys, env, groups, i32, run as run_prefix  # noqa: F401  (env: a fixture)
from test_select_gpu import run

pytestmark = pytest.mark.gpu

# 2-norms relative to the output's, of independent errors, for queries, keys and values of unit variance.  A rounding to
# bf16 is uniform in half a step, 2^-9 .. 2^-8 of the value: 2^-8 / sqrt(3) over the root mean square of a mantissa in
# [1, 2), sqrt(7 / 3), 1.5e-3 (a normal output's mantissas make it 1.66e-3: the tests take it from the reference).  Rotated
# queries and keys in fp16: table, product and sum, three roundings of 1.8e-4 in each of two operands, 4.5e-4 of a score's
# standard deviation, which moves a weight by as much.  Weights in bf16, one rounding each: 1.5e-3; as the sum of two bf16
# numbers 2^-9 of that; in fp16 1.8e-4.
OUT, SCORE, WEIGHT = 1.66e-3, 4.5e-4, 1.48e-3
TWO_PARTS = 1.1 * np.hypot(OUT, SCORE) / OUT                    # 1.14, and a tenth of it for the sample
ONE_PART = 1.1 * np.sqrt(OUT ** 2 + SCORE ** 2 + WEIGHT ** 2) / OUT    # 1.50


def ratio(torch, out, ref):
    """Error of out, relative to that of the exact result rounded once."""
    exact = torch.from_numpy(ref["out"])
    once = (exact.to(out.dtype).double() - exact).norm()
    return float((out.double().cpu() - exact).norm() / once)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (16, 2, 64), (16, 1, 128), (5, 5, 64)])
def test_selected_blocks_round_once(env, kv, Hq, Hkv, d):
    torch, mp, dev = env
    lens = [2000 + 31 * r for r in range(24)]
    t = batch(torch, dev, lens, Hq, Hkv, d, kv, Hq + d)
    n = t["block_tables"].shape[1]
    sel = i32(torch, dev, np.argsort(np.random.default_rng(d).random((len(lens), Hkv, 125)), -1)[..., :64])
    assert n >= 125 and ratio(torch, run(env, t, sel)[0], reference(torch, t, keys_of(torch, t, sel))) <= TWO_PARTS


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (16, 2, 64), (16, 1, 128), (5, 5, 64)])
def test_own_keys_round_once_and_shared_ones_as_the_prefill(env, Hq, Hkv, d):
    torch, mp, dev = env
    t = groups(torch, dev, [1600 + 7 * r for r in range(40)], [0, 40], [100], Hq, Hkv, d, Hq + d)
    ref = reference(torch, t, all_keys(torch, t))
    assert ratio(torch, run_prefix(env, t)[0], ref) <= ONE_PART
    t["blocks"].zero_()
    assert ratio(torch, run_prefix(env, t)[0], ref) <= TWO_PARTS
    assert mp.device_error() == 0
