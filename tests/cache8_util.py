"""Inputs and error bounds for the tests of the 8-bit cache."""

import numpy as np

from oracle import cache8 as c8
import workloads as W

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of a rounding, relative
QK = {"f32": 2.0 ** -24, "bf16": 2.0 ** -11}    # fp32, or fp16 operands of the score product


class Case:
    """Quantised pools, tables with gaps in the starts, ragged lengths; NaN bytes in every slot no length covers."""

    def __init__(self, seed, lens, Hq, Hkv, d, dtype="bf16", base=1e4, pow2=True, spread=1.0, share=True, extra=0,
                 q_lens=None, rows=None):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.dtype, self.base = Hq, Hkv, d, dtype, base
        self.lens = np.array(lens, np.int32)
        B, mb = len(lens), max(1, -(-max(lens) // 16)) + extra
        nb = B * mb + 3
        x = [rng.standard_normal((nb, Hkv, 16, d)) * np.exp2(spread * rng.integers(-6, 7, (nb, Hkv, 1, 1)))
             for _ in range(2)]
        if spread == 1.0:
            x[0] /= np.abs(x[0]).max((2, 3), keepdims=True) / 3.0  # keys of like size: the scales vary through pow2 below
        self.scale = [np.array([[c8.scale_for(t) for t in b] for b in y]) for y in x]
        if not pow2:
            self.scale = [s * rng.uniform(1.0, 1.7, s.shape).astype(np.float32).astype(np.float64) for s in self.scale]
        self.scale = [s.astype(np.float32).astype(np.float64) for s in self.scale]
        self.pool = [c8.encode(y / s[..., None, None]) for y, s in zip(x, self.scale)]
        perm = rng.permutation(nb)[:B * mb].reshape(B, mb)
        self.tables = np.full((B, mb), -1, np.int32)
        self.starts = np.zeros((B, mb), np.int32)
        for r, n in enumerate(lens):
            k = -(-n // 16)
            self.tables[r, :k] = perm[r, :k]
            self.starts[r, :k] = np.arange(k) * 16 + np.cumsum(rng.integers(0, 5, k))
            if share and r and n >= 16 and lens[r - 1] >= 32:   # a full block of the request before, at another offset
                self.tables[r, 0] = self.tables[r - 1, 0]
            if n % 16:
                for p in self.pool:
                    p[self.tables[r, k - 1], :, n % 16:] = 0x7f
        used = np.zeros(nb, bool)
        used[self.tables[self.tables >= 0]] = True
        for p, s in zip(self.pool, self.scale):
            p[~used] = 0xff
            s[~used] = np.nan
        self.max_pos = int(self.starts.max()) + 40
        last = np.maximum(self.lens - 1, 0)
        self.q_pos = (self.starts[np.arange(B), last // 16] + last % 16 + 1).astype(np.int32)
        self.cu = np.arange(B + 1)
        if q_lens is not None:
            self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
            pos = []
            for r, ql in enumerate(q_lens):
                j = lens[r] - ql + np.arange(ql)
                pos.append(self.starts[r, j // 16] + j % 16)
            self.q_pos = np.concatenate(pos).astype(np.int32)
        q = rng.standard_normal((len(self.q_pos), Hq, d)).astype(np.float32)
        self.q_store = q if dtype == "f32" else W.to_bf16_bits(q)
        self.q = (q if dtype == "f32" else W.bf16_bits_to_f32(self.q_store)).astype(np.float64)

    def values(self):
        return [c8.values(p, s) for p, s in zip(self.pool, self.scale)]

    def reference(self, causal=False, **kw):
        k, v = self.values()
        kw.setdefault("max_pos", self.max_pos)
        return c8.attention(self.q, self.cu, self.q_pos, k, v, self.tables, self.starts, self.lens, self.base,
                            causal=causal, **kw)

    def device(self, torch, dev):
        def i32(a):
            return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)
        q = torch.from_numpy(self.q_store.view(np.int16)).to(dev).view(torch.bfloat16) if self.dtype == "bf16" else \
            torch.from_numpy(self.q_store).to(dev)
        pools = [torch.from_numpy(p).to(dev).view(torch.float8_e4m3fn) for p in self.pool]
        scales = [torch.from_numpy(s.astype(np.float32)).to(dev) for s in self.scale]
        return dict(q=q, k_pool=pools[0], v_pool=pools[1], k_scale=scales[0], v_scale=scales[1],
                    block_tables=i32(self.tables), block_starts=i32(self.starts), seq_lens=i32(self.lens),
                    q_pos=i32(self.q_pos), cu=i32(self.cu))


def score_error(ref, dtype, d):
    """Bound of a score's error, per (row, head).  Tensor-core path: each element of the rotated query and of the
    rotated key carries at most three half steps of fp16 (table value, product, sum) on a pair of norm r, so the
    product of the two vectors is off by 2 * 3 * sqrt(2) * 2^-11 |q||k| scale at most; fp32 path: the same with
    2^-24, and the sum over d and the exponent's argument add d + 8 more."""
    c = 6 * 2 ** 0.5 + (0 if dtype == "bf16" else d + 8)
    return c * QK[dtype] * ref["smax"]


def check_attention(got, ref, dtype, d, n_max, what="", p_half=None):
    """|error| of an output element: scores off by eps_s move it by 2 eps_s sum p |v - o| (times e^(2 eps) for the
    second order); each weight is rounded to the product's type (`p_half`, relative, against sum p |v|); sums in
    fp32; one rounding of the output."""
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), what
    eps = score_error(ref, dtype, d)[..., None]
    p_half = p_half if p_half is not None else (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22)
    tol = 2 * eps * np.exp(2 * eps) * ref["spread"] + (p_half + (n_max / 8 + 16) * 2.0 ** -24) * ref["mass"] + \
        HALF[dtype] * np.abs(ref["out"]) + 1e-30
    err = np.abs(got - ref["out"])
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert np.all(err <= tol), f"{what}: error {err[worst]:.3g} at {worst}, bound {tol[worst]:.3g}"
    # the bounds above are worst cases; rounding errors are independent, so their 2-norm stays within half a step
    # of the output's type plus the scores' typical error, d^-1/2 of its bound
    if np.linalg.norm(ref["out"]) > 0 and dtype == "bf16":
        typical = HALF[dtype] + 2 * float(np.median(eps))
        assert np.linalg.norm(err) <= typical * np.linalg.norm(np.abs(ref["out"])), what


def check_weights(got, ref, dtype, d, lens, before, what=""):
    """Block weights: relative error e^(2 eps_s) - 1 plus the roundings of the sum and of the type; entries past a
    request's blocks keep `before`."""
    got = np.asarray(got, np.float64)
    Hkv = got.shape[1]
    G = ref["smax"].shape[1] // Hkv
    for r, n in enumerate(lens):
        nb = -(-int(n) // 16)
        eps = score_error(ref, dtype, d)[r].reshape(Hkv, G).max(1)[:, None]
        w = ref["weights"][r, :, :nb]
        rounding = 2.0 ** -8 + 2.0 ** -8 if dtype == "bf16" else 64 * 2.0 ** -24
        tol = w * (np.expm1(2 * eps) + rounding) + 1e-30
        assert np.all(np.abs(got[r, :, :nb] - w) <= tol), f"{what}: request {r}"
        assert np.all(got[r, :, nb:] == before), f"{what}: entries past request {r} were written"
