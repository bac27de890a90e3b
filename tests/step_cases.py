"""Helpers of the GPU tests of a serving step's calls: a paged cache filled through
kvq_append from seeded rows, the values that it stands for (the oracle's pool),
and error bounds of attention over it, derived from the roundings that the
kernels state.
"""

import numpy as np
import torch

from int8_quantized_paged_quantize_b200 import kvq
from oracle import formats as OF
from oracle import paged as OP

ALL = ["fp8", "int8", "e5m2", "bf16", "int8c", "int8t"]


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Filled:
    """A cache whose sequence b holds ctx[b] tokens on shuffled blocks. Blocks that no
    sequence has, table entries behind a context and tokens behind it in its last
    page hold NaN patterns (codes and scales), which no result may show."""

    def __init__(self, fmt, ctx, Hk=2, G=2, D=64, seed=0, scale=1.0, row_scale=None, extra=3, width=0):
        rng = np.random.default_rng([seed, Hk, G, D])
        self.fmt, self.ctx, self.Hk, self.G, self.D = fmt, list(ctx), Hk, G, D
        pages = [(c + 15) // 16 for c in ctx]
        nb, W = sum(pages) + extra, max(pages + [1, width - 1]) + 1
        perm = rng.permutation(nb)
        self.tables = np.full((len(ctx), W), perm[-1], dtype=np.int32)      # a block of nobody
        at = 0
        for b, p in enumerate(pages):
            self.tables[b, :p] = perm[at:at + p]
            at += p
        self.nb, self.dims = nb, kvq.dims(nb, Hk, Hk * G, D, W)
        n = sum(ctx)
        shift = 0.3 if fmt.startswith("int8") else 0.0
        self.K, self.V = (OF.bf16_round((rng.standard_normal((n, Hk, D)) * scale + shift).astype(np.float32)) for _ in range(2))
        if row_scale is not None:                     # factors of each token's K and V rows
            self.K = OF.bf16_round(self.K * row_scale[0][:n, None, None].astype(np.float32))
            self.V = OF.bf16_round(self.V * row_scale[1][:n, None, None].astype(np.float32))
        self.slots = np.concatenate([self.tables[b][np.arange(c) // 16].astype(np.int64) * 16 + np.arange(c) % 16
                                     for b, c in enumerate(ctx)] + [np.zeros(0, np.int64)])
        static = {}
        if fmt in ("int8c", "int8t"):
            static = {s: OF.int8_static_calibrate(x, fmt == "int8c") for s, x in (("k_static", self.K), ("v_static", self.V))}
        self.static = static
        self.pool = OP.LogicalPool(fmt, nb, Hk, 16, D, **static)
        self.pool.append(self.K, self.V, self.slots)
        self.cache = kvq.LayerCache.allocate(fmt, self.dims, **{s: bf16(x).cuda() for s, x in static.items()})
        self.poison()
        if n:
            self.cache.append(bf16(self.K).cuda(), bf16(self.V).cuda(), torch.from_numpy(self.slots).cuda())
        self.d_tables = torch.from_numpy(self.tables).cuda()

    def poison(self):
        c = self.cache
        if self.fmt == "bf16":
            c.k.fill_(float("nan"))
            c.v.fill_(float("nan"))
        else:
            c.k.fill_(0x7F)                          # E4M3 and E5M2 NaN, an INT8 code like any
            c.v.fill_(0x7F)
        if self.fmt in ("fp8", "e5m2", "int8"):
            c.k_scale.fill_(float("nan"))
            c.v_scale.fill_(float("nan"))

    def kv(self):
        return [self.pool.gather(self.tables[b], c) for b, c in enumerate(self.ctx)]

    @property
    def max_ctx(self):
        return max(self.ctx + [1])


def attention_and_bound(q, cu, kv, sm_scale, Hk, window, fmt, f32, step=False):
    """(out, bound) [T][Hq][D] float64 of ragged attention: the value, and how far the
    kernel may be from it by its stated roundings:
      scores   FP32 output: the operands are exact (static INT8: the query times the
               scale in two f16 parts, 2^-22), sums in FP32. BF16 output: K (static
               INT8: the query) rounded to f16, half a step 2^-11 a product; a BF16
               cache is exact. In both: 2^-13 of the products' sum for sums of up to
               128 terms, kept to at least 20 bits.
      weights  half a step of f16 (BF16 cache: of bf16): 2^-11 (2^-8); FP32 output
               twice that many bits, 2^-22 (BF16 cache: 2^-22 and more). 2^-20 for the exponential and the sum.
      V        BF16 output with per-token scales: 2^-11.
      output   half a step of bf16 2^-8, or of FP32.
    A score off by at most d moves a weight by a factor of at most e^(2d).

    Small weights (not with a BF16 cache, whose weights have FP32's range): a weight is
    held in f16 as P = 2^(s - m + e), e the exponent that its step of 64 tokens takes out
    of V (static INT8: 0), so below 2^-14 its error is not relative: half of f16's
    smallest step, 2^-25. In the output that is
      2^-25 sum_t |V_t| 2^-e(t) * 2^m / sum_u 2^s(u),   m <= max_u (s(u) + e(u)),
    and with 2^m <= sum_u 2^(s(u) + e(u)):  2^-25 sum_t |V_t| 2^-e(t) * sum_u w_u 2^e(u).
    2^e is a power of two above the step's largest scale, less a constant: at most twice
    as far apart between two steps as the scales are, hence the factor 2.

    step: a decode step with an INT8 cache, whose decode kernel holds a weight times its
    token's scale as 24 bits of fixed point below the largest weight times the largest
    scale of a tile of 128 tokens: in the output
      2^-24 w_max sum_t (s_max / s_t) |V_t|,
    and scales are at most twice as far apart as the rows' largest values."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    G = Hq // Hk
    out, bound = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    tok = fmt in ("fp8", "e5m2", "int8")
    ds = 2.0 ** -18 + (0.0 if f32 or fmt == "bf16" else 2.0 ** -11)
    dp = 2.0 ** -22 if f32 else 2.0 ** (-8 if fmt == "bf16" else -11)
    dv = 2.0 ** -11 if tok and not f32 else 0.0
    do = 2.0 ** -23 if f32 else 2.0 ** -8
    for b, (K, V) in enumerate(kv):
        n, ctx = int(cu[b + 1] - cu[b]), K.shape[0]
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            top = np.ones(ctx)                        # 2^e of each token's step, up to a constant
            if tok:
                size = np.abs(v).max(-1)
                for t in range(0, ctx, 64):
                    top[t:t + 64] = size[t:t + 64].max() or 1e-30
            for i in range(n):
                r, p = cu[b] + i, ctx - n + i
                lo = max(0, p - window + 1) if window else 0
                if p < 0:
                    out[r, h] = bound[r, h] = 0.0
                    continue
                kk, vv = k[lo:p + 1], v[lo:p + 1]
                s = (kk @ q[r, h]) * sm_scale
                d = ds * abs(sm_scale) * (np.abs(kk) @ np.abs(q[r, h])).max()
                w = np.exp(s - s.max())
                w /= w.sum()
                out[r, h] = w @ vv
                a = w @ np.abs(vv)
                bound[r, h] = a * (np.expm1(2 * d) + dp + dv + 2.0 ** -20) * 1.01 + np.abs(out[r, h]) * do + 1e-30
                if step and fmt == "int8":
                    size = np.maximum(np.abs(v[:p + 1]).max(-1), 1e-30)
                    far = np.concatenate([size[t:t + 128].max() / size[t:t + 128] for t in range(0, p + 1, 128)])
                    bound[r, h] += 2.0 ** -23 * w.max() * (far @ np.abs(v[:p + 1]))
                if fmt != "bf16":
                    bound[r, h] += 2.0 ** -24 * ((1 / top[lo:p + 1]) @ np.abs(vv)) * (w @ top[lo:p + 1])
    return out, bound


def assert_within(got, out, bound, note=""):
    got = got.double().cpu().numpy()
    e = np.abs(got - out)
    ok = e <= bound
    bound = np.maximum(bound, 1e-300)
    assert np.isfinite(got).all(), (note, "not finite")
    assert ok.all(), (note, "worst", float((e / bound).max()), "at", np.unravel_index(int((e / bound).argmax()), e.shape))
    return float((e / bound).max())
