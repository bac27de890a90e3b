"""GPU tests of how many bits kvq_ragged_attn keeps, on caches whose scores and values
are chosen so that little else than one rounding shows. Each tolerance is a sum of
bounds on what is left.

u = 2^-24 is half a step of FP32. The tensor cores round their sums down: less than 2u
of the running sum for each 16 products added to it.
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from oracle import formats as OF
from oracle import paged as OP
from tests import step_cases as SC

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def given(fmt, ctx, K, V, Hk, G, D):
    """A filled cache that holds these rows."""
    f = SC.Filled(fmt, ctx, Hk=Hk, G=G, D=D)
    f.K, f.V = OF.bf16_round(K.astype(np.float32)), OF.bf16_round(V.astype(np.float32))
    if f.static:
        f.static = {s: OF.int8_static_calibrate(x, fmt == "int8c") for s, x in (("k_static", f.K), ("v_static", f.V))}
    f.pool = OP.LogicalPool(fmt, f.nb, Hk, 16, D, **f.static)
    f.pool.append(f.K, f.V, f.slots)
    f.cache = kvq.LayerCache.allocate(fmt, f.dims, **{s: SC.bf16(x).cuda() for s, x in f.static.items()})
    f.poison()
    f.cache.append(SC.bf16(f.K).cuda(), SC.bf16(f.V).cuda(), torch.from_numpy(f.slots).cuda())
    return f


def shared(f, q, n, B, f32, sm, window=0):
    """B sequences of n new tokens each that share the cache's one sequence, and all have
    the query q [n][Hq][D]: so many that a CTA's share holds whole blocks."""
    L = f.ctx[0]
    out = f.cache.ragged(SC.bf16(np.tile(q, (B, 1, 1))).cuda(), SC.i32(np.arange(B + 1) * n), f.d_tables.expand(B, -1).contiguous(),
                         SC.i32([L] * B), L, sm_scale=sm, window=window, out_dtype=torch.float32 if f32 else torch.bfloat16)
    assert kvq.device_error() == 0
    return out.double().cpu().numpy().reshape(B, n, *q.shape[1:])


def exact(f, q, sm, window=0):
    """64-bit attention of the rows q [n][Hq][D], the cache's last n tokens."""
    (K, V), n, L = f.kv()[0], q.shape[0], f.ctx[0]
    out = np.empty(q.shape)
    for i in range(n):
        end = L - n + i + 1
        lo = max(0, end - window) if window else 0
        for h in range(q.shape[1]):
            s = (K[lo:end, h // f.G] @ q[i, h].astype(np.float64)) * sm
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ V[lo:end, h // f.G]
    return out


def row_error(out, ref):
    return float((np.linalg.norm(out - ref, axis=-1) / np.linalg.norm(ref, axis=-1)).max())


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("nats", [12, 20])
@pytest.mark.parametrize("fmt", ["fp8", "int8", "e5m2", "bf16", "int8c"])
def test_small_weights_beside_a_dominant_one(fmt, nats, n):
    """One token takes nearly all of the softmax and has next to no value; thousands of
    others, `nats` below it, make up the output. Their weights keep their bits.

    FP32 output, relative to a row: the dominant score, of at most 22 nats, is rounded
    three times (scale, product, reference): 66u; the others' (at most 3 nats of
    products, 4 sums of 16 each rounded down): 24u; two exponentials 2^-22 each: 8u; the
    sums of O: 6 steps of 64 tokens are at most 72 additions, to a sum half as large on
    average: 72u; with static scales the query's two f16 parts, 2^-22 of 22 nats: 88u.
    Together below 258u, held to 256u. BF16 output: half a step, and 2^-16 for the rest."""
    L, Hk, G, D, B = 8192, 8, 2, 64, 40
    rng = np.random.default_rng(1)
    u = np.where(rng.standard_normal(D) < 0, -1.0, 1.0)
    static = 5.0 if fmt == "int8c" else 1.0          # a channel's scale is every token's: a longer query, shorter keys
    K, V = rng.standard_normal((L, Hk, D)) * 0.2 / static, rng.standard_normal((L, Hk, D))
    K[5], V[5] = (nats + 0.8) / 8 / static * u, 0.0
    f = given(fmt, [L], K, V, Hk, G, D)
    q = np.tile(u * static, (n, Hk * G, 1)).astype(np.float32)
    # a single token a sequence: with a window, which keeps all but the first token, too,
    # as a step without one may go through the decode kernels (BF16 output: with their roundings)
    for f32, window in ((True, 0), (True, L - 1), (False, L - 1)):
        ref = exact(f, q, D ** -0.5, window)
        out = shared(f, q, n, B, f32, D ** -0.5, window)
        e = max(row_error(o, ref) for o in out)
        assert e <= (256 * U if f32 else 2.0 ** -8 + 2.0 ** -16), (f32, window, e)


@pytest.mark.parametrize("rows", [3, 40, 200])
@pytest.mark.parametrize("fmt", SC.ALL)
def test_weights_of_fp32_output(fmt, rows):
    """Token 0 alone has a value and a weight w in (1/2, 1]; tokens 1 and 2 have the weight
    1, the others none at all: a row gives w / (w + 2), (w + 1 where it sees no token 2).

    The score is one product, of less than a unit; it is rounded three times (3u), the
    exponential is 4u off, the weight times the token's scale u, and w moves the result by
    less than itself: 8u (static scales: the query's two f16 parts, 4u more). The sum of
    weights, its reciprocal, and the product with it: 4u. Up to three additions rounded
    down: 6u. Below 24u; a weight of 17 bits is up to 64u off."""
    Hk, G, D = 2, 8, 64
    rng = np.random.default_rng(rows)
    K, V = np.zeros((rows, Hk, D)), np.zeros((rows, Hk, D))
    K[0, :, 0] = 1.0
    K[3:, :, 1] = -1.0
    V[0] = 1.0
    f = given(fmt, [rows], K, V, Hk, G, D)
    q = np.zeros((rows, Hk * G, D), np.float32)
    q[:, :, 0] = -rng.uniform(0.02, 0.98, (rows, Hk * G)) * np.log(2)
    q[:, :, 1] = 2000.0
    q = OF.bf16_round(q)
    ref = exact(f, q, 1.0)
    n, B = rows, 8
    out = shared(f, q, n, B, True, 1.0)
    e = np.abs(out - ref) / np.abs(ref)
    assert e.max() <= 24 * U, e.max() / U


@pytest.mark.parametrize("n", [1, 20, 200])
@pytest.mark.parametrize("fmt", SC.ALL)
def test_sums_of_fp32_output(fmt, n):
    """8,192 tokens of nearly the same weight and of positive values are added up.

    O is kept by the tensor cores for at most 6 steps of 64 tokens, 12 additions each,
    rounded down by less than 2u of a sum half as large on average: 72u. Those sums are
    added in FP32: 8192 / 768 roundings of u, half as large on average: 6u. The scores, of
    up to 0.7 nats of products (4 sums of 16, rounded down) and three roundings: 8u. The
    exponential, the sum of weights, the two slots, the division: 14u. Together 100u; the
    64 steps of a slot, by the tensor cores alone, lose ten times as much as 6 steps do
    (measured: 19u for 6)."""
    L, Hk, G, D, B = 8192, 8, 1, 64, 40
    rng = np.random.default_rng(n)
    K, V = rng.standard_normal((L, Hk, D)), np.abs(rng.standard_normal((L, Hk, D))) + 0.5
    f = given(fmt, [L], K, V, Hk, G, D)
    q = OF.bf16_round((rng.standard_normal((n, Hk * G, D)) * 0.1).astype(np.float32))
    window = L - 1 if n == 1 else 0                  # no decode step
    ref = exact(f, q, D ** -0.5, window)
    out = shared(f, q, n, B, True, D ** -0.5, window)
    e = np.abs(out - ref) / ref
    assert e.max() <= 100 * U, e.max() / U


@pytest.mark.parametrize("fmt", SC.ALL)
@pytest.mark.parametrize("D,window", [(128, 0), (64, 90)])
def test_bf16_output_is_rounded_once(fmt, D, window):
    """BF16 output is the rounding of what FP32 output holds: all that is rounded on the way
    is a weight, to 16 bits and more: it is off by e = 2^-17 of itself at most. A value that
    is off by e of itself rounds otherwise than the exact one where the border lies
    between, for a share of 2 e / 2^-8 of the values on average: 0.4%, held to 1%. It is off
    by half a step, and sum_t w_t |V_t| e <= 2^-17 max |V| (what FP32 output is off by,
    too: some 2^-19 of it): a value may be far smaller than that sum, so the share says
    nothing of single values, and this bound is theirs."""
    f = SC.Filled(fmt, [700, 333, 90], G=4, D=D, seed=3)
    n = [130, 40, 3]
    cu = np.concatenate([[0], np.cumsum(n)])
    q = OF.bf16_round(np.random.default_rng(4).standard_normal((cu[-1], 8, D)).astype(np.float32))
    args = (SC.bf16(q).cuda(), SC.i32(cu), f.d_tables, SC.i32(f.ctx), f.max_ctx)
    lo = f.cache.ragged(*args, window=window)
    hi = f.cache.ragged(*args, window=window, out_dtype=torch.float32)
    assert kvq.device_error() == 0
    ref, _ = SC.attention_and_bound(q, cu, f.kv(), D ** -0.5, 2, window, fmt, True)
    top = max(np.abs(v).max() for _, v in f.kv())
    for want in (SC.bf16(ref).float(), hi.cpu().bfloat16().float()):
        got = lo.cpu().float()
        off = got != want
        assert off.double().mean() <= 0.01, float(off.double().mean())
        assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -16 * top).all()


@pytest.mark.parametrize("fmt", ["fp8", "bf16", "int8c"])
@pytest.mark.parametrize("n", [17, 130])
def test_long_contexts_lose_nothing_on_the_way(fmt, n):
    """524,288 tokens (512 of them, again and again), positive values, BF16 output: the
    output's own rounding cancels out over 100,000 values and more, what the sums lose
    does not. They are kept by the tensor cores for at most 128 steps of 64 tokens, 8
    additions each, rounded down by less than 2u of a sum half as large on average: 1024u
    of a value. The mean of 2^-9 at most over 17,408 values and more is off by less than
    2^-15 = 512u (4 standard deviations of a 17,408th of 2^-9). Together 1536u."""
    distinct, L, Hk, G, D, B = 512, 524288, 8, 1, 128, 20
    rng = np.random.default_rng(n)
    K, V = rng.standard_normal((distinct, Hk, D)), np.abs(rng.standard_normal((distinct, Hk, D))) + 0.5
    f = given(fmt, [distinct], K, V, Hk, G, D)
    W = L // 16
    d = kvq.dims(f.nb, Hk, Hk * G, D, W)
    cache = kvq.LayerCache(fmt, d, f.cache.k, f.cache.v, f.cache.k_scale, f.cache.v_scale)
    table = torch.from_numpy(np.tile(f.tables[0, :distinct // 16], W * 16 // distinct)).cuda().expand(B, -1).contiguous()
    q = OF.bf16_round(rng.standard_normal((n, Hk * G, D)).astype(np.float32))
    out = cache.ragged(SC.bf16(np.tile(q, (B, 1, 1))).cuda(), SC.i32(np.arange(B + 1) * n), table, SC.i32([L] * B), L)
    assert kvq.device_error() == 0
    out = out.double().cpu().numpy().reshape(B, n, Hk * G, D)
    (K, V), ref = f.kv()[0], np.empty(q.shape)
    for i in range(n):
        seen = (np.arange(distinct) < distinct - n + i + 1) + (L // distinct - 1.0)     # times each token is attended
        for h in range(Hk):
            s = (K[:, h] @ q[i, h].astype(np.float64)) * D ** -0.5
            w = np.exp(s - s.max()) * seen
            ref[i, h] = (w / w.sum()) @ V[:, h]
    for o in out:
        assert abs(np.mean(o / ref - 1)) <= 1536 * U, np.mean(o / ref - 1)


@pytest.mark.parametrize("fmt", ["fp8", "int8", "e5m2", "bf16"])
def test_values_of_any_size(fmt):
    """Tokens whose values are 2^100 or 2^-100, alone and beside ordinary ones; a row that
    does not attend the large ones (they come later, or before its window) keeps its bits.
    BF16 output: half a step and a little; FP32 output: within 2^-17 of a row, more than
    the 130u that scores of this size and two steps of sums may cost."""
    n, ctx = 60, 200
    for small, large in ((1.0, 2.0 ** 100), (2.0 ** -100, 2.0 ** -100), (2.0 ** -60, 1.0), (2.0 ** 100, 2.0 ** 100)):
        vf = np.full(ctx, small)
        vf[170] = large
        f = SC.Filled(fmt, [ctx], Hk=2, G=4, D=64, row_scale=(np.ones(ctx), vf))
        q = OF.bf16_round(np.random.default_rng(3).standard_normal((n, 8, 64)).astype(np.float32))
        for window in (0, 20):
            ref = exact(f, q, 0.125, window)
            for f32 in (True, False):
                out = shared(f, q, n, 3, f32, 0.125, window)
                assert max(row_error(o, ref) for o in out) <= (2.0 ** -17 if f32 else 2.0 ** -8 + 2.0 ** -16), (small, large, window, f32)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("fmt", ["fp8", "int8", "e5m2"])
def test_scales_below_zero(fmt, f32):
    """The quantizers write no negative scale, but a cache may be filled by other means:
    negative V scales turn the output round, and one of minus infinity shows in the rows
    that attend its token and in no other."""
    f = SC.Filled(fmt, [150], D=64, G=2, Hk=1)
    q = SC.bf16(np.random.default_rng(8).standard_normal((150, 2, 64))).cuda()
    dt = torch.float32 if f32 else torch.bfloat16
    call = lambda: f.cache.ragged(q, SC.i32([0, 150]), f.d_tables, SC.i32([150]), 150, out_dtype=dt)  # noqa: E731
    want = call()
    scale = f.cache.v_scale[..., 0] if fmt == "int8" else f.cache.v_scale
    scale.neg_()
    assert torch.equal(call(), -want)
    scale.neg_()
    t = 100
    slot = int(f.slots[t])
    scale[slot // 16, 0, slot % 16] = -float("inf")
    out = call()
    assert (~torch.isfinite(out[t:])).any(-1).all()
    assert torch.equal(out[:t], want[:t])
    assert kvq.device_error() == 0


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("fmt", ["fp8", "int8", "e5m2", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_keys_that_are_not_finite(fmt, f32, bad):
    """A K row (with per-token scales: its scale) that is not finite, or so large that
    scores overflow, changes no row that does not attend its token."""
    f = SC.Filled(fmt, [150], D=64, G=2, Hk=1)
    q = SC.bf16(np.random.default_rng(8).standard_normal((150, 2, 64))).cuda()
    dt = torch.float32 if f32 else torch.bfloat16
    call = lambda w: f.cache.ragged(q, SC.i32([0, 150]), f.d_tables, SC.i32([150]), 150, out_dtype=dt, window=w)  # noqa: E731
    want = {w: call(w) for w in (0, 30)}
    t = 100
    slot = int(f.slots[t])
    if fmt == "bf16":
        f.cache.k[slot // 16, 0, (slot % 16) // 8, :, slot % 8, :] = bad
    else:
        scale = f.cache.k_scale[..., 0] if fmt == "int8" else f.cache.k_scale
        scale[slot // 16, 0, slot % 16] = bad
    for w in (0, 30):
        out = call(w)
        assert torch.equal(out[:t], want[w][:t])
        if w:
            assert torch.equal(out[t + w:], want[w][t + w:])
    assert kvq.device_error() == 0
