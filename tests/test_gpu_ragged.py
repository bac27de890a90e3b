"""GPU tests of attention of ragged chunks over the paged cache (kvq_ragged_attn)
against 64-bit attention over the values that the codes stand for, element by
element within a bound derived from the kernel's stated roundings
(tests/step_cases.py).
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from oracle import formats as OF
from tests import step_cases as SC

pytestmark = pytest.mark.gpu


def query(rng, T, f, spread=1.0):
    return OF.bf16_round((rng.standard_normal((T, f.Hk * f.G, f.D)) * spread).astype(np.float32))


def run(f, n, window=0, f32=True, sm=None, q=None, check=True, seed=1, note="", **kw):
    """One call on a filled cache with n[b] new tokens; the output, checked."""
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    rng = np.random.default_rng(seed)
    q = query(rng, int(cu[-1]), f) if q is None else q
    sm = f.D ** -0.5 if sm is None else sm
    out = f.cache.ragged(SC.bf16(q).cuda(), SC.i32(cu), f.d_tables, SC.i32(f.ctx), f.max_ctx, sm_scale=sm, window=window,
                         out_dtype=torch.float32 if f32 else torch.bfloat16, **kw)
    assert kvq.device_error() == 0
    if check:
        step = int(cu[-1]) == len(n) and window == 0
        SC.assert_within(out, *SC.attention_and_bound(q, cu, f.kv(), sm, f.Hk, window, f.fmt, f32, step), note=note)
    return out


# single tokens, chunks that continue pages, rows before the start, empty sequences
CTX = [1, 2, 17, 64, 65, 0, 130, 200, 33, 5, 300]
NEW = [1, 2, 1, 64, 3, 0, 0, 37, 33, 9, 1]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", SC.ALL)
def test_formats(fmt, D, f32):
    run(SC.Filled(fmt, CTX, D=D), NEW, f32=f32)


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16", "int8c"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_groups(G, fmt):
    """From one row of a block (a single token, G = 1) to a block of 256 and beyond."""
    f = SC.Filled(fmt, [90, 260, 40, 7], Hk=1 if G == 8 else 3, G=G, D=128, seed=G)
    for f32 in (True, False):
        run(f, [1, 260 if G == 1 else 70, 2, 7], f32=f32)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 32, 127, 128, 129, 255, 256, 257, 512])
def test_rows_of_a_block(rows):
    """Row counts around the shapes that a block can have: 16 rows (four copies in a
    slot), 128 (one slot), 256 (two slots), and a block more."""
    f = SC.Filled("fp8", [max(rows, 100), 530], Hk=1, G=1, D=64, seed=rows)
    run(f, [rows, 1], f32=False)
    run(f, [rows, min(rows, 3)], f32=True)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_windows(fmt, window):
    f = SC.Filled(fmt, [1, 64, 200, 333, 90], G=4, D=64)
    run(f, [1, 64, 1, 150, 3], window=window)
    run(f, [1, 3, 9, 150, 90], window=window, f32=False)


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
def test_more_new_tokens_than_context(fmt):
    """Rows that stand before the context's start attend nothing and are zeros."""
    f = SC.Filled(fmt, [3, 0, 70, 1], D=64, G=4)
    for n in ([10, 4, 70, 300], [3, 1, 200, 1]):
        out = run(f, n, f32=fmt == "int8")
        cu = np.concatenate([[0], np.cumsum(n)])
        for b, c in enumerate(f.ctx):
            dead = max(0, n[b] - c)
            assert torch.count_nonzero(out[cu[b]:cu[b] + dead]) == 0
            assert dead == n[b] or torch.count_nonzero(out[cu[b] + dead]) > 0


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_runs_of_rows_that_attend_nothing(fmt):
    """Many blocks in a row without a token to attend, between others, in the share of one
    CTA: no role may wait for a piece that another reaches only later."""
    ctx = [200] + [0] * 30 + [64, 1] + [0] * 9 + [130] + [0] * 40
    n = [3] + [1] * 30 + [64, 2] + [5] * 9 + [1] + [2] * 40
    f = SC.Filled(fmt, ctx, Hk=8, G=1, D=64)
    run(f, n)
    run(f, n[::-1], check=False)
    f = SC.Filled(fmt, [0] * 20 + [50] * 300 + [0] * 20, Hk=4, G=2, D=64)   # one step a piece
    run(f, [1] * 340)


@pytest.mark.parametrize("fmt,f32", [("fp8", False), ("int8", True), ("int8t", False)])
def test_one_long_sequence(fmt, f32):
    """A context that is cut into pieces over many CTAs and joined, alone on the grid:
    a single token, a few, and a chunk of more than one block."""
    f = SC.Filled(fmt, [9001], Hk=1, G=2, D=128)
    for n in ([1], [5], [150]):
        run(f, n, f32=f32)


@pytest.mark.parametrize("fmt,n,G", [("int8", 200, 1), ("int8", 60, 1), ("fp8", 1, 4), ("bf16", 60, 2), ("int8c", 100, 1)])
def test_long_pieces(fmt, n, G):
    """Pieces of many steps in one CTA (sequences that share their blocks, so many that the
    shares hold whole blocks), whose FP32 sums pass through the workspace."""
    B, L = 40, 2900
    f = SC.Filled(fmt, [L], Hk=8, G=G, D=64)
    rng = np.random.default_rng(n)
    rows = [n] * B + ([2] if n == 1 else [])         # not a decode step
    q = query(rng, sum(rows), f)
    cu = np.concatenate([[0], np.cumsum(rows)])
    tables = f.d_tables.expand(len(rows), -1).contiguous()
    kv = f.kv() * len(rows)
    for f32 in (True, False):
        out = f.cache.ragged(SC.bf16(q).cuda(), SC.i32(cu), tables, SC.i32([L] * len(rows)), L, window=L - 1 if n == 1 else 0,
                             out_dtype=torch.float32 if f32 else torch.bfloat16)
        assert kvq.device_error() == 0
        for b in (0, 17, B - 1):                     # some of them, a few rows of each
            pick = [0] if n == 1 else [0, n // 2, n - 1]
            for i in pick:
                p = L - rows[b] + i
                lo = max(0, p - (L - 1) + 1) if n == 1 else 0
                one = [(kv[b][0][lo:p + 1], kv[b][1][lo:p + 1])]
                ref, bound = SC.attention_and_bound(q[cu[b] + i:cu[b] + i + 1], [0, 1], one, f.D ** -0.5, 8, 0, fmt, f32)
                SC.assert_within(out[cu[b] + i:cu[b] + i + 1], ref, bound, note=(fmt, n, b, i, f32))


def test_many_sequences():
    """More sequences than threads of a CTA; most without new tokens, or contexts."""
    rng = np.random.default_rng(0)
    ctx = [int(x) for x in rng.choice([0, 1, 3, 16, 40], 1100)]
    n = [int(x) for x in rng.choice([0, 0, 1, 2], 1100)]
    ctx[0], n[0], ctx[-1], n[-1] = 700, 90, 400, 2
    f = SC.Filled("fp8", ctx, Hk=1, G=2, D=64)
    run(f, n)


@pytest.mark.parametrize("fmt", SC.ALL)
@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_flat_and_sharp_softmax(fmt, spread):
    """Scores that hardly differ, and scores of which one token takes all."""
    f = SC.Filled(fmt, [150, 77], D=128)
    rng = np.random.default_rng(5)
    q = query(rng, 24, f, spread)
    for f32 in (True, False):
        run(f, [20, 4], q=q, f32=f32)


@pytest.mark.parametrize("fmt", ["fp8", "int8", "e5m2"])
@pytest.mark.parametrize("f32", [True, False])
def test_token_scales_far_apart(fmt, f32):
    """Tokens whose V (and K) rows are a thousand times smaller or larger than their
    neighbours', whole steps of zero rows, and rows of tiny values. Per-token scales
    go through a factor of their step; a row that attends only small tokens keeps its
    precision, down to 2^-21 (E5M2: 2^-14) of the step's largest scale."""
    ctx = [200, 64, 70, 40]
    rng = np.random.default_rng(2)
    kf = np.exp2(rng.integers(-3, 1, sum(ctx)).astype(float))
    vf = np.exp2(rng.integers(-10, 1, sum(ctx)).astype(float))
    vf[:64] = 0.0                                   # the first sequence's first step: V is all zero
    kf[200:264] = 0.0                               # the second's: K
    vf[264:334] = 2.0 ** -60                        # the third: everything tiny
    vf[334 + 39] = 2.0 if fmt == "e5m2" else 2.0 ** 10   # the fourth: its last token alone is large
    f = SC.Filled(fmt, ctx, D=64, row_scale=(kf, vf))
    q = query(rng, 30 + 64 + 70 + 39, f, 3.0)
    run(f, [30, 64, 70, 39], q=q, f32=f32)
    run(f, [1, 1, 1, 1], q=q[:4], f32=f32, window=20)


@pytest.mark.parametrize("fmt,lo", [("fp8", 20), ("int8", 21)])
def test_small_tokens_beside_a_large_one(fmt, lo):
    """One token of a step is 2^20 times larger in V than the others, and the query sees
    (almost) none of it: the small ones still come out with 11 bits."""
    D, ctx = 64, 48
    vf, kf = np.full(ctx, 2.0 ** -lo), np.ones(ctx)
    vf[7] = 1.0
    f = SC.Filled(fmt, [ctx], Hk=1, G=1, D=D, row_scale=(kf, vf))
    K = f.kv()[0][0][:, 0]
    q = OF.bf16_round((-40 * K[7] / np.linalg.norm(K[7])).astype(np.float32))[None, None]   # far from token 7
    s = (K @ q[0, 0].astype(np.float64)) * D ** -0.5
    assert s.max() - s[7] > 45 * np.log(2)          # its share is below 2^-24 of the small ones' V
    run(f, [1], q=q, f32=False)


@pytest.mark.parametrize("sm", [0.0, -0.2, 1e-30])
def test_scale_of_the_scores(sm):
    for fmt in ("fp8", "bf16", "int8c"):
        f = SC.Filled(fmt, [80, 130], D=64)
        for f32 in (True, False):
            run(f, [80, 2], sm=sm, f32=f32)


def test_large_and_tiny_queries():
    """The query is scaled row by row; rows of 2^100 or 2^-100 times the usual size keep
    their bits (a score scale brings the scores back)."""
    f = SC.Filled("fp8", [100], D=64)
    rng = np.random.default_rng(1)
    for e in (100, -100, 115):
        q = OF.bf16_round((query(rng, 6, f, 0.5) * 2.0 ** e).astype(np.float32))
        run(f, [6], q=q, sm=float(2.0 ** -e) * 0.125)


@pytest.mark.parametrize("fmt", ["fp8", "bf16", "int8"])
def test_strided_query_and_rows_of_nobody(fmt):
    """The query as a view of a fused projection's output; rows before the first and
    behind the last sequence stay as they were."""
    f = SC.Filled(fmt, [50, 120, 9], D=64, G=2)
    n, T, first = [4, 20, 9], 40, 3
    cu = np.concatenate([[0], np.cumsum(n)]) + first
    rng = np.random.default_rng(3)
    fused = SC.bf16(rng.standard_normal((T, 4 + 2 + 2, f.D)).astype(np.float32)).cuda()
    q = fused[:, :4]
    out = torch.full((T, 4, f.D), 7.0, device="cuda")
    got = f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(f.ctx), f.max_ctx, out=out)
    assert got is out and kvq.device_error() == 0
    ref, bound = SC.attention_and_bound(q.float().cpu().numpy(), cu, f.kv(), f.D ** -0.5, f.Hk, 0, fmt, True)
    rows = slice(first, int(cu[-1]))
    SC.assert_within(out[rows], ref[rows], bound[rows])
    assert (out[:first] == 7).all() and (out[int(cu[-1]):] == 7).all()
    # a place that is 16 bytes off a 32-byte boundary
    flat = torch.empty(T * 4 * f.D + 4, device="cuda")
    odd = flat[4:].view(T, 4, f.D)
    odd.fill_(7.0)
    f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(f.ctx), f.max_ctx, out=odd)
    assert torch.equal(odd, out)


def test_bf16_output_is_near_the_f32_output_and_runs_repeat():
    """The same call gives the same bits; pieces are joined in the order of the tokens."""
    f = SC.Filled("int8", [700, 33, 2000, 5], G=4, D=128)
    for f32 in (True, False):
        a = run(f, [100, 1, 3, 5], f32=f32, check=False)
        for _ in range(3):
            assert torch.equal(a, run(f, [100, 1, 3, 5], f32=f32, check=False))


def test_agrees_with_decode_and_prefill():
    """On batches that the other attention calls take too."""
    f = SC.Filled("fp8", [129, 700, 64, 2000], G=4, D=128)
    rng = np.random.default_rng(4)
    q = query(rng, 4, f)
    a = run(f, [1] * 4, q=q, check=False)
    b = f.cache.decode(SC.bf16(q).cuda(), f.d_tables, SC.i32(f.ctx), f.max_ctx, out_dtype=torch.float32)
    assert (a - b).abs().max() < 2e-5
    q = query(rng, 4 * 30, f)
    a = run(f, [30] * 4, q=q, check=False).view(4, 30, 8, 128).transpose(1, 2)
    qp = SC.bf16(q).cuda().view(4, 30, 8, 128).transpose(1, 2).contiguous()
    b = f.cache.prefill(qp, f.d_tables, SC.i32(f.ctx), f.max_ctx, out_dtype=torch.float32)
    assert (a - b).abs().max() < 2e-5


# ------------------------------------------------------------------ decode steps
# As many new tokens as sequences and no window: the call's single tokens go through the
# decode kernels (8-bit floats: with BF16 output).
STEP_LEN = 16 * 80


def decode_step(fmt, G=2, D=64, seed=0, B=64, Hk=8):
    rng = np.random.default_rng([seed, G])
    ctx = [int(x) for x in rng.choice([0, 1, 16, 17, 100, 128, 129, 300], B)]
    ctx[5], ctx[-1] = 900, 131
    return SC.Filled(fmt, ctx, Hk=Hk, G=G, D=D, width=STEP_LEN // 16, seed=seed)


def step_call(f, n, q, tables=None, ctx=None, **kw):
    cu = np.concatenate([[0], np.cumsum(n)])
    return f.cache.ragged(q if isinstance(q, torch.Tensor) else SC.bf16(q).cuda(), SC.i32(cu), f.d_tables if tables is None else tables,
                          SC.i32(f.ctx if ctx is None else ctx), STEP_LEN, **kw)


@pytest.mark.parametrize("fmt", SC.ALL)
@pytest.mark.parametrize("D,G", [(64, 1), (128, 2), (64, 4), (128, 8)])
def test_decode_steps(fmt, D, G):
    """One token a sequence; and the same shape of call with sequences that bring none or
    several beside it."""
    f = decode_step(fmt, G=G, D=D, B=64 if G < 8 else 24, Hk=8 if G < 8 else 17)
    B = len(f.ctx)
    rng = np.random.default_rng(G)
    q = query(rng, B, f)
    mixed = [1] * B
    mixed[0], mixed[1], mixed[2], mixed[7], mixed[8], mixed[B - 1] = 0, 2, 0, 0, 3, 0
    more = [1] * B                                   # more tokens than sequences: chunks beside single tokens
    more[5], more[9], more[11], more[B - 1] = 37, 0, 2, 9
    q = query(rng, sum(more), f)
    for n in ([1] * B, mixed, more):
        m = sum(n)
        for f32 in (False, True):
            out = step_call(f, n, q[:m], out_dtype=torch.float32 if f32 else torch.bfloat16)
            assert kvq.device_error() == 0
            ref, bound = SC.attention_and_bound(q[:m], np.concatenate([[0], np.cumsum(n)]), f.kv(), D ** -0.5, f.Hk, 0, fmt, f32)
            SC.assert_within(out[:m], ref, bound)


def test_decode_steps_that_are_not_legal_or_not_whole():
    """Contexts, ranges and block ids that are not legal, rows of nobody, a strided query."""
    f = decode_step("fp8")
    B, rng = len(f.ctx), np.random.default_rng(1)
    fused = SC.bf16(rng.standard_normal((B, 16 + 16, 64)).astype(np.float32)).cuda()
    q = fused[:, :16]
    base = step_call(f, [1] * B, q)
    assert kvq.device_error() == 0
    ctx = list(f.ctx)
    ctx[3], ctx[4] = -1, STEP_LEN + 1
    out = step_call(f, [1] * B, q, ctx=ctx)
    assert kvq.device_error() == kvq.DEVERR_CONTEXT
    assert torch.count_nonzero(out[3:5]) == 0 and torch.equal(out[:3], base[:3]) and torch.equal(out[5:], base[5:])
    out = torch.full_like(base, 7.0)                 # the last ten sequences have no tokens
    cu = np.minimum(np.arange(B + 1), B - 10)
    f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(f.ctx), STEP_LEN, out=out)
    assert kvq.device_error() == 0 and torch.equal(out[:B - 10], base[:B - 10]) and (out[B - 10:] == 7).all()
    cu = np.arange(B + 1)
    cu[9] = 100                                      # falls again: two ranges that are not
    out.fill_(7.0)
    f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(f.ctx), STEP_LEN, out=out)
    assert kvq.device_error() == kvq.DEVERR_RANGE
    assert (out[8:10] == 7).all() and torch.equal(out[:8], base[:8]) and torch.equal(out[10:], base[10:])
    t = f.tables.copy()
    t[5, :57] = -1                                   # all pages of sequence 5, one of the last
    t[B - 1, 8] = f.nb
    out = step_call(f, [1] * B, q, tables=torch.from_numpy(t).cuda())
    assert kvq.device_error() == kvq.DEVERR_BLOCK
    assert torch.count_nonzero(out[5]) == 0 and torch.equal(out[:5], base[:5]) and torch.equal(out[6:B - 1], base[6:B - 1])
    K, V = f.kv()[B - 1]
    ref, bound = SC.attention_and_bound(q[B - 1:].float().cpu().numpy(), [0, 1], [(K[:128], V[:128])], 0.125, 8, 0, "fp8", False)
    SC.assert_within(out[B - 1:], ref, bound)


def test_a_captured_decode_step():
    """A graph of a decode step, replayed as one and as a step of another make-up."""
    f = decode_step("int8", G=4)
    B, rng = len(f.ctx), np.random.default_rng(2)
    ws = f.cache.ragged_workspace(B)
    q, out = SC.bf16(query(rng, B, f)).cuda(), torch.zeros(B, 32, 64, dtype=torch.bfloat16, device="cuda")
    cu, ctx = SC.i32(np.arange(B + 1)), SC.i32(f.ctx)
    call = lambda: f.cache.ragged(q, cu, f.d_tables, ctx, STEP_LEN, out=out, workspace=ws)  # noqa: E731
    call()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    n = [0] * B
    n[5], n[-1] = 60, 4
    c0 = np.concatenate([[0], np.cumsum(n)])
    cu.copy_(SC.i32(c0))
    g.replay()
    assert kvq.device_error() == 0
    ref, bound = SC.attention_and_bound(q.float().cpu().numpy(), c0, f.kv(), 0.125, 8, 0, "int8", False)
    SC.assert_within(out, ref, bound)
    cu.copy_(SC.i32(np.arange(B + 1)))
    g.replay()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ bad input on the device
def test_lengths_that_are_not_legal():
    f = SC.Filled("fp8", [50, 60, 70, 80], D=64)
    rng = np.random.default_rng(6)
    q = SC.bf16(query(rng, 20, f)).cuda()
    call = lambda cu, ctx, out: f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(ctx), 70, out=out)  # noqa: E731
    good = torch.full((20, 4, 64), 7.0, device="cuda")
    call([0, 5, 10, 15, 15], [50, 60, 70, 0], good)
    assert kvq.device_error() == 0
    # ranges that fall, or pass the rows: their sequences are skipped, the others are served
    for cu, left in (([0, 5, 3, 3, 3], slice(5, 20)), ([0, 5, 10, 21, 21], slice(10, 20)), ([-1, 5, 10, 10, 10], None),
                     ([0, 5, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], slice(5, 20)), ([0, 5, -2 ** 31, 0, 0], slice(5, 20))):
        out = torch.full((20, 4, 64), 7.0, device="cuda")
        call(cu, [50, 60, 70, 0], out)
        assert kvq.device_error() == kvq.DEVERR_RANGE
        if left is not None:
            assert (out[left] == 7).all() and torch.equal(out[:5], good[:5])
    # contexts: negative, above max_context_len, far above
    for bad in (-1, 71, 2 ** 31 - 1, -2 ** 31):
        out = torch.full((20, 4, 64), 7.0, device="cuda")
        call([0, 5, 10, 15, 15], [50, bad, 70, 0], out)
        assert kvq.device_error() == kvq.DEVERR_CONTEXT
        assert torch.count_nonzero(out[5:10]) == 0 and torch.equal(out[:5], good[:5]) and torch.equal(out[10:15], good[10:15])


@pytest.mark.parametrize("fmt", SC.ALL)
def test_block_ids_outside_the_pool(fmt):
    """Their tokens are not attended; a sequence of none but such blocks gives zeros."""
    f = SC.Filled(fmt, [100, 40, 130], D=64)
    t = f.tables.copy()
    for b, i, v in ((0, 0, -1), (0, 3, f.nb), (1, 0, 2 ** 31 - 1), (1, 1, -2 ** 31), (1, 2, -7), (2, 8, -1)):
        t[b, i] = v
    rng = np.random.default_rng(7)
    q = query(rng, 60, f)
    cu = np.array([0, 20, 40, 60])
    for f32 in (True, False):
        out = f.cache.ragged(SC.bf16(q).cuda(), SC.i32(cu), torch.from_numpy(t).cuda(), SC.i32(f.ctx), f.max_ctx,
                             out_dtype=torch.float32 if f32 else torch.bfloat16)
        assert kvq.device_error() == kvq.DEVERR_BLOCK
        assert torch.count_nonzero(out[20:40]) == 0
        kv = f.kv()
        for b in (0, 2):
            K, V = kv[b]
            keep = np.array([0 <= t[b, i // 16] < f.nb for i in range(f.ctx[b])])
            n, c = 20, f.ctx[b]
            for i in range(n):                        # the tokens left, row by row
                p = c - n + i + 1
                m = keep[:p]
                ref, bound = SC.attention_and_bound(q[cu[b] + i:cu[b] + i + 1], [0, 1], [(K[:p][m], V[:p][m])], f.D ** -0.5,
                                                    f.Hk, 0, fmt, f32)
                SC.assert_within(out[cu[b] + i:cu[b] + i + 1], ref, bound, note=(fmt, b, i))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "e5m2", "int8"])
def test_values_that_are_not_finite(fmt):
    """A NaN or an infinity in a V row (with per-token scales: a scale that is one) shows
    in the rows that attend its token and in no other."""
    f = SC.Filled(fmt, [150, 90], D=64, G=2, Hk=1)
    rng = np.random.default_rng(8)
    q = query(rng, 150 + 20, f)
    refs = [SC.attention_and_bound(q, [0, 150, 170], f.kv(), f.D ** -0.5, 1, 0, fmt, f32) for f32 in (True, False)]
    for t, value in ((100, float("nan")), (3, float("inf")), (149, float("nan"))):
        g = SC.Filled(fmt, [150, 90], D=64, G=2, Hk=1)
        slot = int(g.slots[t])
        if fmt == "bf16":
            g.cache.v[slot // 16, 0, (slot % 16) // 8, 11, slot % 8] = value
        elif fmt == "int8":
            g.cache.v_scale[slot // 16, 0, slot % 16, 0] = value
        else:
            g.cache.v_scale[slot // 16, 0, slot % 16] = value
        for f32, (ref, bound) in zip((True, False), refs):
            out = run(g, [150, 20], q=q, f32=f32, check=False)
            assert (~torch.isfinite(out[t:150])).any(-1).all()       # every row that attends the token
            for rows in (slice(0, t), slice(150, 170)):              # and no other
                SC.assert_within(out[rows], ref[rows], bound[rows])
        win = run(g, [150, 20], q=q, f32=True, check=False, window=10)
        wild = ~torch.isfinite(win).all(-1).all(-1)
        want = torch.zeros(170, dtype=torch.bool, device="cuda")
        want[t:min(t + 10, 150)] = True
        assert torch.equal(wild, want)


# ------------------------------------------------------------------ streams, graphs, workspaces
def test_one_captured_graph_serves_other_lengths():
    """Lengths are read on the device: a graph is replayed with other cu_q, contexts and
    queries, and two graphs replayed in turn share a workspace."""
    f = SC.Filled("fp8", [300, 150, 90, 500], G=4, D=64)
    rng = np.random.default_rng(9)
    T = 130
    ws = f.cache.ragged_workspace(T)
    q, cu, ctx = torch.zeros(T, 8, 64, dtype=torch.bfloat16, device="cuda"), SC.i32([0] * 5), SC.i32([0] * 4)
    out, out2 = torch.zeros(T, 8, 64, device="cuda"), torch.zeros(T, 8, 64, dtype=torch.bfloat16, device="cuda")
    calls = [lambda: f.cache.ragged(q, cu, f.d_tables, ctx, 500, out=out, workspace=ws),
             lambda: f.cache.ragged(q, cu, f.d_tables, ctx, 500, out=out2, workspace=ws, window=40)]
    for c in calls:
        c()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for n, cl in (([1, 1, 1, 1], [300, 150, 90, 500]), ([100, 1, 0, 29], [120, 1, 90, 444]), ([0, 0, 0, 130], [0, 0, 5, 500]),
                  ([0, 0, 0, 0], [1, 2, 3, 4])):
        c0 = np.concatenate([[0], np.cumsum(n)])
        x = query(rng, T, f)
        q.copy_(SC.bf16(x))
        cu.copy_(SC.i32(c0))
        ctx.copy_(SC.i32(cl))
        out.fill_(7.0)
        out2.fill_(7.0)
        graphs[0].replay()
        graphs[1].replay()
        assert kvq.device_error() == 0
        kv = [(k[:c], v[:c]) for (k, v), c in zip(f.kv(), cl)]
        m = int(c0[-1])
        for o, win, f32 in ((out, 0, True), (out2, 40, False)):
            ref, bound = SC.attention_and_bound(x, c0, kv, 64 ** -0.5, f.Hk, win, "fp8", f32)
            if m:
                SC.assert_within(o[:m], ref[:m], bound[:m], note=(n, win))
            assert (o[m:] == 7).all()


def test_another_stream_and_two_at_once():
    f = SC.Filled("int8", [400, 900, 64], G=2, D=128)
    a = run(f, [10, 1, 64], check=False)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [run_on(f, s) for s in (s1, s2, s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for o in outs) and kvq.device_error() == 0


def run_on(f, stream):
    cu = np.array([0, 10, 11, 75])
    q = SC.bf16(query(np.random.default_rng(1), 75, f)).cuda()
    cu_d, ctx = SC.i32(cu), SC.i32(f.ctx)
    ws = f.cache.ragged_workspace(75)
    torch.cuda.synchronize()
    return f.cache.ragged(q, cu_d, f.d_tables, ctx, f.max_ctx, out_dtype=torch.float32, workspace=ws, stream=stream)


def test_binding_refuses():
    f = SC.Filled("fp8", [40], D=64)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu, ctx = SC.i32([0, 3]), SC.i32([40])
    ok = dict(q=q, cu_q=cu, block_tables=f.d_tables, context_lens=ctx, max_context_len=40)
    f.cache.ragged(**ok)
    for bad in (dict(q=q.half()), dict(q=q[:, :2]), dict(q=q[:, ::2]), dict(q=q.transpose(1, 2)), dict(cu_q=cu.long()),
                dict(cu_q=cu[:1]), dict(cu_q=cu.cpu()), dict(context_lens=ctx.long()), dict(block_tables=f.d_tables[:, :1]),
                dict(block_tables=f.d_tables.long()), dict(max_context_len=10 ** 6), dict(window=-1),
                dict(out=torch.empty(3, 4, 64, dtype=torch.float16, device="cuda")), dict(out=torch.empty(2, 4, 64, device="cuda")),
                dict(out=torch.empty(3, 4, 64)), dict(out_dtype=torch.float16), dict(out=q), dict(sm_scale=float("nan")),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), dict(workspace=torch.empty(1 << 20))):
        with pytest.raises(kvq.KvqError):
            f.cache.ragged(**{**ok, **bad})
    assert f.cache.ragged(**{**ok, "window": 2 ** 40}).shape == q.shape       # wider than any context
    assert f.cache.ragged(q[:0], SC.i32([0, 0]), f.d_tables, ctx, 40).shape == (0, 4, 64)
    assert kvq.device_error() == 0


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16"])
def test_waits_that_run_out(fmt):
    """A limit of some hundred cycles ends the waits: rows come out as NaN with
    KVQ_DEVERR_TIMEOUT set, and the next call is right."""
    f = SC.Filled(fmt, [700, 2100, 90], G=4, D=128)
    n = [40, 1, 90]
    run(f, n)
    try:
        kvq.set_wait_limit(300)
        out = run_unchecked(f, n)
        torch.cuda.synchronize()
    finally:
        kvq.set_wait_limit(0)
    flags = kvq.device_error()
    assert flags == kvq.DEVERR_TIMEOUT and torch.isnan(out).any()
    run(f, n)
    run(f, n, f32=False)


def run_unchecked(f, n):
    cu = np.concatenate([[0], np.cumsum(n)])
    q = SC.bf16(query(np.random.default_rng(1), int(cu[-1]), f)).cuda()
    return f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(f.ctx), f.max_ctx, out_dtype=torch.float32)
