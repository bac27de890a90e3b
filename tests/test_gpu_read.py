"""GPU tests of the dequantizing read-back (kvq_read): FP32 values bit for bit those
that the oracle's codes stand for (code * scale has at most 17 bits; the low-bit
formats' code * s + z is rounded once), BF16 values their rounding.
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from oracle import formats as OF
from oracle import kivi as OK
from tests import step_cases as SC
from tests.test_gpu_kivi import _build

pytestmark = pytest.mark.gpu


def expect(kv, starts, n):
    """float32 rows (K, V): the 64-bit values, rounded once."""
    return [np.concatenate([x[s:s + m] for x, s, m in zip((a[w] for a in kv), starts, n)]).astype(np.float32) for w in (0, 1)]


def check(cache, tables, kv, starts, n, pad=0, first=0):
    cu = np.concatenate([[0], np.cumsum(n)]) + first
    total = int(cu[-1]) + pad
    ref = expect(kv, starts, n)
    shape = (total, cache.dims.n_kv_heads, cache.dims.head_dim)
    for dt in (torch.float32, torch.bfloat16):
        out = [torch.full(shape, 7.0, dtype=dt, device="cuda") for _ in range(2)]
        got = cache.read(tables, SC.i32(starts), SC.i32(cu), total, k_out=out[0], v_out=out[1])
        assert got[0] is out[0] and got[1] is out[1] and kvq.device_error() == 0
        for o, r in zip(out, ref):
            rows = o[first:int(cu[-1])].float().cpu().numpy()
            assert np.array_equal(rows, r if dt == torch.float32 else OF.bf16_round(r))
            assert (o[:first] == 7).all() and (o[int(cu[-1]):] == 7).all()


CTX = [1, 16, 17, 100, 255, 3, 64]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", SC.ALL)
def test_formats(fmt, D):
    f = SC.Filled(fmt, CTX, D=D, Hk=3, G=1)
    kv = f.kv()
    check(f.cache, f.d_tables, kv, [0] * 7, CTX)                                           # whole contexts
    check(f.cache, f.d_tables, kv, [0, 5, 16, 33, 200, 2, 63], [1, 9, 1, 40, 55, 0, 1], pad=21, first=5)   # runs, rows of nobody
    check(f.cache, f.d_tables, kv, [0] * 7, [0] * 7, pad=3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["kivi2", "kivi4"])
def test_low_bit_groups(fmt, D):
    w, bits, cache, qt, rt, hist, groups, res = _build(fmt, [128, 400, 60, 1025], D=D)
    tables = torch.from_numpy(qt).cuda()
    kv = []
    for k, v in hist:
        K, V = OK.dequantize_sequence(OK.quantize_sequence(k.float().numpy(), v.float().numpy(), bits=bits))
        kv.append((K, V))
    n = [128 * g for g in groups]
    check(cache, tables, kv, [0] * 4, n)
    check(cache, tables, kv, [5, 127, 0, 1000], [100, 130, 0, 24], pad=2, first=1)


@pytest.mark.parametrize("Hk", [1, 2, 8])
def test_many_sequences(Hk):
    """Runs of no, one and many tokens; several sequences inside one window of 16 rows, and
    more of them than a search step takes."""
    rng = np.random.default_rng(Hk)
    ctx = [int(x) for x in rng.choice([1, 2, 5, 40, 90], 300)]
    f = SC.Filled("int8", ctx, Hk=Hk, G=1, D=64)
    starts = [int(rng.integers(0, c)) for c in ctx]
    n = [int(rng.choice([0, 1, c - s])) for c, s in zip(ctx, starts)]
    check(f.cache, f.d_tables, f.kv(), starts, n, pad=40)


def test_one_of_the_two_and_odd_places():
    f = SC.Filled("fp8", [77, 30], D=128)
    ref = expect(f.kv(), [3, 0], [70, 30])
    starts, cu = SC.i32([3, 0]), SC.i32([0, 70, 100])
    for dt in (torch.float32, torch.bfloat16):
        k, none = f.cache.read(f.d_tables, starts, cu, 100, v_out=False, out_dtype=dt)
        assert none is None and np.array_equal(k.float().cpu().numpy(), ref[0] if dt == torch.float32 else OF.bf16_round(ref[0]))
        none, v = f.cache.read(f.d_tables, starts, cu, 100, k_out=False, out_dtype=dt)
        assert none is None and np.array_equal(v.float().cpu().numpy(), ref[1] if dt == torch.float32 else OF.bf16_round(ref[1]))
        # a place 16 bytes off a 32-byte boundary
        step = 16 // v.element_size()
        odd = torch.empty(v.numel() + step, dtype=dt, device="cuda")[step:].view(v.shape)
        assert torch.equal(f.cache.read(f.d_tables, starts, cu, 100, k_out=False, v_out=odd)[1], v)


def test_what_is_not_there_reads_as_zeros():
    f = SC.Filled("fp8", [40, 50, 60], D=64)
    t = f.tables.copy()
    t[0, 1], t[1, 0], t[1, 3] = -1, f.nb, 2 ** 31 - 1
    W = t.shape[1]
    tables = torch.from_numpy(t).cuda()
    ref = expect(f.kv(), [0, 0, 0], [40, 50, 60])
    dead = np.zeros(150, bool)
    dead[16:32] = dead[40:56] = dead[88:90] = True
    got = f.cache.read(tables, SC.i32([0, 0, 0]), SC.i32([0, 40, 90, 150]), 150, out_dtype=torch.float32)
    assert kvq.device_error() == kvq.DEVERR_BLOCK
    for o, r in zip(got, ref):
        assert np.array_equal(o.cpu().numpy(), np.where(dead[:, None, None], 0, r))
    # starts outside the table
    for bad in (-1, 16 * W, 2 ** 31 - 1, -2 ** 31, 16 * W - 2):
        got = f.cache.read(f.d_tables, SC.i32([0, bad, 0]), SC.i32([0, 5, 9, 20]), 20, out_dtype=torch.float32)
        assert kvq.device_error() == kvq.DEVERR_CONTEXT
        for o, r in zip(got, ref):
            o = o.cpu().numpy()
            first = 2 if bad == 16 * W - 2 else 0
            assert np.array_equal(o[:5], r[:5]) and np.array_equal(o[9:], r[90:101]) and (o[5 + first:9] == 0).all()


def test_ranges_that_are_not_legal():
    f = SC.Filled("int8", [40, 50], D=64)
    for cu in ([0, 30, 20], [-5, 10, 20], [0, 10, 21], [0, 2 ** 31 - 1, 20], [20, 10, 0], [0, -2 ** 31, 20]):
        out = [torch.full((20, 2, 64), 7.0, device="cuda") for _ in range(2)]
        f.cache.read(f.d_tables, SC.i32([0, 0]), SC.i32(cu), 20, k_out=out[0], v_out=out[1])
        assert kvq.device_error() & kvq.DEVERR_RANGE
    check(f.cache, f.d_tables, f.kv(), [0, 0], [40, 50])


def test_captured_and_on_another_stream():
    f = SC.Filled("fp8", [100, 64], D=128)
    kv = f.kv()
    starts, cu = SC.i32([0, 0]), SC.i32([0, 50, 100])
    out = [torch.zeros(100, 2, 128, device="cuda") for _ in range(2)]
    call = lambda s=None: f.cache.read(f.d_tables, starts, cu, 100, k_out=out[0], v_out=out[1], stream=s)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for st, n in (([0, 0], [50, 50]), ([60, 1], [40, 60]), ([3, 0], [0, 64])):
        starts.copy_(SC.i32(st))
        cu.copy_(SC.i32(np.concatenate([[0], np.cumsum(n)])))
        g.replay()
        ref = expect(kv, st, n)
        assert all(np.array_equal(o[:sum(n)].cpu().numpy(), r) for o, r in zip(out, ref))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out[0].zero_()
    torch.cuda.synchronize()
    call(s)
    s.synchronize()
    assert np.array_equal(out[0][:64].cpu().numpy(), expect(kv, [3, 0], [0, 64])[0])


def test_binding_refuses():
    f = SC.Filled("fp8", [40], D=64)
    ok = dict(block_tables=f.d_tables, starts=SC.i32([0]), cu_tokens=SC.i32([0, 9]), total_tokens=9)
    out = torch.empty(9, 2, 64, device="cuda")
    for bad in (dict(block_tables=f.d_tables.long()), dict(block_tables=f.d_tables[:, :2]), dict(starts=SC.i32([0, 0])),
                dict(starts=SC.i32([0]).long()), dict(cu_tokens=SC.i32([0])), dict(cu_tokens=SC.i32([0, 9]).cpu()),
                dict(total_tokens=-1), dict(k_out=False, v_out=False), dict(k_out=out, v_out=out), dict(k_out=out[:8]),
                dict(k_out=out, v_out=out.bfloat16()), dict(k_out=out.half()), dict(out_dtype=torch.float16),
                dict(k_out=out.cpu()), dict(k_out=out.transpose(0, 1))):
        with pytest.raises(kvq.KvqError):
            f.cache.read(**{**ok, **bad})
    k, v = f.cache.read(f.d_tables, ok["starts"], SC.i32([0, 0]), 0)
    assert k.shape == v.shape == (0, 2, 64) and kvq.device_error() == 0
