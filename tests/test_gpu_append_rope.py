"""GPU tests of the cache write with rotary embedding (kvq_append_rope): the rotated
query bit for bit (float32 products and sums rounded one by one, then BF16) and
within the roundings of the 64-bit rotation; codes and scales bit for bit those
of the oracle's pool for the rotated keys, and those of kvq_append.
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from oracle import formats as OF
from oracle import paged as OP
from oracle import rope as OR
from tests import step_cases as SC

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, fmt, T, Hk=2, G=2, D=64, rotary=None, interleaved=False, seed=0, nb=24, max_pos=600, slots=None,
                 fused=True):
        rng = np.random.default_rng([seed, T, Hk, G, D])
        self.fmt, self.T, self.Hk, self.Hq, self.D, self.nb = fmt, T, Hk, Hk * G, D, nb
        self.rotary, self.interleaved = rotary or D, interleaved
        x = rng.standard_normal((T, self.Hq + 2 * Hk, D)).astype(np.float32) + np.float32(0.3 * fmt.startswith("int8"))
        x[:, self.Hq:, ::31] *= 6
        self.x = OF.bf16_round(x)
        fused_d = SC.bf16(self.x).cuda()
        self.q, self.k, self.v = fused_d[:, :self.Hq], fused_d[:, self.Hq:self.Hq + Hk], fused_d[:, self.Hq + Hk:]
        if not fused:
            self.q, self.k, self.v = (y.contiguous() for y in (self.q, self.k, self.v))
        self.pos = rng.integers(0, max_pos, T)
        self.table = OR.table(max_pos, self.rotary)
        self.slots = np.arange(T, dtype=np.int64) if slots is None else np.asarray(slots, dtype=np.int64)
        kr = OR.rotate(self.x[:, self.Hq:self.Hq + Hk], self.pos, self.table, interleaved)
        self.q_ref = OR.rotate(self.x[:, :self.Hq], self.pos, self.table, interleaved)
        static = {}
        if fmt in ("int8c", "int8t"):
            static = {s: OF.int8_static_calibrate(y, fmt == "int8c") * np.float32(0.8) for s, y in
                      (("k_static", kr), ("v_static", self.x[:, self.Hq + Hk:]))}
            static = {s: OF.bf16_round(y) for s, y in static.items()}      # below the largest: some codes saturate
        self.kr, self.static = kr, static
        self.dims = kvq.dims(nb, Hk, self.Hq, D, nb)

    def cache(self):
        c = kvq.LayerCache.allocate(self.fmt, self.dims, **{s: SC.bf16(y).cuda() for s, y in self.static.items()})
        c.k.fill_(3)
        c.v.fill_(5)
        return c

    def write(self, cache, q=True, stream=None, q_out=None):
        return cache.append_rope(self.q if q else None, self.k, self.v, SC.i32(self.pos), torch.from_numpy(self.table).cuda(),
                                 torch.from_numpy(self.slots).cuda(), q_out=q_out, interleaved=self.interleaved, stream=stream)

    def expect(self, keep=None):
        """The cache that kvq_append leaves, and the oracle's pool, for the rotated keys."""
        keep = np.ones(self.T, bool) if keep is None else keep
        slots = np.where(keep, self.slots, -1)
        c = self.cache()
        c.append(SC.bf16(self.kr).cuda(), self.v.contiguous(), torch.from_numpy(slots).cuda())
        pool = OP.LogicalPool(self.fmt, self.nb, self.Hk, 16, self.D, **self.static)
        ok = slots < self.nb * 16
        pool.append(self.kr[ok], self.x[ok, self.Hq + self.Hk:], slots[ok])
        return c, pool, slots[ok & (slots >= 0)]

    def check(self, cache, keep=None):
        c, pool, slots = self.expect(keep)
        for a, b in ((cache.k, c.k), (cache.v, c.v), (cache.k_scale, c.k_scale), (cache.v_scale, c.v_scale)):
            same = a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            assert same
        blk, off = slots // 16, slots % 16
        for got, ref in ((cache.k_logical(), pool.k), (cache.v_logical(), pool.v)):
            got = got.float().cpu().numpy() if self.fmt == "bf16" else got.cpu().numpy().view(pool.k.dtype)
            assert np.array_equal(got[blk, :, off], ref[blk, :, off])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("fmt", SC.ALL)
def test_formats(fmt, D, rotary, interleaved):
    c = Case(fmt, 37, D=D, rotary=rotary, interleaved=interleaved)
    cache = c.cache()
    q = c.write(cache)
    assert kvq.device_error() == 0
    c.check(cache)
    assert np.array_equal(q.float().cpu().numpy(), c.q_ref)
    # and the rotation itself: half a BF16 step of the value, three FP32 roundings of the pair's size
    exact = OR.rotate(c.x[:, :c.Hq], c.pos, c.table, interleaved, np.float64)
    assert np.all(np.abs(q.double().cpu().numpy() - exact) <= np.abs(exact) * 2.0 ** -8 + 3 * np.abs(c.x).max() * 2.0 ** -23)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 100, 384])
def test_counts(T):
    c = Case("fp8", T, D=128, G=4)
    cache = c.cache()
    assert np.array_equal(c.write(cache).float().cpu().numpy(), c.q_ref)
    c.check(cache)


@pytest.mark.parametrize("Hk,G", [(1, 1), (1, 8), (3, 4), (5, 8), (8, 8)])
def test_heads(Hk, G):
    """Query heads that fill no, one or several groups of 16."""
    for D in (64, 128):
        c = Case("int8", 21, Hk=Hk, G=G, D=D, rotary=32, fused=G != 4)
        cache = c.cache()
        assert np.array_equal(c.write(cache).float().cpu().numpy(), c.q_ref)
        c.check(cache)


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16", "int8c"])
def test_slots_that_skip_continue_and_scatter(fmt):
    """Runs that begin and end inside pages, single scattered slots, padding (slot < 0):
    skipped tokens' queries are rotated all the same."""
    rng = np.random.default_rng(3)
    slots = np.concatenate([np.arange(5, 40), [-1, -1], np.arange(64, 80), rng.permutation(np.arange(100, 140))[:20], [-7, 383]])
    c = Case(fmt, len(slots), slots=slots)
    cache = c.cache()
    assert np.array_equal(c.write(cache).float().cpu().numpy(), c.q_ref)
    assert kvq.device_error() == 0
    c.check(cache)


def test_without_a_query_and_into_a_given_one():
    c = Case("e5m2", 20)
    cache = c.cache()
    assert c.write(cache, q=False) is None
    c.check(cache)
    out = torch.empty(20, c.Hq, c.D, dtype=torch.bfloat16, device="cuda")
    assert c.write(cache, q_out=out) is out and np.array_equal(out.float().cpu().numpy(), c.q_ref)


def test_positions_and_slots_outside():
    """A position outside the table skips its token (the query's row too) and sets the error
    bit, unless the slot skips it already; a slot behind the pool sets its own."""
    c = Case("fp8", 40)
    keep = np.ones(40, bool)
    for t, p in ((3, -1), (17, 600), (18, 2 ** 31 - 1), (35, -2 ** 31)):
        c.pos[t] = p
        keep[t] = False
    cache, out = c.cache(), torch.full((40, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    c.write(cache, q_out=out)
    assert kvq.device_error() == kvq.DEVERR_POSITION
    c.check(cache, keep)
    got = out.float().cpu().numpy()
    assert np.array_equal(got[keep], c.q_ref[keep]) and (got[~keep] == 7).all()
    c.slots[~keep] = -1                              # padding with whatever position
    cache = c.cache()
    c.write(cache, q_out=out)
    assert kvq.device_error() == 0
    c.check(cache, keep)
    c = Case("fp8", 20)
    c.slots[4], c.slots[9] = c.nb * 16, 2 ** 62
    cache = c.cache()
    c.write(cache)
    assert kvq.device_error() == kvq.DEVERR_SLOT
    c.check(cache, ~np.isin(np.arange(20), [4, 9]))


def test_far_positions():
    c = Case("bf16", 12, max_pos=131072, rotary=64)
    c.pos[:3] = [131071, 131070, 65536]
    c.q_ref = OR.rotate(c.x[:, :c.Hq], c.pos, c.table)
    c.kr = OR.rotate(c.x[:, c.Hq:c.Hq + c.Hk], c.pos, c.table)
    cache = c.cache()
    assert np.array_equal(c.write(cache).float().cpu().numpy(), c.q_ref)
    c.check(cache)


def test_captured_and_on_another_stream():
    c = Case("int8", 33, D=128)
    cache, out = c.cache(), torch.empty(33, c.Hq, c.D, dtype=torch.bfloat16, device="cuda")
    pos, table, slots = SC.i32(c.pos), torch.from_numpy(c.table).cuda(), torch.from_numpy(c.slots).cuda()
    call = lambda: cache.append_rope(c.q, c.k, c.v, pos, table, slots, q_out=out)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    cache.k.fill_(3)
    cache.v.fill_(5)
    out.zero_()
    g.replay()
    assert np.array_equal(out.float().cpu().numpy(), c.q_ref)
    c.check(cache)
    s = torch.cuda.Stream()
    cache2 = c.cache()
    torch.cuda.synchronize()
    c.write(cache2, stream=s)
    s.synchronize()
    c.check(cache2)


def test_binding_refuses():
    c = Case("fp8", 6)
    cache = c.cache()
    ok = dict(q=c.q, k=c.k, v=c.v, positions=SC.i32(c.pos), cos_sin=torch.from_numpy(c.table).cuda(),
              slot_mapping=torch.from_numpy(c.slots).cuda())
    for bad in (dict(k=c.k.float()), dict(k=c.k[:, :1]), dict(v=c.v[..., :32]), dict(v=c.v[:5]), dict(q=c.q[:5]),
                dict(k=c.k.transpose(0, 1)), dict(v=c.v.cpu()), dict(positions=ok["positions"].long()),
                dict(positions=ok["positions"][:5]), dict(slot_mapping=ok["slot_mapping"].int()),
                dict(slot_mapping=ok["slot_mapping"][1:]), dict(cos_sin=ok["cos_sin"].half()), dict(cos_sin=ok["cos_sin"][0]),
                dict(cos_sin=ok["cos_sin"][:, :24].contiguous()), dict(cos_sin=ok["cos_sin"][:, :32]),
                dict(cos_sin=ok["cos_sin"][:0]), dict(q_out=c.q), dict(q=None, q_out=torch.empty(6, c.Hq, c.D, dtype=torch.bfloat16, device="cuda")),
                dict(q_out=torch.empty(6, c.Hq, c.D, device="cuda")),
                dict(k=c.k.expand(6, c.Hk, c.D)[:1].expand(6, c.Hk, c.D))):
        with pytest.raises(kvq.KvqError):
            cache.append_rope(**{**ok, **bad})
    empty = cache.append_rope(c.q[:0], c.k[:0], c.v[:0], ok["positions"][:0], ok["cos_sin"], ok["slot_mapping"][:0])
    assert empty.shape == (0, c.Hq, c.D) and kvq.device_error() == 0
    assert (cache.k == 3).all() and (cache.v == 5).all()
