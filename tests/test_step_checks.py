"""CPU tests of the calls of a serving step (kvq_append_rope, kvq_read,
kvq_ragged_attn): what they refuse, checked before any launch (aligned fake
pointers never reach a kernel), workspace sizes, the binding's own checks, and
the oracle's rotary embedding and ragged attention against independent forms.
"""

import ctypes as C
import math

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from oracle import attention as OA
from oracle import rope as OR

OK, ARG, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
NULL, ODD = 0, (1 << 20) + 8
# distinct fake device addresses, far apart
Q, K, V, OUT, KC, VC, KS, VS, TAB, CTX, CU, CS, POS, SLOT, WS = [(i + 1) << 32 for i in range(15)]
DIMS = kvq.dims(64, 2, 8, 128, 8)          # G = 4


def _scales(a=KS, b=VS):
    return (C.c_void_p * 2)(a, b)


def rope(**kw):
    a = dict(q=Q, qs=1024, k=K, ks=256, v=V, vs=256, pos=POS, cs=CS, mp=4096, rd=128, pairs=0, slots=SLOT, n=5, qo=OUT,
             kc=KC, vc=VC, ksc=KS, vsc=VS, fmt=1, d=DIMS)
    a.update(kw)
    return kvq.lib().kvq_append_rope(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["cs"], a["mp"], a["rd"],
                                     a["pairs"], a["slots"], a["n"], a["qo"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["fmt"],
                                     C.byref(a["d"]), None)


@pytest.mark.parametrize("bad,rc", [
    (dict(k=NULL), ARG), (dict(k=ODD), ARG), (dict(v=NULL), ARG), (dict(pos=NULL), ARG), (dict(cs=NULL), ARG),
    (dict(cs=ODD), ARG), (dict(slots=NULL), ARG), (dict(kc=NULL), ARG), (dict(vc=ODD), ARG),
    (dict(ksc=NULL), ARG), (dict(vsc=NULL), ARG),
    (dict(q=NULL), ARG), (dict(qo=NULL), ARG), (dict(q=ODD), ARG), (dict(qo=ODD), ARG),
    (dict(ks=248), ARG), (dict(ks=260), ARG), (dict(vs=128), ARG), (dict(qs=1016), ARG), (dict(qs=1028), ARG),
    (dict(ks=0), ARG), (dict(ks=-256), ARG),
    (dict(rd=0), ARG), (dict(rd=24), ARG), (dict(rd=144), ARG), (dict(rd=-16), ARG), (dict(mp=0), ARG),
    (dict(pairs=2), ARG), (dict(n=-1), ARG), (dict(fmt=6), ARG), (dict(fmt=8), ARG), (dict(fmt=-1), ARG),
    (dict(qo=Q), ARG), (dict(qo=K + 16), ARG), (dict(qo=V - 16), ARG),      # the output over an input
    (dict(d=kvq.dims(64, 2, 6, 128, 8)), UNSUPPORTED), (dict(d=kvq.dims(64, 2, 8, 96, 8)), UNSUPPORTED),
])
def test_append_rope_refuses(bad, rc):
    assert rope(**bad) == rc


def test_append_rope_of_no_tokens():
    none = dict(n=0, q=NULL, k=NULL, v=NULL, pos=NULL, cs=NULL, slots=NULL, qo=NULL, kc=NULL, vc=NULL)
    assert rope(**none) == OK
    assert rope(**none, rd=24) == ARG                    # sizes are checked all the same


def read(**kw):
    a = dict(kc=KC, vc=VC, sc=_scales(), tab=TAB, st=CTX, cu=CU, b=3, n=50, ko=OUT, vo=Q, dt=0, fmt=1, d=DIMS)
    a.update(kw)
    return kvq.lib().kvq_read(a["kc"], a["vc"], a["sc"], a["tab"], a["st"], a["cu"], a["b"], a["n"], a["ko"], a["vo"], a["dt"],
                              a["fmt"], C.byref(a["d"]), None)


@pytest.mark.parametrize("bad,rc", [
    (dict(kc=NULL), ARG), (dict(vc=NULL), ARG), (dict(sc=None), ARG), (dict(sc=_scales(0, VS)), ARG),
    (dict(sc=_scales(KS, 0)), ARG), (dict(sc=_scales(KS, 0), fmt=6), ARG), (dict(tab=NULL), ARG), (dict(tab=ODD), ARG),
    (dict(st=NULL), ARG), (dict(cu=NULL), ARG), (dict(cu=ODD), ARG), (dict(b=-1), ARG), (dict(n=-1), ARG),
    (dict(ko=NULL, vo=NULL), ARG), (dict(ko=ODD), ARG), (dict(vo=ODD), ARG), (dict(dt=2), ARG), (dict(fmt=8), ARG),
    (dict(vo=OUT), ARG), (dict(vo=OUT + 1024), ARG),     # both outputs in one place
    (dict(d=kvq.dims(64, 2, 8, 128, 0)), ARG), (dict(d=kvq.dims(64, 2, 32, 128, 8)), UNSUPPORTED),
])
def test_read_refuses(bad, rc):
    assert read(**bad) == rc


def test_read_of_nothing():
    for none in (dict(b=0), dict(n=0)):
        assert read(kc=NULL, vc=NULL, sc=None, tab=NULL, st=NULL, cu=NULL, ko=NULL, vo=NULL, **none) == OK
        assert read(dt=5, **none) == ARG


def ragged(**kw):
    a = dict(q=Q, qs=1024, cu=CU, b=3, n=50, kc=KC, vc=VC, sc=_scales(), tab=TAB, ctx=CTX, mc=100, win=0, sm=0.1, out=OUT, dt=0,
             ws=WS, wsn=1 << 40, fmt=1, d=DIMS)
    a.update(kw)
    return kvq.lib().kvq_ragged_attn(a["q"], a["qs"], a["cu"], a["b"], a["n"], a["kc"], a["vc"], a["sc"], a["tab"], a["ctx"], a["mc"],
                                     a["win"], a["sm"], a["out"], a["dt"], a["ws"], a["wsn"], a["fmt"], C.byref(a["d"]), None)


@pytest.mark.parametrize("bad,rc", [
    (dict(q=NULL), ARG), (dict(q=ODD), ARG), (dict(qs=1016), ARG), (dict(qs=1026), ARG), (dict(qs=-1024), ARG), (dict(cu=NULL), ARG),
    (dict(cu=ODD), ARG), (dict(kc=NULL), ARG), (dict(vc=NULL), ARG), (dict(sc=None), ARG), (dict(sc=_scales(0, VS)), ARG),
    (dict(tab=NULL), ARG), (dict(ctx=NULL), ARG), (dict(out=NULL), ARG), (dict(out=ODD), ARG), (dict(ws=NULL), ARG),
    (dict(ws=ODD), ARG), (dict(wsn=1024), WORKSPACE), (dict(wsn=0), WORKSPACE), (dict(b=-1), ARG), (dict(n=-1), ARG),
    (dict(mc=-1), ARG), (dict(mc=129), ARG), (dict(win=-1), ARG), (dict(dt=2), ARG), (dict(sm=math.nan), ARG),
    (dict(sm=math.inf), ARG), (dict(fmt=6), ARG), (dict(fmt=99), ARG), (dict(out=Q), ARG), (dict(out=Q + 2048), ARG),
    (dict(d=kvq.dims(64, 2, 6, 128, 8)), UNSUPPORTED), (dict(n=1 << 30), UNSUPPORTED),
])
def test_ragged_refuses(bad, rc):
    assert ragged(**bad) == rc


def test_ragged_of_nothing_and_its_workspace():
    for none in (dict(b=0), dict(n=0)):
        assert ragged(q=NULL, cu=NULL, kc=NULL, vc=NULL, sc=None, tab=NULL, ctx=NULL, out=NULL, ws=NULL, wsn=0, **none) == OK
        assert ragged(win=-1, **none) == ARG
    size = lambda n, fmt=1, d=DIMS: kvq.lib().kvq_ragged_attn_workspace_bytes(n, fmt, C.byref(d))  # noqa: E731
    assert size(0) == size(-1) == size(4, 6) == size(4, 99) == size(4, 1, kvq.dims(64, 2, 6, 128, 8)) == 0
    sizes = [size(n) for n in (1, 2, 16, 64, 65, 256, 257, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] == sizes[-3]   # grows up to 256 tokens


# ------------------------------------------------------------------ the binding
def test_binding_takes_device_tensors_only():
    d = kvq.dims(4, 2, 4, 64, 2)
    c = kvq.LayerCache.allocate("fp8", d, device="cpu")
    q, kv = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(kvq.KvqError, match="CUDA device"):
        c.append_rope(q, kv, kv, i32, torch.zeros(8, 64), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(kvq.KvqError, match="CUDA device"):
        c.read(torch.zeros(1, 2, dtype=torch.int32), i32[:1], i32[:2], 3)
    with pytest.raises(kvq.KvqError, match="CUDA device"):
        c.ragged(q, i32[:2], torch.zeros(1, 2, dtype=torch.int32), i32[:1], 32)


def test_binding_row_layouts():
    """Views of a fused projection pass, with the stride between their tokens;
    other types, shapes and orders do not. (The helper's device index of a CPU
    tensor is -1.)"""
    x = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    assert kvq._rows_at(-1, x[:, 2:6], "q", 5, 4, 64) == (x.data_ptr() + 2 * 64 * 2, 512)
    assert kvq._rows_at(-1, x[::2, 2:6], "q", 3, 4, 64)[1] == 1024
    assert kvq._rows_at(-1, x[:1, 2:3].expand(1, 1, 64), "q", 1, 1, 64)[1] == 64
    for bad in (x[:, ::2], x[..., :32], x.float(), x[:, :3], x.transpose(0, 1), x[..., ::2]):
        with pytest.raises(kvq.KvqError):
            kvq._rows_at(-1, bad, "q", 5, 4, 64)


# ------------------------------------------------------------------ the oracle's pins
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [16, 48, 64])
def test_oracle_rotation(interleaved, rotary):
    rng = np.random.default_rng(rotary)
    x = OR.bf16_round(rng.standard_normal((6, 3, 64)).astype(np.float32))
    cs = OR.table(500, rotary)
    pos = np.array([0, 1, 7, 7, 123, 499])
    y = OR.rotate(x, pos, cs, interleaved, np.float64)
    # as a complex product, pair by pair, with angles of its own
    half = rotary // 2
    for t in range(6):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            z = (x[t, :, a] + 1j * x[t, :, b].astype(np.float64)) * np.exp(1j * pos[t] * 10000.0 ** (-i / half))
            assert np.allclose(z, y[t, :, a] + 1j * y[t, :, b], atol=1e-6)      # the table holds 24 bits
    assert np.array_equal(y[..., rotary:], x[..., rotary:]) and np.array_equal(y[0], x[0])
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)
    # rounded: at most half a BF16 step, and three float32 roundings of the pair's size
    r = OR.rotate(x, pos, cs, interleaved)
    pair = np.abs(x).max()
    assert np.all(np.abs(r - y) <= np.abs(y) * 2.0 ** -8 + 3 * pair * 2.0 ** -23)
    # scores depend on the distance of the positions alone
    a, b = x[:1], x[1:2]
    dot = lambda p, q: (OR.rotate(a, [p], cs, interleaved, np.float64) * OR.rotate(b, [q], cs, interleaved, np.float64)).sum()  # noqa: E731
    assert abs(dot(5, 3) - dot(205, 203)) < 1e-4


@pytest.mark.parametrize("window", [0, 1, 5, 64])
def test_oracle_ragged_attention(window):
    rng = np.random.default_rng(window)
    n, ctx, Hk, G, D = [3, 0, 12, 1, 4], [40, 9, 12, 33, 2], 2, 2, 16
    cu = np.concatenate([[0], np.cumsum(n)])
    q = rng.standard_normal((cu[-1] + 2, Hk * G, D))
    kv = [(rng.standard_normal((c, Hk, D)), rng.standard_normal((c, Hk, D))) for c in ctx]
    out = OA.ragged_attention(q, cu, kv, 0.25, Hk, window)
    assert np.isnan(out[cu[-1]:]).all()
    for b in range(5):
        if n[b] == 0:
            continue
        rows = torch.from_numpy(q[cu[b]:cu[b + 1]]).transpose(0, 1)
        k, v = (torch.from_numpy(x).repeat_interleave(G, 1).transpose(0, 1) for x in kv[b])
        p, t = torch.arange(n[b])[:, None] + ctx[b] - n[b], torch.arange(ctx[b])[None]
        mask = (t <= p) & ((t > p - window) | (window == 0))
        ref = torch.nn.functional.scaled_dot_product_attention(rows, k, v, attn_mask=mask, scale=0.25)
        ref = torch.where(mask.any(1)[None, :, None], ref, torch.zeros_like(ref)).transpose(0, 1).numpy()
        assert np.allclose(out[cu[b]:cu[b + 1]], ref, atol=1e-12)
    # without a window and with equal counts it is the multi-query decode
    same = OA.ragged_attention(q[:12], [0, 4, 8, 12], [kv[0], kv[2], kv[3]], 0.25, Hk)
    ver = OA.verify_attention(q[:12].reshape(3, 4, Hk * G, D).transpose(0, 2, 1, 3), [kv[0], kv[2], kv[3]], 0.25, Hk)
    assert np.allclose(same, ver.transpose(0, 2, 1, 3).reshape(12, Hk * G, D), atol=1e-12)
