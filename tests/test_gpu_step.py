"""GPU test of a server's steps as they run together: prompts in chunks beside
sequences that decode (kvq_append_rope, kvq_ragged_attn), on blocks that the
library's pool gives out; then a prefix read back (kvq_read) and written into
another cache. Compared with 64-bit attention over the oracle's pool, which the
oracle's rotation and quantization fill; and the whole step in one CUDA graph.
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

HK, G, D, B, NB, W = 2, 4, 128, 4, 64, 32
PLAN = [[40, 1, 0, 7], [60, 1, 100, 1], [1, 1, 33, 1], [1, 0, 1, 1]]     # new tokens of each step


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16"])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_server(fmt, graph):
    rng = np.random.default_rng(11)
    d = kvq.dims(NB, HK, HK * G, D, W)
    cache, pool = kvq.LayerCache.allocate(fmt, d), OP.LogicalPool(fmt, NB, HK, 16, D)
    blocks = kvq.Pool(d, fmt)
    rows = [[-1] * W for _ in range(B)]
    table = OR.table(512, D)
    T = 176                                          # every step padded to this many rows
    fused = torch.zeros(T, HK * G + 2 * HK, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = fused[:, :HK * G], fused[:, HK * G:HK * (G + 1)], fused[:, HK * (G + 1):]
    pos, slots = SC.i32(np.zeros(T)), torch.full((T,), -1, dtype=torch.int64, device="cuda")
    cu, ctx, tables = SC.i32(np.zeros(B + 1)), SC.i32(np.zeros(B)), SC.i32(np.full((B, W), -1))
    cs, ws = torch.from_numpy(table).cuda(), cache.ragged_workspace(T)
    q_rot, out = torch.empty(T, HK * G, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, HK * G, D, device="cuda")

    def step():
        cache.append_rope(q, k, v, pos, cs, slots, q_out=q_rot)
        cache.ragged(q_rot, cu, tables, ctx, 16 * W, out=out, workspace=ws)

    step()                                           # nothing but padding
    assert kvq.device_error() == 0
    g = None
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    length = np.zeros(B, int)
    for new in PLAN:
        n = sum(new)
        x = OF.bf16_round(rng.standard_normal((T, HK * G + 2 * HK, D)).astype(np.float32))
        p, s = np.zeros(T, np.int64), np.full(T, -1, np.int64)
        c0 = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            if new[b]:
                s[c0[b]:c0[b + 1]] = blocks.extend_seq(rows[b], int(length[b]), new[b])
            p[c0[b]:c0[b + 1]] = length[b] + np.arange(new[b])
            length[b] += new[b]
        fused.copy_(SC.bf16(x))
        pos.copy_(SC.i32(p))
        slots.copy_(torch.from_numpy(s))
        cu.copy_(SC.i32(c0))
        ctx.copy_(SC.i32(length))
        tables.copy_(SC.i32(rows))
        out.fill_(7.0)
        g.replay() if g else step()
        assert kvq.device_error() == 0
        qr = OR.rotate(x[:, :HK * G], p, table)
        kr = OR.rotate(x[:, HK * G:HK * (G + 1)], p, table)
        pool.append(kr, x[:, HK * (G + 1):], s)
        assert np.array_equal(q_rot.float().cpu().numpy(), qr)
        kv = [pool.gather(rows[b], length[b]) for b in range(B)]
        ref, bound = SC.attention_and_bound(qr[:n], c0, kv, D ** -0.5, HK, 0, fmt, True)
        SC.assert_within(out[:n], ref, bound)
        assert (out[n:] == 7).all()
    # sequence 2's prefix out of the cache and into one of another format
    n = int(length[2])
    kk, vv = cache.read(SC.i32([rows[2]]), SC.i32([0]), SC.i32([0, n]), n)
    K, V = pool.gather(rows[2], n)
    assert np.array_equal(kk.float().cpu().numpy(), OF.bf16_round(K.astype(np.float32)))
    other = kvq.LayerCache.allocate("e5m2", d)
    other.append(kk, vv, torch.arange(n, device="cuda"))
    opool = OP.LogicalPool("e5m2", NB, HK, 16, D)
    opool.append(OF.bf16_round(K.astype(np.float32)), OF.bf16_round(V.astype(np.float32)), np.arange(n))
    row = SC.i32([list(range(W))])
    k2, _ = other.read(row, SC.i32([0]), SC.i32([0, n]), n, out_dtype=torch.float32)
    assert np.array_equal(k2.double().cpu().numpy(), opool.gather(list(range(W)), n)[0])
    assert kvq.device_error() == 0
