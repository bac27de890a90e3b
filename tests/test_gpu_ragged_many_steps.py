"""GPU tests of steps of hundreds of sequences with one new token each, and a few with more
or none: up to 1,024 sequences share the decode kernels' workspace, more go through the
ragged kernel alone.
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from tests import step_cases as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16"])
@pytest.mark.parametrize("B", [256, 257, 683, 1024, 1025])
def test_steps_of_many_sequences(fmt, B):
    rng = np.random.default_rng(B)
    ctx = [int(x) for x in rng.choice([0, 1, 16, 17, 40, 129], B)]
    ctx[3], ctx[B - 1] = 900, 131
    f = SC.Filled(fmt, ctx, Hk=2, G=2, D=64, width=64)
    some = [1] * B                                   # the same shape of call with other make-ups
    some[0], some[1], some[3], some[7] = 0, 2, 0, 2
    for n in ([1] * B, some):
        cu = np.concatenate([[0], np.cumsum(n)])
        q = torch.randn(B, 4, 64, generator=torch.Generator().manual_seed(B)).bfloat16().cuda()
        out = f.cache.ragged(q, SC.i32(cu), f.d_tables, SC.i32(f.ctx), 1024)
        assert kvq.device_error() == 0
        m = int(cu[-1])
        ref, bound = SC.attention_and_bound(q[:m].float().cpu().numpy(), cu, f.kv(), 0.125, 2, 0, fmt, False, step=True)
        SC.assert_within(out[:m], ref, bound)
