"""GPU test of decode steps whose max_context_len is the model's maximum, as a captured
graph has to pass it: the same rows, bit for bit, as with the batch's own longest context,
since the shares are sized by the batch.
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from tests import step_cases as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16"])
@pytest.mark.parametrize("B", [1, 9, 64])
def test_a_loose_bound_changes_nothing(fmt, B):
    ctx = [3840 if b == B // 2 else 100 + 37 * b for b in range(B)]
    f = SC.Filled(fmt, ctx, Hk=4, G=2, D=64, width=131072 // 16)
    q = torch.randn(B, 8, 64, generator=torch.Generator().manual_seed(B)).bfloat16().cuda()
    args = (q, SC.i32(np.arange(B + 1)), f.d_tables, SC.i32(f.ctx))
    want = f.cache.ragged(*args, 3840)
    assert torch.equal(f.cache.ragged(*args, 131072), want)
    ref, bound = SC.attention_and_bound(q.float().cpu().numpy(), np.arange(B + 1), f.kv(), 0.125, 4, 0, fmt, False, step=True)
    SC.assert_within(want, ref, bound)
    assert kvq.device_error() == 0
