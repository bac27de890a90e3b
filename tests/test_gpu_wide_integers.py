"""GPU tests of sizes that do not fit the 32 bits in which the C ABI takes them: the
binding refuses them (before any launch) instead of passing their low bits on.
"""

import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from tests import step_cases as SC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [2 ** 32, 2 ** 32 + 40, -2 ** 32, -2 ** 32 + 40, 2 ** 31, 2 ** 64 + 40])
def test_sizes_beyond_32_bits_are_refused(wide):
    f = SC.Filled("fp8", [40], D=64)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu, ctx = SC.i32([0, 3]), SC.i32([40])
    for calls in (lambda: f.cache.ragged(q, cu, f.d_tables, ctx, wide),
                  lambda: f.cache.ragged_workspace(wide),
                  lambda: f.cache.read(f.d_tables, SC.i32([0]), SC.i32([0, 3]), wide)):
        with pytest.raises(kvq.KvqError):
            calls()
    if wide < 0:                                     # a window wider than any context hides nothing
        with pytest.raises(kvq.KvqError):
            f.cache.ragged(q, cu, f.d_tables, ctx, 40, window=wide)
    else:
        assert torch.equal(f.cache.ragged(q, cu, f.d_tables, ctx, 40, window=wide), f.cache.ragged(q, cu, f.d_tables, ctx, 40))
    assert kvq.device_error() == 0
