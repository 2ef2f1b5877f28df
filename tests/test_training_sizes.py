"""Sizes beyond 32 bits in the training calls' size queries (no GPU)."""
import pytest

import fp4_routed_mixture_b200 as moe

W = 1 << 32


@pytest.mark.parametrize("query,args", [
    (moe.moe_balance_workspace_bytes, (8, 256, 1)), (moe.moe_router_backward_workspace_bytes, (8, 128, 16)),
    (moe.moe_ckpt_wgrad_workspace_bytes, (8, 64, 128, 2)),
])
def test_size_beyond_32_bits_is_refused(query, args):
    assert query(*args) > 0
    for i, v in enumerate(args):
        for big in (v + W, v - W, 1 << 70):
            with pytest.raises(moe.MoeError) as e:
                query(*args[:i], big, *args[i + 1:])
            assert e.value.status == -2
