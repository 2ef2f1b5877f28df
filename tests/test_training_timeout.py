"""The gradient GEMM's bounded waits, made to run out on purpose.

MOE_OPT_TEST_GRAD_TIMEOUT makes the next weight gradient withhold each SM pair's
first stage (no copy and no arrival: a barrier that nothing completes);
with a short limit the wait ends in milliseconds.  The call must raise
MOE_FLAG_TIMEOUT and return, and the next call in the same process be exact.
Nothing faults, traps or hangs.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp4_routed_mixture_b200 as m
    return m


@pytest.mark.parametrize("R,groups", [(40, None), (1000, None), (1000, [0, 333, 333, 1000]), (90, [0, 10, 10, 85]),
                                      (600, None)])
def test_withheld_stage_times_out_then_next_call_is_exact(moe, R, groups):
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    codes, scales = moe.moe_ckpt_pack(torch.randn(R, 256, generator=g, device="cuda").bfloat16())
    dy = torch.randn(R, 512, generator=g, device="cuda").bfloat16()
    off = None if groups is None else torch.tensor(groups, dtype=torch.int32, device="cuda")
    G = 1 if groups is None else len(groups) - 1
    ws = torch.empty(moe.moe_ckpt_wgrad_workspace_bytes(R, 512, 256, G), dtype=torch.uint8, device="cuda")
    want = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0
    old = moe.moe_get_option(moe.MOE_OPT_WAIT_LIMIT_US)
    try:
        moe.moe_set_option(moe.MOE_OPT_WAIT_LIMIT_US, 20000)
        moe.moe_set_option(moe.MOE_OPT_TEST_GRAD_TIMEOUT, 1)
        moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws)
        assert moe.moe_check_device_flag(ws) & moe.FLAG_TIMEOUT
        assert moe.moe_get_option(moe.MOE_OPT_TEST_GRAD_TIMEOUT) == 0
    finally:
        moe.moe_set_option(moe.MOE_OPT_WAIT_LIMIT_US, old)
        moe.moe_set_option(moe.MOE_OPT_TEST_GRAD_TIMEOUT, 0)
    assert torch.equal(moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws), want)
    assert moe.moe_check_device_flag(ws) == 0


def test_option_validation(moe):
    for bad in (-1, 2):
        with pytest.raises(moe.MoeError):
            moe.moe_set_option(moe.MOE_OPT_TEST_GRAD_TIMEOUT, bad)
