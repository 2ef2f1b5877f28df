"""The gradient GEMM's bounded waits in calls that take longer than the limit.

MOE_OPT_WAIT_LIMIT_US bounds one hand-over between the kernel's roles (a stage,
an accumulator: microseconds), not a call, however long it runs: a healthy call
raises nothing and stores everything.
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


@pytest.fixture
def limit(moe):
    old = moe.moe_get_option(moe.MOE_OPT_WAIT_LIMIT_US)
    yield lambda us: moe.moe_set_option(moe.MOE_OPT_WAIT_LIMIT_US, us)
    moe.moe_set_option(moe.MOE_OPT_WAIT_LIMIT_US, old)


def signs(shape, g):
    """-1 and 1 as E4M3 codes, all scales 1."""
    c = torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8).mul_(0x80).add_(0x38)
    return c, torch.full((shape[0], shape[1] // 128), 127, dtype=torch.uint8, device="cuda")


def test_call_longer_than_the_limit(moe, limit):
    """2.1e14 operations: 0.13 s at the highest rate measured, and waits for what
    is in flight last 0.1 s at the least.  Sums of at most 2^18 ones: exact."""
    R, N, K = 1 << 18, 16384, 24576
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    codes, scales = signs((R, K), g)
    dy = torch.randint(-1, 2, (R, N), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    ws = torch.empty(moe.moe_ckpt_wgrad_workspace_bytes(R, N, K), dtype=torch.uint8, device="cuda")
    dw = torch.full((N, K), float("nan"), device="cuda")
    limit(50000)
    moe.moe_ckpt_wgrad(dy, codes, scales, dw=dw, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0
    rows = torch.arange(5, N, 64, device="cuda")          # of every half tile
    want = torch.zeros((len(rows), K), device="cuda")
    for i in range(0, R, 8192):
        want += dy[i:i + 8192][:, rows].float().t() @ (1.0 - 2.0 * (codes[i:i + 8192] >> 7).float())
    assert torch.equal(dw[rows], want)


def test_stage_with_a_tail_far_behind_the_first(moe, limit):
    """A first group of whole stages, 0.15 ms of work, in front of a group that ends
    inside a stage with rows behind it: the warps that clear those rows wait for
    longer than the limit, for a stage that is on its way."""
    R, N, K, cut = 16384, 4096, 4096, 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    codes, scales = signs((R, K), g)
    dy = torch.randint(-1, 2, (R, N), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    last = R - 77
    dy[last:] = float("nan")
    off = torch.tensor([0, cut, last], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ckpt_wgrad_workspace_bytes(R, N, K, 2), dtype=torch.uint8, device="cuda")
    x = 1.0 - 2.0 * (codes >> 7).float()
    want = torch.stack([dy[a:b].float().t() @ x[a:b] for a, b in ((0, cut), (cut, last))])
    limit(100)
    dw = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0
    assert torch.equal(dw, want)


@pytest.mark.parametrize("groups", [None, [0, 10, 10, 33]])
def test_error_word_is_cleared_in_front_of_the_product(moe, limit, groups):
    """Few rows, where the product reads the codes itself: the word is cleared by a
    launch in front (a clear by one block of the product's own grid may come after
    another block's flag and take it away), and a flag raised at once stays."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    codes, scales = signs((40, 256), g)
    dy = torch.randn(40, 512, generator=g, device="cuda").bfloat16()
    off = None if groups is None else torch.tensor(groups, dtype=torch.int32, device="cuda")
    G = 1 if groups is None else len(groups) - 1
    ws = torch.full((moe.moe_ckpt_wgrad_workspace_bytes(40, 512, 256, G),), 0xA5, dtype=torch.uint8, device="cuda")
    before = moe.moe_launch_count()
    want = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws)
    assert moe.moe_launch_count() - before == 2
    assert moe.moe_check_device_flag(ws) == 0
    limit(1)
    moe.moe_set_option(moe.MOE_OPT_TEST_GRAD_TIMEOUT, 1)
    try:
        moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws)
        assert moe.moe_check_device_flag(ws) == moe.FLAG_TIMEOUT
    finally:
        moe.moe_set_option(moe.MOE_OPT_TEST_GRAD_TIMEOUT, 0)
    limit(1000000)
    assert torch.equal(moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws), want)
    assert moe.moe_check_device_flag(ws) == 0
