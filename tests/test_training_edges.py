"""The training operators at the edges of their documentation."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp4_routed_mixture_b200 as m
    return m


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def routed(moe, T, E, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn(T, E, generator=g, device="cuda")
    return z, *moe.moe_route(z, k)


@pytest.mark.parametrize("E", [8, 7, 256, 300])
@pytest.mark.parametrize("coef,dloss", [(1.0, 1.0), (0.0, 1.0), (1.0, 0.0)])
def test_route_backward_keeps_nan_at_weight_zero(moe, E, coef, dloss):
    """The balance term is weight * p * (f - p f): NaN in a row whose softmax is,
    whatever the weight; 0 in the others at weight 0; masked rows are out of it."""
    z, idx, _ = routed(moe, 9, E, 2, E)
    z[2, 3] = float("nan")
    z[4, 1] = float("inf")
    z[6, 0] = float("nan")
    mask = torch.ones(9, dtype=torch.bool, device="cuda")
    mask[6] = False
    _, counts, _, tokens = moe.moe_balance_loss(z, idx, 1.0, seq_offsets=i32(0, 4, 8), token_mask=mask)
    d = moe.moe_route_backward(z, idx, dloss=torch.full((1,), dloss, device="cuda"), coef=coef, counts=counts,
                               tokens=tokens, seq_offsets=i32(0, 4, 8), token_mask=mask)
    nan = torch.isnan(d)
    assert nan.all(1).tolist() == nan.any(1).tolist() == [t in (2, 4) for t in range(9)]
    rest = [0, 1, 3, 5, 7]
    assert bool((d[rest] != 0).any(1).all()) == (coef * dloss != 0)
    assert not d[[6, 8]].any()                  # masked; behind the last sequence


@pytest.mark.parametrize("seq,bad", [((0, 0, 0), 0), ((0, 5, 0), 1), ((0, 0, 3), 1), ((-1, 0, 0), 1),
                                     ((0,) * 700 + (2,), 1), ((0,) * 701, 0)])
def test_balance_of_no_tokens_checks_the_offsets(moe, seq, bad):
    S, E = len(seq) - 1, 8
    ws = torch.full((moe.moe_balance_workspace_bytes(0, E, S),), 0xA5, dtype=torch.uint8, device="cuda")
    z, idx = torch.empty((0, E), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    loss, counts, prob, tokens = moe.moe_balance_loss(z, idx, 1.0, seq_offsets=i32(*seq), ws=ws)
    assert moe.moe_check_device_flag(ws) == (moe.FLAG_BOUNDS if bad else 0)
    assert not loss.any() and not counts.any() and not prob.any() and not tokens.any()


@pytest.mark.parametrize("seq", [(0, 700, 300, 1000), (0, 900, 100, 200, 1000), (400, 0, 1000), (0, 500, 1001)])
def test_balance_bad_offsets_in_a_used_workspace(moe, seq):
    """Many rows, where offsets that do not ascend make the sum read places of the
    workspace that the call has not written: no bits but the documented ones."""
    T, E = 1000, 16
    z, idx, _ = routed(moe, T, E, 2, 3)
    n = moe.moe_balance_workspace_bytes(T, E, len(seq) - 1)
    for fill in (0xA5, 0xFF, 0):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        moe.moe_balance_loss(z, idx, 1.0, seq_offsets=i32(*seq), ws=ws)
        flag = moe.moe_check_device_flag(ws)
        assert flag & moe.FLAG_BOUNDS and not flag & ~(moe.FLAG_BOUNDS | moe.FLAG_BAD_EXPERT)
    a = moe.moe_balance_loss(z, idx, 1.0, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0
    assert all(torch.equal(u, v) for u, v in zip(a, moe.moe_balance_loss(z, idx, 1.0)))


def test_sizes_beyond_32_bits_are_refused(moe):
    """2^32 + 8 rows and k = 2^32 + 1 would arrive in C as 8 and 1."""
    T = (1 << 32) + 8
    z, idx = torch.zeros((T, 1), device="cuda"), torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_balance_workspace_bytes(8, 1, 1), dtype=torch.uint8, device="cuda")
    out = (torch.empty(1, device="cuda"), i32(0).view(1, 1), None, i32(0, 0))
    before = moe.moe_launch_count()
    with pytest.raises(moe.MoeError) as e:
        moe.moe_balance_loss(z, idx, 1.0, ws=ws, out=out)
    assert e.value.status == -2
    del z, idx
    codes, scales = moe.moe_ckpt_pack(torch.zeros((16, 128), dtype=torch.bfloat16, device="cuda"))
    dy = torch.zeros((16, 8), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_ckpt_wgrad(dy, codes, scales, perm=torch.arange(16, dtype=torch.int32, device="cuda"), k=(1 << 32) + 1)
    assert e.value.status == -2
    assert moe.moe_launch_count() == before + 1          # the pack alone
