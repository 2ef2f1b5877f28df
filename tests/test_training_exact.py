"""The gradient GEMM on sums that are exact in fp32, where a row lost, counted
twice or taken from a wrong place shows in every bit, and its error in the norm
on random ones.

Exact: the factors are integers other than 0, of magnitude 3 and 4 at most, all
partial sums integers below 2^24; or one term a sum.  Norm: an accumulator takes
n MMAs (64 of the weight gradient, 48 of the router's) before it is drained, each
truncating by at most a step 2 u (half of it on average) of a running value that
grows as sqrt(j / n): 2 n / 3 of them u; then T / 1024 (T / 256) additions that
round to nearest.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp4_routed_mixture_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(g, m, *shape):
    """Integers from -m to m without 0."""
    v = torch.randint(1, m + 1, shape, generator=g, device="cuda").float()
    return v * (1 - 2 * torch.randint(0, 2, shape, generator=g, device="cuda").float())


def stored(moe, x):
    """A checkpoint of integers that hold in 4 bits: exact."""
    codes, scales = moe.moe_ckpt_pack(x.bfloat16())
    assert torch.equal(moe.moe_ckpt_unpack(codes, scales).float(), x)
    return codes, scales


def norm_error(got, want):
    return float((got.double() - want).norm() / want.norm())


ROWS = [1, 15, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 1023, 1024, 1025, 1151, 1152, 1153, 1216, 1217, 1281,
        2047, 2048, 2049, 4095, 4604, 8191]


@pytest.mark.parametrize("R,N,K", [(R, 264, 384) for R in ROWS] + [
    (4604, 128, 128), (5000, 512, 1024), (1300, 520, 640), (3000, 2056, 2176), (1100, 4104, 2304), (700, 2312, 2048)])
def test_wgrad_exact(moe, R, N, K):
    g = gen(R + N)
    x, dy = ints(g, 4, R, K), ints(g, 3, R, N)
    codes, scales = stored(moe, x)
    want = dy.double().t() @ x.double()
    dw = moe.moe_ckpt_wgrad(dy.bfloat16(), codes, scales)
    assert torch.equal(dw.double(), want)
    base = ints(g, 100, N, K)
    got = moe.moe_ckpt_wgrad(dy.bfloat16(), codes, scales, dw=base.clone(), accumulate=True)
    assert torch.equal(got.double(), base.double() + want)


SPLIT = [  # rows of each group, N, K: 19 stages of 64 rows or more on average, and few tiles
    ((0, 700, 1500, 6000), 264, 384), ((6001, 0, 130, 1, 4200), 264, 384), ((0, 5000, 1), 264, 384),
    ((1500, 1499, 1501), 136, 640), ((4001,), 264, 384), ((64, 7040, 128), 520, 256), ((1, 1, 9999, 0), 512, 512),
    # whole tiles in front of the split ones; pairs whose parts lie in two groups
    ((4100, 9000, 0, 3333, 3600), 1032, 1024), ((9000, 63, 9100), 776, 640),
]
WHOLE = [((2500, 63, 3700), 1288, 640)]      # 54 tiles on 74 pairs of SMs: splitting would save too little


@pytest.mark.parametrize("perm", [False, True])
@pytest.mark.parametrize("sizes,N,K", SPLIT + WHOLE)
def test_wgrad_groups_whose_tiles_are_split(moe, sizes, N, K, perm):
    """Groups of very different sizes and empty ones, rows in front of the first
    and behind the last that hold NaN and bad table entries."""
    g = gen(sum(sizes) + N)
    G, k = len(sizes), 2 if perm else 1
    front, behind = 14, 78
    off = torch.tensor([front, *sizes]).cumsum(0)
    R = int(off[-1]) + behind
    R += R % k
    X = R // k
    x, dy = ints(g, 4, X, K), ints(g, 3, R, N).bfloat16()
    dy[:front] = float("nan")
    dy[int(off[-1]):] = float("inf")
    codes, scales = stored(moe, x)
    kw, rows = {}, torch.arange(R, device="cuda")
    if perm:
        table = torch.randperm(R, generator=g, device="cuda").int()
        rows = table.long() // k
        table[:front] = -7
        table[int(off[-1]):] = 3 * R
        kw = dict(perm=table, k=k)
    else:
        codes[:front] = 0x7F
        codes[int(off[-1]):] = 0xFF
    offsets = off.int().cuda()
    ws = torch.full((moe.moe_ckpt_wgrad_workspace_bytes(R, N, K, G),), 0xFF, dtype=torch.uint8, device="cuda")
    want = torch.stack([dy[a:b].double().t() @ x[rows[a:b]].double()
                        for a, b in zip(off[:-1].tolist(), off[1:].tolist())])
    before = moe.moe_launch_count()
    dw = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=offsets, ws=ws, **kw)
    # (the third adds the parts of split tiles)
    assert moe.moe_launch_count() - before == (2 if (sizes, N, K) in WHOLE else 3)
    assert moe.moe_check_device_flag(ws) == 0
    assert torch.equal(dw.double(), want)
    base = ints(g, 100, G, N, K)
    got = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=offsets, dw=base.clone(), accumulate=True, ws=ws, **kw)
    assert torch.equal(got.double(), base.double() + want)
    assert moe.moe_check_device_flag(ws) == 0


@pytest.mark.parametrize("R,N,K", [(1000, 256, 896), (4604, 128, 128), (5000, 512, 1024), (16384, 264, 384)])
def test_wgrad_norm(moe, R, N, K):
    g = gen(R)
    codes, scales = moe.moe_ckpt_pack(torch.randn(R, K, generator=g, device="cuda").bfloat16())
    dy = torch.randn(R, N, generator=g, device="cuda").bfloat16()
    want = dy.double().t() @ moe.moe_ckpt_unpack(codes, scales).double()
    assert norm_error(moe.moe_ckpt_wgrad(dy, codes, scales), want) <= (2 * 64 / 3 + (R / 1024) ** 0.5) * U


# tokens, H, experts: one launch (the first three), and the tensor cores' form
ROUTER = [(96, 128, 32), (400, 256, 70), (512, 512, 513), (513, 256, 70), (600, 128, 257), (1300, 384, 300),
          (4604, 128, 33), (5000, 640, 1024), (300, 2048, 600)]


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("T,H,E", ROUTER)
def test_router_wgrad_keeps_every_bit_of_dlogits(moe, T, H, E, ckpt):
    """One token an expert and x = 1 (2, -0.5 in places): dw is that entry of
    dlogits, all 24 bits of it, whatever its size; without the third of its bf16
    parts the last 8 bits or so are lost."""
    g = gen(T + E)
    at = torch.randperm(max(T, E), generator=g, device="cuda")[:E] % T
    v = torch.randn(E, generator=g, device="cuda") * torch.exp2(
        torch.randint(-60, 60, (E,), generator=g, device="cuda").float())
    dl = torch.zeros((T, E), device="cuda")
    dl[at, torch.arange(E, device="cuda")] = v
    x = torch.ones((T, H), device="cuda")
    x[:, 1::7] = 2.0
    x[::3, 5::11] = -0.5
    w = torch.randn(E, H, generator=g, device="cuda")
    codes, scales = stored(moe, x)
    src = dict(codes=codes, scales=scales) if ckpt else dict(x=x.bfloat16())
    _, dw, db = moe.moe_router_logits_backward(dl, w, **src)
    assert torch.equal(dw, v.unsqueeze(1) * x[at])
    assert torch.equal(db, v)
    base = torch.zeros_like(dw)
    _, dw, _ = moe.moe_router_logits_backward(dl, w, accumulate=True, out=(None, base, None), **src)
    assert torch.equal(dw, v.unsqueeze(1) * x[at])


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("T,H,E", ROUTER)
def test_router_exact_sums(moe, T, H, E, ckpt):
    """Integers: dw and dbias exact; dx the exact sum rounded once to bf16 (its
    factors hold in one bf16 part)."""
    g = gen(T * E)
    dl, x, w = ints(g, 3, T, E), ints(g, 4, T, H), ints(g, 5, E, H)
    codes, scales = stored(moe, x)
    src = dict(codes=codes, scales=scales) if ckpt else dict(x=x.bfloat16())
    dx, dw, db = moe.moe_router_logits_backward(dl, w, **src)
    assert torch.equal(dw.double(), dl.double().t() @ x.double())
    assert torch.equal(db.double(), dl.double().sum(0))
    assert torch.equal(dx, (dl.double() @ w.double()).float().bfloat16())


@pytest.mark.parametrize("T,H,E", ROUTER)
def test_router_norm(moe, T, H, E):
    """dw as the formula above.  dx before its rounding: each operand without its third
    part, two roundings of 2^-8 or 2^-16 of a value at most, and without the product
    of the seconds, 2^-16 too; then the rounding, uniform in a step of 2^-7 of a value at
    most: 2^-7 / sqrt(12) of the norm."""
    g = gen(T + H + E)
    dl, w = torch.randn(T, E, generator=g, device="cuda"), torch.randn(E, H, generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dx, dw, db = moe.moe_router_logits_backward(dl, w, x=x)
    assert norm_error(dw, dl.double().t() @ x.double()) <= (2 * 48 / 3 + (T / 256) ** 0.5 + 1) * U
    want = dl.double() @ w.double()
    size = dl.double().abs() @ w.double().abs()
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -60))) - 7)     # of bf16
    slack = (3 * 2.0 ** -16 + (3 * E + 8) * 2 * U) * size
    assert bool(((dx.double() - want).abs() <= 0.5 * step + 2 * slack).all())
    assert norm_error(dx, want) <= 2.0 ** -7 / 12 ** 0.5 + 3 * 2.0 ** -16
    plain = want.float().bfloat16()
    off = dx != plain                     # only where the exact value lies next to the border of two steps
    border = (want - (torch.floor(want / step) + 0.5) * step).abs()
    assert bool((border[off] <= 2 * slack[off]).all())


def test_gradient_of_an_fp8_projections_input(moe):
    """dx = dy W through moe_fp8_linear on the packed transpose: blocks of 128 x 128
    stay blocks.  dy is quantised as the call quantises its input (E4M3 per row
    and 128 outputs), which the reference does too."""
    T, N, K = 70, 384, 256
    g = gen(0)
    codes = torch.randint(0, 256, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    scales = torch.randint(118, 126, (N // 128, K // 128), generator=g, device="cuda", dtype=torch.uint8)
    dy = (1e-3 * torch.randn(T, N, generator=g, device="cuda")).bfloat16()
    packed = moe.moe_fp8_pack_weights(codes.t().contiguous(), scales.t().contiguous())
    dx = moe.moe_fp8_linear(dy, packed, K).double()
    w = codes.view(torch.float8_e4m3fn).double() * torch.exp2(
        scales.double() - 127).repeat_interleave(128, 0).repeat_interleave(128, 1)
    dq, ds = moe.moe_ckpt_pack(dy)
    d = dq.view(torch.float8_e4m3fn).double() * torch.exp2(ds.double() - 127).repeat_interleave(128, 1)
    want, size = d @ w, d.abs() @ w.abs()
    # one bf16 rounding and the accumulation of N exact products (the projection's own bound)
    assert bool(((dx - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * size).all())
    # and the quantisation of dy: half a step, 2^-4 of a value, or 2^-10 of the scale below 2^-6 of it
    bound = (2.0 ** -4 * dy.double().abs() + 2.0 ** -10 * torch.exp2(ds.double() - 127).repeat_interleave(128, 1)) @ w.abs()
    assert bool(((d @ w - dy.double() @ w).abs() <= bound).all())
