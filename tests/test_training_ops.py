"""The training operators against their 64-bit definitions.

Bounds (u = 2^-24, half an fp32 step; eps/2 of bf16 = 2^-8):
  softmax     p is exp(x - m) / sum: the subtraction moves the exponent by
              u |x - m|, expf is within 2 ulp (4 u), the sum of E positive
              terms and the quotient add E u / 32 + 10 u: relative.
  sums        n positive terms in any order: n u relative; with signs n u of
              the sum of magnitudes.  A tensor-core accumulation truncates, a
              whole step 2 u per addition.
  bf16        one rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from tests import training_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp4_routed_mixture_b200 as m
    return m


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    return cu(a.astype(np.float32)).to(torch.bfloat16)


def host(t):
    t = t.detach().cpu()
    return (t.float() if t.dtype == torch.bfloat16 else t).numpy()


def close(got, want, bound, name):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), name
    err = np.where(nan, 0.0, np.abs(got - want))
    bound = np.broadcast_to(np.where(nan, 0.0, bound), err.shape)
    bad = err > bound
    assert not bad.any(), (name, int(bad.sum()), float((err / np.maximum(bound, 1e-300)).max()))


def routed(T, E, k, seed, spread=1.5):
    r = np.random.default_rng(seed)
    logits = (spread * r.standard_normal((T, E))).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    top = np.take_along_axis(logits.astype(np.float64), idx, axis=1)
    gates = ref.softmax(top).astype(np.float32)
    dgates = r.standard_normal((T, k)).astype(np.float32)
    return logits, idx, gates, dgates


def rel_softmax(logits):
    fin = np.where(np.isfinite(logits), logits, 0.0)
    span = (fin.max() - fin.min()) if logits.size else 0.0
    return (span + logits.shape[1] / 32 + 20) * U


# ---- balance loss and its gradient ----------------------------------------------

BALANCE = [  # T, E, k, sequence bounds (None: one), masked share
    (1, 1, 1, None, 0), (1, 256, 6, None, 0), (8, 256, 6, None, 0), (3, 5, 2, [0, 1, 3], 0), (17, 33, 4, None, 0.3),
    (64, 128, 8, [0, 10, 10, 64], 0), (100, 130, 16, [5, 40, 90], 0.5), (300, 7, 3, [0, 0, 0, 300, 300], 0.2),
    (700, 256, 6, [0, 7, 8, 9, 650, 691], 0.1), (513, 300, 5, None, 0), (257, 1024, 16, [0, 128, 257], 0.1),
    (90, 1023, 2, None, 0), (6000, 64, 2, [0, 1, 4000, 5999], 0.1), (40, 16, 2, list(range(0, 41)), 0.1),
    (9000, 16, 1, None, 0.02), (50, 256, 6, [0, 20, 50], 1.0), (0, 16, 2, None, 0), (0, 16, 2, [0, 0, 0], 0),
    (20, 16, 2, [20, 20], 0), (129, 4, 4, [0, 129], 0),
]


@pytest.mark.parametrize("T,E,k,seq,masked", BALANCE)
def test_balance_loss_and_gradient(moe, T, E, k, seq, masked):
    logits, idx, gates, dgates = routed(T, E, k, 1000 + T + E)
    r = np.random.default_rng(5)
    mask = (r.random(T) >= masked) if masked else None
    coef, dloss = 0.02, 0.5
    kw = dict(seq_offsets=None if seq is None else cu(np.array(seq, np.int32)),
              token_mask=None if mask is None else cu(mask))
    S = 1 if seq is None else len(seq) - 1
    ws = torch.full((moe.moe_balance_workspace_bytes(T, E, S),), 0xA5, dtype=torch.uint8, device="cuda")
    loss, counts, prob, tokens = moe.moe_balance_loss(cu(logits), cu(idx), coef, ws=ws, **kw)
    assert moe.moe_check_device_flag(ws) == 0
    rl, rc, rp, rt = ref.balance(logits, idx, coef, seq, mask)
    assert np.array_equal(host(counts), rc) and np.array_equal(host(tokens), rt)
    rel = rel_softmax(logits) + (T + 40) * U
    close(host(prob), rp, rel * rp, "mean_prob")
    close(host(loss), [rl], (rel + 8 * U) * abs(rl), "loss")
    for dg, dl in ((dgates, dloss), (None, dloss), (dgates, None)):
        got = moe.moe_route_backward(cu(logits), cu(idx), gates=cu(gates), dgates=None if dg is None else cu(dg),
                                     dloss=None if dl is None else torch.full((1,), dl, device="cuda"), coef=coef,
                                     counts=counts, tokens=tokens, ws=ws, **kw)
        want, size = ref.route_backward(logits, idx, gates, dg, dl, coef, seq, mask)
        close(host(got), want, (rel_softmax(logits) + (E / 32 + 2 * k + 20) * U) * size, "dlogits")
        assert moe.moe_check_device_flag(ws) == 0


def test_balance_many_sequences(moe):
    """More sequences than rows, runs of empty ones, the last rows in none."""
    T, E, k, S = 3000, 24, 3, 5000
    logits, idx, gates, dgates = routed(T, E, k, 3)
    r = np.random.default_rng(1)
    seq = np.sort(r.integers(0, T - 20, S + 1)).astype(np.int32)
    seq[1000:3000] = seq[1000]
    kw = dict(seq_offsets=cu(seq))
    ws = torch.zeros(moe.moe_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device="cuda")
    loss, counts, prob, tokens = moe.moe_balance_loss(cu(logits), cu(idx), 1.0, ws=ws, **kw)
    assert moe.moe_check_device_flag(ws) == 0
    rl, rc, rp, rt = ref.balance(logits, idx, 1.0, seq)
    assert np.array_equal(host(counts), rc) and np.array_equal(host(tokens), rt)
    rel = rel_softmax(logits) + (T + 40) * U
    close(host(prob), rp, rel * rp, "mean_prob")
    close(host(loss), [rl], (rel + 8 * U) * abs(rl), "loss")
    d = moe.moe_route_backward(cu(logits), cu(idx), dloss=torch.ones(1, device="cuda"), coef=1.0, counts=counts,
                               tokens=tokens, **kw)
    want, size = ref.route_backward(logits, idx, None, None, 1.0, 1.0, seq)
    close(host(d), want, (rel_softmax(logits) + 30 * U) * size, "dlogits")


def test_balance_gradient_against_differences(moe):
    """The loss's slope along a direction, from the loss itself (the counts are
    constants): central differences of the 64-bit definition."""
    T, E, k, seq = 24, 20, 3, [0, 9, 24]
    logits, idx, gates, dgates = routed(T, E, k, 77)
    kw = dict(seq_offsets=cu(np.array(seq, np.int32)))
    loss, counts, prob, tokens = moe.moe_balance_loss(cu(logits), cu(idx), 1.0, **kw)
    d = host(moe.moe_route_backward(cu(logits), cu(idx), gates=cu(gates), dgates=cu(dgates),
                                    dloss=torch.ones(1, device="cuda"), coef=1.0, counts=counts, tokens=tokens, **kw))

    def value(z):
        top = np.take_along_axis(z, idx, axis=1)
        return ref.balance(z, idx, 1.0, seq)[0] + (ref.softmax(top) * dgates).sum()

    r = np.random.default_rng(3)
    for _ in range(4):
        v = r.standard_normal((T, E))
        h = 1e-4
        z = logits.astype(np.float64)
        slope = (value(z + h * v) - value(z - h * v)) / (2 * h)
        # third derivatives of order 10 |v|^3 h^2, and the fp32 gradient
        assert abs(slope - (d * v).sum()) <= 10 * T * 27 * h * h + 1e-5 * np.abs(d * v).sum()


def test_balance_odd_rows(moe):
    """Rows of -inf, NaN, +inf, the type's lowest value, and masked logits."""
    T, E, k = 12, 40, 4
    logits, idx, gates, dgates = routed(T, E, k, 9)
    low = np.finfo(np.float32).min
    logits[0] = -np.inf
    logits[1, 5:] = -np.inf
    logits[2] = low
    logits[3, 1:] = low
    logits[4] = 80.0
    z = cu(logits)
    mask = np.ones(T, bool)
    loss, counts, prob, tokens = moe.moe_balance_loss(z, cu(idx), 1.0, token_mask=cu(mask))
    rl, rc, rp, rt = ref.balance(logits, idx, 1.0, None, mask)
    rel = (200 + E / 32 + 20 + T) * U
    close(host(prob), rp, rel * rp, "mean_prob")
    close(host(loss), [rl], rel * rl, "loss")
    d = moe.moe_route_backward(z, cu(idx), dloss=torch.ones(1, device="cuda"), coef=1.0, counts=counts, tokens=tokens,
                               token_mask=cu(mask))
    want, size = ref.route_backward(logits, idx, None, None, 1.0, 1.0, None, mask)
    close(host(d), want, 2 * rel * size + 1e-40, "dlogits")
    # NaN and +inf stay in their rows, and outside the loss when masked
    logits[6, 3] = np.nan
    logits[7, 3] = np.inf
    mask[6] = mask[7] = False
    loss, counts, prob, tokens = moe.moe_balance_loss(cu(logits), cu(idx), 1.0, token_mask=cu(mask))
    d = moe.moe_route_backward(cu(logits), cu(idx), dloss=torch.ones(1, device="cuda"), coef=1.0, counts=counts,
                               tokens=tokens, token_mask=cu(mask))
    assert np.isfinite(host(loss)).all() and np.isfinite(host(prob)).all() and np.isfinite(host(d)).all()
    mask[6] = True
    d = host(moe.moe_route_backward(cu(logits), cu(idx), dloss=torch.ones(1, device="cuda"), coef=1.0, counts=counts,
                                    tokens=tokens, token_mask=cu(mask)))
    assert np.isnan(d[6]).all() and np.isfinite(np.delete(d, 6, axis=0)).all()


def test_route_backward_same_expert_twice_and_bad_ids(moe):
    T, E, k = 5, 12, 3
    logits, idx, gates, dgates = routed(T, E, k, 21)
    idx[1] = [4, 4, 4]
    idx[2, 1] = E
    idx[3, 2] = -1
    ws = torch.zeros(moe.moe_balance_workspace_bytes(T, E, 1), dtype=torch.uint8, device="cuda")
    loss, counts, prob, tokens = moe.moe_balance_loss(cu(logits), cu(idx), 1.0, ws=ws)
    assert moe.moe_check_device_flag(ws) == moe.FLAG_BAD_EXPERT
    assert np.array_equal(host(counts), ref.balance(logits, idx, 1.0)[1])
    flag = torch.zeros(4, dtype=torch.uint8, device="cuda")
    d = moe.moe_route_backward(cu(logits), cu(idx), gates=cu(gates), dgates=cu(dgates), ws=flag)
    assert moe.moe_check_device_flag(flag) == moe.FLAG_BAD_EXPERT
    want, size = ref.route_backward(logits, idx, gates, dgates)
    # (a bad id takes part in its row's sum of gates and gradients)
    close(host(d), want, 40 * U * size, "dlogits")


def test_balance_bad_offsets_raise_the_flag(moe):
    T, E, k = 40, 16, 2
    logits, idx, _, _ = routed(T, E, k, 31)
    for bad in ([0, 30, 20, 40], [-3, 10, 40], [0, 10, 41]):
        ws = torch.zeros(moe.moe_balance_workspace_bytes(T, E, len(bad) - 1), dtype=torch.uint8, device="cuda")
        moe.moe_balance_loss(cu(logits), cu(idx), 1.0, seq_offsets=cu(np.array(bad, np.int32)), ws=ws)
        assert moe.moe_check_device_flag(ws) == moe.FLAG_BOUNDS


# ---- router projection --------------------------------------------------------------

def pow2_rows(x):
    """A few rows and channels far from 1."""
    x[::7] *= 2.0 ** 9
    x[3::11] *= 2.0 ** -14
    x[:, ::13] *= 16.0
    return x


@pytest.mark.parametrize("T,H,E,kind", [
    (1, 128, 1, "ckpt"), (1, 32, 3, "bf16"), (5, 96, 7, "bf16"), (64, 256, 16, "ckpt"), (63, 128, 65, "ckpt"),
    (130, 512, 256, "ckpt"), (257, 288, 100, "bf16"), (40, 4096, 256, "bf16"), (1000, 256, 33, "ckpt"),
    (129, 384, 1024, "ckpt"), (70, 160, 1023, "bf16"), (2500, 640, 8, "ckpt"), (333, 1056, 260, "bf16"),
    # either side of the rule on the number of tokens, with the smallest and odd sizes
    (65, 32, 1, "bf16"), (300, 128, 1, "ckpt"), (66, 96, 3, "bf16"), (100, 32, 7, "bf16"), (65, 128, 65, "ckpt"),
    (64, 160, 1023, "bf16"), (31, 32, 1024, "bf16"), (33, 640, 130, "ckpt"), (1, 4096, 2, "bf16"),
    (1500, 256, 5, "bf16"), (1100, 512, 513, "ckpt"),
    (128, 96, 70, "bf16"), (129, 2048, 600, "bf16"), (256, 1024, 512, "ckpt"), (256, 1056, 512, "bf16"),
    (257, 32, 1, "bf16"), (300, 96, 3, "bf16"), (290, 32, 7, "bf16"), (320, 128, 65, "ckpt"), (200, 256, 100, "ckpt"),
    (512, 1024, 512, "ckpt"), (511, 1056, 510, "bf16"), (512, 1152, 512, "ckpt"), (513, 32, 1, "bf16"),
    (513, 128, 3, "ckpt"),
    (512, 64, 130, "bf16"), (700, 384, 70, "ckpt"), (640, 896, 300, "ckpt"), (1030, 128, 9, "ckpt"),
])
def test_router_backward(moe, T, H, E, kind):
    r = np.random.default_rng(T + H + E)
    dl = (1e-3 * r.standard_normal((T, E)) * np.exp(2 * r.standard_normal((T, E)))).astype(np.float32)
    dl[T // 2] = 0
    w = (0.02 * r.standard_normal((E, H))).astype(np.float32)
    xb = bf16(pow2_rows(r.standard_normal((T, H))))
    src = dict(x=xb)
    x = host(xb).astype(np.float64)
    if kind == "ckpt":
        codes, scales = moe.moe_ckpt_pack(xb)
        src = dict(codes=codes, scales=scales)
        x = ref.ckpt_value(host(codes), host(scales))
    ws = torch.full((moe.moe_router_backward_workspace_bytes(T, H, E),), 0xA5, dtype=torch.uint8, device="cuda")
    dx, dw, db = moe.moe_router_logits_backward(cu(dl), cu(w), ws=ws, **src)
    assert moe.moe_check_device_flag(ws) == 0
    d64, w64 = dl.astype(np.float64), w.astype(np.float64)
    want = d64 @ w64
    size = np.abs(d64) @ np.abs(w64)
    close(host(dx), want, BF * np.abs(want) + (2.0 ** -14 + (3 * E + 8) * 2 * U) * size, "dx")
    size = np.abs(d64).T @ np.abs(x)
    bw = (3 * T + 8) * 2 * U * size
    close(host(dw), d64.T @ x, bw, "dw")
    close(host(db), d64.sum(0), (T + 8) * U * np.abs(d64).sum(0), "dbias")
    # accumulation, and each output alone
    base = r.standard_normal((E, H)).astype(np.float32)
    bb = r.standard_normal(E).astype(np.float32)
    _, dw2, db2 = moe.moe_router_logits_backward(cu(dl), cu(w), accumulate=True, out=(None, cu(base), cu(bb)), **src)
    close(host(dw2), base + d64.T @ x, bw + U * np.abs(base) + U * size, "dw accumulated")
    close(host(db2), bb + d64.sum(0), (T + 9) * U * np.abs(d64).sum(0) + U * np.abs(bb), "dbias accumulated")
    dx3 = moe.moe_router_logits_backward(cu(dl), cu(w), out=(torch.empty_like(dx), None, None))[0]
    assert torch.equal(dx3, dx)


@pytest.mark.parametrize("T", [96, 400])
def test_router_backward_wide_range(moe, T):
    """Gradients whose parts span the exponent range: the three bf16 parts of an
    fp32 value are exact, so large and small rows do not disturb each other."""
    r = np.random.default_rng(8)
    H, E = 128, 32
    dl = (r.standard_normal((T, E)) * np.exp2(r.integers(-60, 20, (T, E)))).astype(np.float32)
    xb = bf16(r.standard_normal((T, H)))
    _, dw, db = moe.moe_router_logits_backward(cu(dl), cu(np.zeros((E, H), np.float32)), x=xb)
    d64, x = dl.astype(np.float64), host(xb).astype(np.float64)
    close(host(dw), d64.T @ x, (3 * T + 8) * 2 * U * (np.abs(d64).T @ np.abs(x)), "dw")
    close(host(db), d64.sum(0), (T + 8) * U * np.abs(d64).sum(0), "dbias")


@pytest.mark.parametrize("T,E", [(40, 17), (300, 100), (600, 70), (1300, 300)])
def test_router_backward_not_finite(moe, T, E):
    """A NaN or infinity in dlogits, or in a checkpoint, reaches the sums that hold
    it and no others."""
    r = np.random.default_rng(T)
    H = 384
    dl = (1e-3 * r.standard_normal((T, E))).astype(np.float32)
    xb = bf16(r.standard_normal((T, H)))
    w = (0.02 * r.standard_normal((E, H))).astype(np.float32)
    codes, scales = moe.moe_ckpt_pack(xb)
    clean = moe.moe_router_logits_backward(cu(dl), cu(w), codes=codes, scales=scales)
    bad = dl.copy()
    bad[3, 5] = np.nan
    bad[T - 1, E - 1] = np.inf
    codes[T // 2, 7] = 0x7F
    codes[T - 2, H - 1] = 0xFF
    scales[1, 1] = 255
    dx, dw, db = moe.moe_router_logits_backward(cu(bad), cu(w), codes=codes, scales=scales)
    rows, cols = np.isin(np.arange(E), (5, E - 1)), np.isin(np.arange(H), (7, H - 1)) | (np.arange(H) // 128 == 1)
    hit = torch.from_numpy(rows[:, None] | cols[None]).cuda()
    assert not torch.isfinite(dw[hit]).any() and torch.equal(dw[~hit], clean[1][~hit])
    hit = torch.from_numpy(rows).cuda()
    assert not torch.isfinite(db[hit]).any() and torch.equal(db[~hit], clean[2][~hit])
    hit = torch.from_numpy(np.isin(np.arange(T), (3, T - 1))).cuda()
    assert not torch.isfinite(dx[hit]).any() and torch.equal(dx[~hit], clean[0][~hit])


@pytest.mark.parametrize("T,H,E", [(33, 128, 5), (500, 1152, 70), (600, 384, 33), (2000, 640, 256), (4604, 128, 257),
                                   (700, 2048, 1000)])
def test_router_backward_checkpoint_is_its_values(moe, T, H, E):
    """From a checkpoint and from the bf16 values it restores: the same bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    codes, scales = moe.moe_ckpt_pack(torch.randn(T, H, generator=g, device="cuda").bfloat16())
    dl, w = torch.randn(T, E, generator=g, device="cuda"), torch.randn(E, H, generator=g, device="cuda")
    a = moe.moe_router_logits_backward(dl, w, codes=codes, scales=scales)
    b = moe.moe_router_logits_backward(dl, w, x=moe.moe_ckpt_unpack(codes, scales))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_router_backward_no_tokens(moe):
    E, H = 9, 128
    dl = torch.empty((0, E), device="cuda")
    x = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    dx, dw, db = moe.moe_router_logits_backward(dl, torch.zeros((E, H), device="cuda"), x=x)
    assert dx.shape == (0, H) and not dw.any() and not db.any()
    one = torch.ones((E, H), device="cuda")
    _, dw, db = moe.moe_router_logits_backward(dl, torch.zeros((E, H), device="cuda"), x=x, accumulate=True,
                                               out=(None, one, torch.ones(E, device="cuda")))
    assert bool((dw == 1).all()) and bool((db == 1).all())


# ---- 8-bit checkpoints ------------------------------------------------------------------

@pytest.mark.parametrize("T,K", [(1, 128), (3, 256), (61, 4096), (257, 640), (1000, 128), (5, 16384)])
def test_ckpt_pack_unpack(moe, T, K):
    r = np.random.default_rng(T + K)
    x = r.standard_normal((T, K)) * np.exp2(r.integers(-20, 20, (T, K // 128)).repeat(128, axis=1))
    x[T // 2, :128] = 0
    xb = bf16(x)
    codes, scales = moe.moe_ckpt_pack(xb)
    rc, rs = ref.ckpt_pack(host(xb))
    assert np.array_equal(host(scales), rs)
    assert np.array_equal(host(codes), rc)
    assert np.array_equal(host(moe.moe_ckpt_unpack(codes, scales)), ref.ckpt_value(rc, rs).astype(np.float32))


def test_ckpt_is_the_fp8_projection_input(moe):
    """Codes and scales are those moe_fp8_linear quantises its input to."""
    T, K, N = 37, 512, 128
    r = np.random.default_rng(0)
    x = bf16(r.standard_normal((T, K)) * np.exp2(r.integers(-30, 30, (T, 1))))
    packed = moe.moe_fp8_pack_weights(torch.zeros((N, K), dtype=torch.uint8, device="cuda"),
                                      torch.full((1, K // 128), 127, dtype=torch.uint8, device="cuda"))
    dbg = dict(q=torch.empty((T, K), dtype=torch.uint8, device="cuda"),
               s=torch.empty((T, K // 128), dtype=torch.uint8, device="cuda"))
    moe.moe_fp8_linear(x, packed, N, debug=dbg)
    codes, scales = moe.moe_ckpt_pack(x)
    assert torch.equal(codes, dbg["q"]) and torch.equal(scales, dbg["s"])


def test_ckpt_every_bf16_value(moe):
    """All 65536 bf16 patterns, each in the first place of a block beside a
    neighbour of its own size; and NaN and infinities beside finite values."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    x = np.zeros((65536, 128), np.uint16)
    x[:, 0] = bits
    x[:, 1] = bits ^ 0x8001
    x[:, 77] = 0x3F80
    t = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    codes, scales = moe.moe_ckpt_pack(t)
    rc, rs = ref.ckpt_pack(host(t))
    assert np.array_equal(host(scales), rs)
    assert np.array_equal(host(codes), rc)
    back = host(moe.moe_ckpt_unpack(codes, scales))
    assert np.array_equal(np.isfinite(back), np.isfinite(host(t)))
    # the value: nearest multiple of 2^-3 of its own power of two, inside the block's range
    want = ref.ckpt_value(rc, rs)
    near = torch.from_numpy(np.where(np.isnan(want), 0, want).astype(np.float32)).to(torch.bfloat16).float().numpy()
    assert np.array_equal(np.where(np.isnan(back), 0, back), near)


def test_ckpt_strided_rows(moe):
    """Halves of a wider tensor, and rows that must stay untouched."""
    r = np.random.default_rng(4)
    wide = bf16(r.standard_normal((19, 640)))
    a = moe.moe_ckpt_pack(wide[:, 128:512])
    b = moe.moe_ckpt_pack(wide[:, 128:512].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out = torch.full((20, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_ckpt_unpack(*a, out=out[:19, 128:512])
    assert torch.equal(out[:19, 128:512].contiguous(), moe.moe_ckpt_unpack(*b))
    assert bool((out[:, :128] == 7).all()) and bool((out[:, 512:] == 7).all()) and bool((out[19] == 7).all())
    with pytest.raises(moe.MoeError):
        moe.moe_ckpt_pack(wide[:, 4:132])          # rows that start off a 16-byte bound
    with pytest.raises(moe.MoeError):
        moe.moe_ckpt_pack(wide.t())
    with pytest.raises(moe.MoeError):
        moe.moe_ckpt_pack(wide.float())


def test_ckpt_no_rows(moe):
    codes, scales = moe.moe_ckpt_pack(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    assert moe.moe_ckpt_unpack(codes, scales).shape == (0, 256)


def test_ckpt_nan_scale_byte(moe):
    codes = torch.full((2, 256), 0x38, dtype=torch.uint8, device="cuda")
    scales = torch.tensor([[127, 255], [0, 254]], dtype=torch.uint8, device="cuda")
    x = host(moe.moe_ckpt_unpack(codes, scales))
    assert (x[0, :128] == 1).all() and np.isnan(x[0, 128:]).all()
    assert (x[1, :128] == 2.0 ** -127).all() and (x[1, 128:] == 2.0 ** 127).all()


# ---- SwiGLU ------------------------------------------------------------------------------

@pytest.mark.parametrize("T,I,need_h", [(1, 128, False), (2, 256, True), (33, 2048, True), (500, 384, False),
                                        (129, 1408, True), (0, 128, True)])
def test_swiglu_backward(moe, T, I, need_h):
    r = np.random.default_rng(T + I)
    gu = 3 * r.standard_normal((T, 2 * I))
    if T:
        gu[0, :64] = np.linspace(-100, 100, 64)
        gu[T // 2, I:I + 128] = 0
    dhb = bf16(r.standard_normal((T, I)))
    codes, scales = moe.moe_ckpt_pack(bf16(gu))
    dgu, h = moe.moe_ckpt_swiglu_backward(codes, scales, dhb, need_h=need_h)
    v = ref.ckpt_value(host(codes), host(scales))
    g, u, dh = v[:, :I], v[:, I:], host(dhb).astype(np.float64)
    dg, du, hh, size = ref.swiglu_backward(g, u, dh)
    # __expf: 2 + 1.173 |x| ulp, __fdividef 2 ulp, then a few fp32 roundings
    slack = (2 * (4 + 1.173 * np.abs(g)) + 12) * 2 * U
    tiny = 1e-36                        # below it exp(-|g|) and bf16 leave the normal range
    got = host(dgu).astype(np.float64)
    close(got[:, :I], dg, BF * np.abs(dg) + slack * size + tiny, "dg")
    close(got[:, I:], du, (BF + 2 * slack) * np.abs(du) + tiny, "du")
    if need_h:
        close(host(h), hh, (BF + 2 * slack) * np.abs(hh) + tiny, "h")
    else:
        assert h is None
    # dh as a slice of a wider tensor
    if T > 1:
        wide = torch.zeros((T, I + 64), dtype=torch.bfloat16, device="cuda")
        wide[:, 32:32 + I] = dhb
        assert torch.equal(moe.moe_ckpt_swiglu_backward(codes, scales, wide[:, 32:32 + I])[0], dgu)


def test_swiglu_gradient_against_differences(moe):
    r = np.random.default_rng(6)
    T, I = 3, 128
    codes, scales = moe.moe_ckpt_pack(bf16(r.standard_normal((T, 2 * I))))
    v = ref.ckpt_value(host(codes), host(scales))
    dhb = bf16(r.standard_normal((T, I)))
    dh = host(dhb).astype(np.float64)
    d = host(moe.moe_ckpt_swiglu_backward(codes, scales, dhb)[0]).astype(np.float64)

    def value(v):
        g, u = v[:, :I], v[:, I:]
        return (dh * g / (1 + np.exp(-g)) * u).sum()

    t = r.standard_normal((T, 2 * I))
    e = 1e-4
    slope = (value(v + e * t) - value(v - e * t)) / (2 * e)
    # third derivatives below 1 per term times |t|^3 u, and bf16 rounding of each entry
    assert abs(slope - (d * t).sum()) <= BF * np.abs(d * t).sum() + T * I * 100 * e * e


# ---- weight gradient -----------------------------------------------------------------------

def wgrad_case(moe, X, R, N, K, seed):
    r = np.random.default_rng(seed)
    codes, scales = moe.moe_ckpt_pack(bf16(pow2_rows(r.standard_normal((X, K)))))
    dyb = bf16(1e-2 * r.standard_normal((R, N)) * np.exp2(r.integers(-6, 6, (R, 1))))
    return codes, scales, dyb, ref.ckpt_value(host(codes), host(scales)), host(dyb).astype(np.float64)


def wgrad_bound(dy, x):
    return (len(dy) + 8) * 2 * U * (np.abs(dy).T @ np.abs(x))


@pytest.mark.parametrize("R,N,K", [(1, 8, 128), (1, 256, 256), (2, 136, 128), (7, 64, 384),
                                   (31, 264, 128), (64, 128, 512),
                                   (65, 512, 256), (127, 1024, 128), (200, 248, 640), (513, 256, 256), (1000, 72, 896),
                                   (4604, 128, 128), (5000, 512, 1024), (0, 64, 128)])
def test_wgrad_dense(moe, R, N, K):
    codes, scales, dyb, x, dy = wgrad_case(moe, R, R, N, K, R + N + K)
    ws = torch.full((moe.moe_ckpt_wgrad_workspace_bytes(R, N, K),), 0xA5, dtype=torch.uint8, device="cuda")
    dw = moe.moe_ckpt_wgrad(dyb, codes, scales, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0
    want, bound = dy.T @ x, wgrad_bound(dy, x)
    close(host(dw), want, bound, "dw")
    assert torch.equal(dw, moe.moe_ckpt_wgrad(dyb, codes, scales))       # the same bits each time
    base = torch.randn((N, K), device="cuda")
    b64 = host(base).astype(np.float64)
    got = moe.moe_ckpt_wgrad(dyb, codes, scales, dw=base, accumulate=True, ws=ws)
    close(host(got), b64 + want, bound + U * (np.abs(b64) + np.abs(want)) + U * bound, "dw accumulated")


@pytest.mark.parametrize("T,k,G,N,K,via", [
    (1, 1, 2, 64, 128, "perm"), (9, 2, 5, 136, 256, "perm"), (100, 6, 16, 128, 128, "perm"),
    (300, 3, 7, 264, 384, "sorted"), (64, 1, 64, 8, 128, "sorted"), (700, 2, 3, 512, 256, "perm"),
    (50, 4, 256, 128, 128, "perm"), (30, 1, 1, 256, 128, "sorted"),
])
def test_wgrad_by_expert(moe, T, k, G, N, K, via):
    """The groups of moe_sort: empty experts, odd sizes, rows through perm."""
    r = np.random.default_rng(T * k + G)
    R = T * k
    # an uneven draw that leaves some experts without a token
    p = 1.0 / np.arange(1, G + 1) ** 1.2
    idx = r.choice(G, size=(T, k), p=p / p.sum()).astype(np.int32)
    perm, pos, offsets = moe.moe_sort(cu(idx), G)
    codes, scales, dyb, x, dy = wgrad_case(moe, T if via == "perm" else R, R, N, K, R)
    ws = torch.full((moe.moe_ckpt_wgrad_workspace_bytes(R, N, K, G),), 0xA5, dtype=torch.uint8, device="cuda")
    kw = dict(perm=perm, k=k) if via == "perm" else {}
    dw = moe.moe_ckpt_wgrad(dyb, codes, scales, offsets=offsets, ws=ws, **kw)
    assert moe.moe_check_device_flag(ws) == 0
    off, pm = host(offsets), host(perm)
    got = host(dw)
    for g in range(G):
        rows = np.arange(off[g], off[g + 1])
        xr = x[pm[rows] // k] if via == "perm" else x[rows]
        close(got[g], dy[rows].T @ xr, wgrad_bound(dy[rows], xr), f"dw[{g}]")
    base = torch.ones_like(dw)
    acc = moe.moe_ckpt_wgrad(dyb, codes, scales, offsets=offsets, dw=base, accumulate=True, ws=ws, **kw)
    empty = np.flatnonzero(off[1:] == off[:-1])
    assert (host(acc)[empty] == 1).all() and (got[empty] == 0).all()


@pytest.mark.parametrize("R,N,K,G,seed", [
    (1, 8, 128, 1, 0), (40, 520, 640, 1, 1), (63, 256, 128, 3, 2), (128, 1032, 384, 1, 3), (129, 264, 256, 1, 4),
    (200, 64, 512, 40, 5), (500, 776, 256, 4, 6), (900, 328, 1152, 16, 7), (2000, 136, 128, 16, 8), (5, 512, 512, 9, 9),
])
def test_wgrad_through_the_identity_table(moe, R, N, K, G, seed):
    """With perm = 0, 1, .. a call takes the checkpoint's values from the
    workspace, without it it may convert the codes in the product: the same bits,
    for groups of any sizes, empty ones and rows in front and behind included."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes, scales = moe.moe_ckpt_pack(torch.randn(R, K, generator=g, device="cuda").bfloat16())
    dy = torch.randn(R, N, generator=g, device="cuda").bfloat16()
    cut = torch.randint(0, R + 1, (G + 1,), generator=g, device="cuda").sort()[0]
    dy[int(cut[-1]):] = float("nan")
    dy[: int(cut[0])] = float("inf")
    off, perm = cut.int(), torch.arange(R, dtype=torch.int32, device="cuda")
    ws = torch.full((moe.moe_ckpt_wgrad_workspace_bytes(R, N, K, G),), 0xFF, dtype=torch.uint8, device="cuda")
    a = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0
    b = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, perm=perm)
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    base = torch.randn(a.shape, generator=g, device="cuda")
    c = moe.moe_ckpt_wgrad(dy, codes, scales, offsets=off, dw=base.clone(), accumulate=True)
    assert torch.equal(c, base + a)


def test_wgrad_groups_do_not_touch(moe):
    """NaN and infinities in one group's rows, and in rows behind the last one,
    stay out of the other groups."""
    N, K, G = 128, 256, 3
    off = np.array([0, 37, 37 + 61, 37 + 61 + 5], np.int32)
    R = 120
    codes, scales, dyb, x, dy = wgrad_case(moe, R, R, N, K, 99)
    dyb[40, 3] = float("inf")
    dyb[41, 4] = float("nan")
    dyb[103:] = float("nan")
    codes[50, 130] = 0x7F
    codes[105:] = 0xFF
    dw = host(moe.moe_ckpt_wgrad(dyb, codes, scales, offsets=cu(off)))
    for g in (0, 2):
        rows = np.arange(off[g], off[g + 1])
        close(dw[g], dy[rows].T @ x[rows], wgrad_bound(dy[rows], x[rows]), f"dw[{g}]")
    assert np.isnan(dw[1][4]).all() and not np.isfinite(dw[1][3]).any() and np.isnan(dw[1][:, 130]).all()
    rest = np.delete(np.delete(dw[1], [3, 4], axis=0), 130, axis=1)
    assert np.isfinite(rest).all()


def test_wgrad_strided_gradient_and_bad_tables(moe):
    R, N, K = 90, 128, 128
    codes, scales, dyb, x, dy = wgrad_case(moe, R, R, N, K, 5)
    wide = torch.full((R, N + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 24:24 + N] = dyb
    want = moe.moe_ckpt_wgrad(dyb, codes, scales)
    assert torch.equal(moe.moe_ckpt_wgrad(wide[:, 24:24 + N], codes, scales), want)
    ws = torch.zeros(moe.moe_ckpt_wgrad_workspace_bytes(R, N, K, 2), dtype=torch.uint8, device="cuda")
    for off in ([0, 60, 40], [-1, 5, 90], [0, 50, 91]):
        moe.moe_ckpt_wgrad(dyb, codes, scales, offsets=cu(np.array(off, np.int32)), ws=ws)
        assert moe.moe_check_device_flag(ws) == moe.FLAG_BOUNDS
    perm = cu(np.arange(R, dtype=np.int32))
    perm[7] = 5 * R
    moe.moe_ckpt_wgrad(dyb, codes, scales, perm=perm, ws=ws)
    assert moe.moe_check_device_flag(ws) == moe.FLAG_BOUNDS
    moe.moe_ckpt_wgrad(dyb, codes, scales, ws=ws)
    assert moe.moe_check_device_flag(ws) == 0


def test_wgrad_exponent_range(moe):
    """Blocks near both ends of the scale range keep their values as bf16."""
    R, N, K = 40, 64, 256
    codes, scales, dyb, x, dy = wgrad_case(moe, R, R, N, K, 12)
    scales[:, 0] = 3
    scales[:, 1] = 230
    x = ref.ckpt_value(host(codes), host(scales))
    dyb = bf16(2.0 ** -20 * np.random.default_rng(1).standard_normal((R, N)))
    dy = host(dyb).astype(np.float64)
    dw = host(moe.moe_ckpt_wgrad(dyb, codes, scales)).astype(np.float64)
    close(dw[:, 128:], (dy.T @ x)[:, 128:], wgrad_bound(dy, x)[:, 128:], "large")
    # sums below fp32's normal range may be flushed
    close(dw[:, :128], (dy.T @ x)[:, :128], wgrad_bound(dy, x)[:, :128] + R * 2.0 ** -126, "small")


def test_wgrad_rows_behind_the_last_group_take_no_part(moe):
    """A sort that left pairs out: rows and table entries behind the last group."""
    R, N, K, k = 200, 64, 128, 2
    codes, scales, dyb, x, dy = wgrad_case(moe, R // k, R, N, K, 77)
    perm = np.random.default_rng(0).permutation(R).astype(np.int32)
    off = np.array([0, 70, 131], np.int32)
    bad = perm.copy()
    bad[131:] = -12345
    ws = torch.zeros(moe.moe_ckpt_wgrad_workspace_bytes(R, N, K, 2), dtype=torch.uint8, device="cuda")
    got = host(moe.moe_ckpt_wgrad(dyb, codes, scales, offsets=cu(off), perm=cu(bad), k=k, ws=ws))
    assert moe.moe_check_device_flag(ws) == 0
    for g in range(2):
        rows = np.arange(off[g], off[g + 1])
        close(got[g], dy[rows].T @ x[perm[rows] // k], wgrad_bound(dy[rows], x[perm[rows] // k]), f"dw[{g}]")
    bad[3] = -1
    moe.moe_ckpt_wgrad(dyb, codes, scales, offsets=cu(off), perm=cu(bad), k=k, ws=ws)
    assert moe.moe_check_device_flag(ws) == moe.FLAG_BOUNDS


# ---- offsets beyond 32 bits -----------------------------------------------------------------

def test_element_offsets_beyond_32_bits(moe):
    """The last rows of tensors of more than 2^31 elements are those of the rows
    alone, and the sum over all rows is that of its parts."""
    T, K = 530000, 4096                       # 2.17e9 elements
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = moe.moe_ckpt_pack(x)
    c, s = moe.moe_ckpt_pack(x[-3:].clone())
    assert torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s)
    moe.moe_ckpt_unpack(codes, scales, out=x)
    assert torch.equal(x[-3:], moe.moe_ckpt_unpack(c, s))
    dgu, h = moe.moe_ckpt_swiglu_backward(codes, scales, x[:, :K // 2], need_h=True)
    d2, h2 = moe.moe_ckpt_swiglu_backward(c, s, x[-3:, :K // 2])
    assert torch.equal(dgu[-3:], d2)
    del dgu, h, d2
    dy = x[:, 128:136]
    whole = moe.moe_ckpt_wgrad(dy, codes, scales).double()
    parts = sum(moe.moe_ckpt_wgrad(dy[a:b], codes[a:b], scales[a:b]).double()
                for a, b in ((0, T // 3), (T // 3, T - 7), (T - 7, T)))
    # two sums of T terms, drained every 1024 rows (64 truncations) into fp32
    size = float((dy.double() ** 2).sum(0).max().sqrt()) * float((x.double()[:, 0] ** 2).sum().sqrt())
    assert float((whole - parts).abs().max()) <= 2 * (64 * 2 * U + T / 1024 * U) * size
    del x, codes, scales, dy, whole, parts
    T, E, k = 2200000, 1000, 2                # 2.2e9 logits
    z = torch.empty((T, E), device="cuda").normal_()
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    gates = torch.rand((T, k), device="cuda")
    d = moe.moe_route_backward(z, idx, gates, dgates=gates)
    assert torch.equal(d[-5:], moe.moe_route_backward(z[-5:].clone(), idx[-5:], gates[-5:], dgates=gates[-5:]))
    del d
    seq = torch.tensor([0, T - 5, T], dtype=torch.int32, device="cuda")
    _, counts, prob, tokens = moe.moe_balance_loss(z, idx, 1.0, seq_offsets=seq)
    _, c1, p1, _ = moe.moe_balance_loss(z[-5:].clone(), idx[-5:], 1.0)
    assert torch.equal(counts[1], c1[0]) and torch.allclose(prob[1], p1[0], rtol=1e-5, atol=0)
    assert tokens.tolist() == [T - 5, 5, 2]
