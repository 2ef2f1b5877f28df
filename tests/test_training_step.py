"""The training operators together, as a training step uses them, on streams,
in graphs and in parallel."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp4_routed_mixture_b200 as m
    return m


def restored(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double().view(codes.shape[0], -1, 128)
    return (v * torch.exp2(scales.double() - 127).unsqueeze(2)).view(codes.shape)


def make(T=200, H=256, I=128, E=24, k=3, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return dict(T=T, H=H, I=I, E=E, k=k, x=n(T, H).bfloat16(), wr=0.1 * n(E, H), bias=0.1 * n(E),
                gu=n(T, 2 * I).bfloat16(), dy=(0.1 * n(T, H)).bfloat16(), dgates=n(T, k),
                dh=(0.1 * n(T, I)).bfloat16(), seq=torch.tensor([0, 70, 70, T - 11], dtype=torch.int32, device="cuda"),
                dloss=torch.ones(1, device="cuda"))


def buffers(moe, d):
    T, H, I, E, k = (d[n] for n in ("T", "H", "I", "E", "k"))
    S = d["seq"].numel() - 1
    f = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")
    u8 = torch.uint8
    return dict(logits=f(T, E), route=(f(T, k, t=torch.int32), f(T, k)),
                bal=(f(1), f(S, E, t=torch.int32), f(S, E), f(S + 1, t=torch.int32)),
                bws=f(moe.moe_balance_workspace_bytes(T, E, S), t=u8), dlogits=f(T, E),
                xs=(f(T, H, t=u8), f(T, H // 128, t=u8)), gus=(f(T, 2 * I, t=u8), f(T, 2 * I // 128, t=u8)),
                hs=(f(T, I, t=u8), f(T, I // 128, t=u8)),
                rws=f(moe.moe_router_backward_workspace_bytes(T, H, E), t=u8),
                rout=(f(T, H, t=torch.bfloat16), f(E, H), f(E)),
                sout=(f(T, 2 * I, t=torch.bfloat16), f(T, I, t=torch.bfloat16)),
                wws=f(moe.moe_ckpt_wgrad_workspace_bytes(T, 2 * I, H), t=u8), dw1=f(2 * I, H),
                wws2=f(moe.moe_ckpt_wgrad_workspace_bytes(T, H, I), t=u8), dw2=f(H, I))


def step(moe, d, b):
    """Forward of the router with the loss, the checkpoints, and the backward
    pass of the router and of a SwiGLU projection pair."""
    moe.moe_router_logits(d["x"], d["wr"], d["bias"], out=b["logits"])
    idx, gates = moe.moe_route(b["logits"], d["k"], out=b["route"])
    loss, counts, prob, tokens = moe.moe_balance_loss(b["logits"], idx, 0.05, seq_offsets=d["seq"], ws=b["bws"],
                                                      out=b["bal"])
    moe.moe_ckpt_pack(d["x"], out=b["xs"])
    moe.moe_ckpt_pack(d["gu"], out=b["gus"])
    moe.moe_route_backward(b["logits"], idx, gates, dgates=d["dgates"], dloss=d["dloss"], coef=0.05, counts=counts,
                           tokens=tokens, seq_offsets=d["seq"], ws=b["bws"], out=b["dlogits"])
    dx, dwr, db = moe.moe_router_logits_backward(b["dlogits"], d["wr"], codes=b["xs"][0], scales=b["xs"][1],
                                                 ws=b["rws"], out=b["rout"])
    dgu, h = moe.moe_ckpt_swiglu_backward(*b["gus"], d["dh"], need_h=True, out=b["sout"])
    moe.moe_ckpt_pack(h, out=b["hs"])
    moe.moe_ckpt_wgrad(dgu, *b["xs"], dw=b["dw1"], ws=b["wws"])
    moe.moe_ckpt_wgrad(d["dy"], *b["hs"], dw=b["dw2"], ws=b["wws2"])
    return dict(loss=loss, counts=counts, dlogits=b["dlogits"], dx=dx, dwr=dwr, db=db, dgu=dgu, h=h, dw1=b["dw1"],
                dw2=b["dw2"])


def reference(moe, d, b):
    """float64 autograd from the stored activations."""
    x = restored(*b["xs"])
    wr = d["wr"].double().requires_grad_()
    bias = d["bias"].double().requires_grad_()
    xin = d["x"].double().requires_grad_()
    logits = xin @ wr.t() + bias
    logits.retain_grad()
    idx = b["route"][0].long()
    gates = torch.softmax(logits.gather(1, idx), dim=1)
    p = torch.softmax(logits, dim=1)
    off = d["seq"].tolist()
    terms = []
    for a, e in zip(off[:-1], off[1:]):
        if e > a:
            c = torch.bincount(idx[a:e].flatten(), minlength=d["E"]).double()
            terms.append((c * d["E"] / (d["k"] * (e - a)) * p[a:e].mean(0)).sum())
    loss = 0.05 * sum(terms) / len(terms)
    (loss + (gates * d["dgates"].double()).sum()).backward()
    gu = restored(*b["gus"]).requires_grad_()
    g, u = gu.chunk(2, dim=1)
    h = g * torch.sigmoid(g) * u
    h.backward(d["dh"].double())
    return dict(loss=loss.detach().view(1), dlogits=logits.grad, dx=xin.grad, db=bias.grad,
                dwr=logits.grad.t() @ x, dgu=gu.grad, h=h.detach(),
                dw1=b["sout"][0].double().t() @ x, dw2=d["dy"].double().t() @ restored(*b["hs"]))


# relative to the tensor's norm: fp32 sums of up to 256 signed terms, and one
# bf16 rounding (2^-8 at most, so 2^-8 of the norm) where the output is bf16
TOL = dict(loss=1e-5, dlogits=1e-5, dx=2.0 ** -8, db=1e-5, dwr=1e-5, dgu=2.0 ** -8, h=2.0 ** -8, dw1=1e-5, dw2=1e-5)


def test_training_step_matches_autograd(moe):
    d = make()
    b = buffers(moe, d)
    out = step(moe, d, b)
    torch.cuda.synchronize()
    want = reference(moe, d, b)
    for n, tol in TOL.items():
        err = (out[n].double() - want[n]).norm() / want[n].norm()
        assert float(err) <= tol, (n, float(err))
    for w in ("bws", "rws", "wws", "wws2"):
        assert moe.moe_check_device_flag(b[w]) == 0


def snapshot(out):
    return {n: t.clone() for n, t in out.items()}


def same(a, b):
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_captured_step_replays_with_new_inputs(moe):
    d, b = make(seed=1), None
    b = buffers(moe, d)
    step(moe, d, b)                       # warm-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        out = step(moe, d, b)
    for seed in (2, 3):
        new = make(seed=seed)
        for n in ("x", "wr", "bias", "gu", "dy", "dgates", "dh"):
            d[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        eager = step(moe, new, buffers(moe, new))
        torch.cuda.synchronize()
        same(snapshot(out), eager)


def test_two_steps_at_once_on_two_streams(moe):
    """Two steps with workspaces of their own on two streams give the bits of
    the steps run alone."""
    ds = [make(T=900, H=512, I=256, E=40, seed=s) for s in (4, 5)]
    alone = []
    for d in ds:
        out = step(moe, d, buffers(moe, d))
        torch.cuda.synchronize()
        alone.append(snapshot(out))
    bs = [buffers(moe, d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for d, b, s in zip(ds, bs, streams):
            with torch.cuda.stream(s):
                outs.append(step(moe, d, b))
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            same(snapshot(o), a)


def test_stream_argument(moe):
    """Calls on a given stream see that stream's earlier work and allocate there."""
    s = torch.cuda.Stream()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn(64, 256, generator=g, device="cuda").bfloat16()
    dy = torch.randn(64, 128, generator=g, device="cuda").bfloat16()
    want = moe.moe_ckpt_wgrad(dy, *moe.moe_ckpt_pack(x))
    s.wait_stream(torch.cuda.current_stream())
    got = moe.moe_ckpt_wgrad(dy, *moe.moe_ckpt_pack(x, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_captured_autograd_backward(moe):
    """The weight gradient inside a torch.autograd function, its forward and
    backward captured.  (No eager graph over the same leaves may be alive during
    the capture: torch then ties the legacy stream to it.)"""

    class Project(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(*moe.moe_ckpt_pack(x))
            return (x.float() @ w.t()).bfloat16()

        @staticmethod
        def backward(ctx, dy):
            return None, moe.moe_ckpt_wgrad(dy.contiguous(), *ctx.saved_tensors)

    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn(96, 128, generator=g, device="cuda").bfloat16()
    w = torch.randn(64, 128, generator=g, device="cuda", requires_grad=True)
    one = torch.ones(96, 64, device="cuda", dtype=torch.bfloat16)
    want, = torch.autograd.grad(Project.apply(x, w), w, one)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(Project.apply(x, w), w, one)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(Project.apply(x, w), w, one)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_calls_allocate_nothing(moe):
    """With outputs and workspaces given, no call allocates device memory."""
    d = make()
    b = buffers(moe, d)
    step(moe, d, b)
    torch.cuda.synchronize()
    before, free = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0]
    peak = torch.cuda.max_memory_allocated()
    for _ in range(3):
        step(moe, d, b)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before and torch.cuda.max_memory_allocated() == peak
    assert torch.cuda.mem_get_info()[0] == free


def test_one_workspace_for_smaller_calls(moe):
    """A workspace sized for T_max serves smaller calls, whatever an earlier call
    left in it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    T, H, E = 3000, 256, 40
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dl = torch.randn(T, E, generator=g, device="cuda")
    w = torch.randn(E, H, generator=g, device="cuda")
    rws = torch.full((moe.moe_router_backward_workspace_bytes(T, H, E),), 0xFF, dtype=torch.uint8, device="cuda")
    wws = torch.full((moe.moe_ckpt_wgrad_workspace_bytes(T, 64, H),), 0xFF, dtype=torch.uint8, device="cuda")
    bws = torch.full((moe.moe_balance_workspace_bytes(T, E, 5),), 0xFF, dtype=torch.uint8, device="cuda")
    for n in (T, 1, 70, 1500, 128, 129, 257, 700):
        a = moe.moe_router_logits_backward(dl[:n], w, x=x[:n], ws=rws)
        b = moe.moe_router_logits_backward(dl[:n], w, x=x[:n])
        for u, v in zip(a, b):
            assert torch.equal(u, v), n
        ck = moe.moe_ckpt_pack(x[:n])
        dy = x[:n, :64]
        assert torch.equal(moe.moe_ckpt_wgrad(dy, *ck, ws=wws), moe.moe_ckpt_wgrad(dy, *ck)), n
        idx, _ = moe.moe_route(dl[:n].contiguous(), 4)
        seq = torch.tensor([0, n // 3, n // 3, n - n // 5, n], dtype=torch.int32, device="cuda")
        for u, v in zip(moe.moe_balance_loss(dl[:n], idx, 1.0, seq_offsets=seq, ws=bws),
                        moe.moe_balance_loss(dl[:n], idx, 1.0, seq_offsets=seq)):
            assert torch.equal(u, v), n
    for ws in (rws, wws, bws):
        assert moe.moe_check_device_flag(ws) == 0


def test_binding_refusals(moe):
    """Wrong types, shapes, layouts and missing parts are refused by name."""
    d = make(T=32)
    b = buffers(moe, d)
    idx, gates = moe.moe_route(torch.randn(32, 24, device="cuda"), 3)
    logits = torch.randn(32, 24, device="cuda")
    ck = moe.moe_ckpt_pack(d["x"])
    for call in (
            lambda: moe.moe_balance_loss(logits.double(), idx, 0.1),
            lambda: moe.moe_balance_loss(logits, idx.long(), 0.1),
            lambda: moe.moe_balance_loss(logits, idx[:31], 0.1),
            lambda: moe.moe_balance_loss(logits.t(), idx, 0.1),
            lambda: moe.moe_balance_loss(logits, idx, 0.1, token_mask=torch.ones(31, dtype=torch.bool, device="cuda")),
            lambda: moe.moe_balance_loss(logits, idx, 0.1, seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
            lambda: moe.moe_balance_loss(logits, idx, 0.1, seq_offsets=torch.zeros(3, dtype=torch.int32)),
            lambda: moe.moe_balance_loss(logits, idx, 0.1, ws=torch.empty(8, dtype=torch.uint8, device="cuda")),
            lambda: moe.moe_route_backward(logits, idx),
            lambda: moe.moe_route_backward(logits, idx, dgates=gates),
            lambda: moe.moe_route_backward(logits, idx, gates, dgates=gates, out=logits),
            lambda: moe.moe_route_backward(logits, idx, dloss=torch.ones(1, device="cuda"), coef=1.0),
            lambda: moe.moe_router_logits_backward(logits, d["wr"]),
            lambda: moe.moe_router_logits_backward(logits, d["wr"], x=d["x"], codes=ck[0], scales=ck[1]),
            lambda: moe.moe_router_logits_backward(logits, d["wr"], codes=ck[0]),
            lambda: moe.moe_router_logits_backward(logits, d["wr"], x=d["x"], accumulate=True),
            lambda: moe.moe_router_logits_backward(logits, d["wr"][:, :64], x=d["x"]),
            lambda: moe.moe_ckpt_unpack(ck[0], ck[1][:, :1]),
            lambda: moe.moe_ckpt_unpack(ck[0].view(torch.int8), ck[1]),
            lambda: moe.moe_ckpt_swiglu_backward(*ck, d["dh"][:, :64]),
            lambda: moe.moe_ckpt_swiglu_backward(*ck, d["dh"], need_h=True, out=(d["x"], None)),
            lambda: moe.moe_ckpt_wgrad(d["dy"].float(), *ck),
            lambda: moe.moe_ckpt_wgrad(d["dy"].t(), *ck),
            lambda: moe.moe_ckpt_wgrad(d["dy"], ck[0][:31], ck[1][:31]),
            lambda: moe.moe_ckpt_wgrad(d["dy"], *ck, accumulate=True),
            lambda: moe.moe_ckpt_wgrad(d["dy"], *ck, dw=torch.empty(256, 255, device="cuda")),
            lambda: moe.moe_ckpt_wgrad(d["dy"], *ck, perm=idx[:, 0].contiguous(), k=0),
            lambda: moe.moe_ckpt_wgrad(d["dy"], *ck, offsets=torch.zeros(1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(moe.MoeError):
            call()
