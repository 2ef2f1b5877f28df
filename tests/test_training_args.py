"""What the training calls refuse, checked on the host before any launch (no
GPU: the pointers are aligned numbers that nothing reads)."""
import ctypes

import pytest

import fp4_routed_mixture_b200 as moe

L = moe.lib
P = 1 << 20                       # a pointer, 256-byte aligned
Q = 1 << 30                       # another, far from it
BIG = ctypes.c_size_t(1 << 40)
INVALID, SHAPE = -1, -2


def balance(logits=P, idx=P, seq=None, mask=None, T=4, E=16, k=2, S=1, counts=P, prob=P, tokens=P, loss=P, ws=P,
            n=BIG):
    return L.moe_balance_loss(logits, idx, seq, mask, T, E, k, S, 0.01, counts, prob, tokens, loss, ws, n, None)


def route(logits=P, idx=P, gates=P, dgates=P, dloss=P, counts=P, tokens=P, seq=None, mask=None, T=4, E=16, k=2, S=1,
          out=Q, flag=None):
    return L.moe_route_backward(logits, idx, gates, dgates, dloss, counts, tokens, seq, mask, T, E, k, S, 0.01, out,
                                flag, None)


def router(dl=P, x=P, codes=None, scales=None, w=P, T=4, H=128, E=16, dx=P, dw=P, db=P, acc=0, ws=P, n=BIG):
    return L.moe_router_logits_backward(dl, x, codes, scales, w, T, H, E, dx, dw, db, acc, ws, n, None)


def pack(x=P, ld=128, T=4, K=128, codes=P, scales=P):
    return L.moe_ckpt_pack(x, ld, T, K, codes, scales, None)


def unpack(x=P, ld=128, T=4, K=128, codes=P, scales=P):
    return L.moe_ckpt_unpack(codes, scales, T, K, x, ld, None)


def swiglu(codes=P, scales=P, dh=P, ld=128, T=4, I=128, dgu=P, h=None):
    return L.moe_ckpt_swiglu_backward(codes, scales, dh, ld, T, I, dgu, h, None)


def wgrad(dy=P, ld=64, codes=P, scales=P, off=None, perm=None, k=1, R=4, X=4, N=64, K=128, G=1, dw=P, acc=0, ws=P,
          n=BIG):
    return L.moe_ckpt_wgrad(dy, ld, codes, scales, off, perm, k, R, X, N, K, G, dw, acc, ws, n, None)


@pytest.mark.parametrize("fn,args,status", [
    (balance, dict(logits=None), INVALID), (balance, dict(idx=None), INVALID), (balance, dict(counts=None), INVALID),
    (balance, dict(tokens=None), INVALID), (balance, dict(loss=None), INVALID), (balance, dict(ws=None), INVALID),
    (balance, dict(T=-1), INVALID), (balance, dict(E=0), SHAPE), (balance, dict(E=1025), SHAPE),
    (balance, dict(k=0), SHAPE), (balance, dict(k=17, E=64), SHAPE), (balance, dict(E=2, k=3), SHAPE),
    (balance, dict(S=0, seq=P), SHAPE), (balance, dict(S=65536, seq=P), SHAPE), (balance, dict(S=2), INVALID),
    (balance, dict(ws=P + 16), INVALID), (balance, dict(logits=P + 2), INVALID),
    (balance, dict(n=ctypes.c_size_t(100)), INVALID),
    (route, dict(dgates=None, dloss=None), INVALID), (route, dict(logits=None), INVALID),
    (route, dict(gates=None), INVALID), (route, dict(idx=None), INVALID), (route, dict(counts=None), INVALID),
    (route, dict(tokens=None), INVALID), (route, dict(out=None), INVALID), (route, dict(out=P), INVALID),
    (route, dict(out=P + 4 * 16 * 4 - 4), INVALID), (route, dict(S=3), INVALID), (route, dict(E=1025), SHAPE),
    (router, dict(dl=None), INVALID), (router, dict(x=None), INVALID), (router, dict(w=None), INVALID),
    (router, dict(dx=None, dw=None, db=None), INVALID), (router, dict(codes=P, scales=P), INVALID),
    (router, dict(x=None, codes=P), INVALID), (router, dict(x=None, scales=P), INVALID),
    (router, dict(x=None, codes=P, scales=P, H=160), SHAPE), (router, dict(H=48), SHAPE), (router, dict(H=0), SHAPE),
    (router, dict(E=0), SHAPE), (router, dict(E=1025), SHAPE), (router, dict(T=-1), INVALID),
    (router, dict(acc=2), INVALID), (router, dict(dl=P + 4), INVALID), (router, dict(dw=P + 4), INVALID),
    (router, dict(ws=P + 128), INVALID), (router, dict(n=ctypes.c_size_t(8)), INVALID),
    (pack, dict(x=None), INVALID), (pack, dict(codes=None), INVALID), (pack, dict(scales=None), INVALID),
    (pack, dict(K=64, ld=64), SHAPE), (pack, dict(K=0), SHAPE), (pack, dict(T=-1), INVALID),
    (pack, dict(ld=120), INVALID), (pack, dict(ld=132), INVALID), (pack, dict(x=P + 8), INVALID),
    (pack, dict(codes=P + 8), INVALID),
    (unpack, dict(x=None), INVALID), (unpack, dict(K=130, ld=136), SHAPE), (unpack, dict(ld=127), INVALID),
    (unpack, dict(x=P + 2), INVALID),
    (swiglu, dict(codes=None), INVALID), (swiglu, dict(dh=None), INVALID), (swiglu, dict(dgu=None), INVALID),
    (swiglu, dict(I=64, ld=64), SHAPE), (swiglu, dict(ld=64), INVALID), (swiglu, dict(h=P + 2), INVALID),
    (swiglu, dict(T=-3), INVALID),
    (wgrad, dict(dy=None), INVALID), (wgrad, dict(codes=None), INVALID), (wgrad, dict(scales=None), INVALID),
    (wgrad, dict(dw=None), INVALID), (wgrad, dict(ws=None), INVALID), (wgrad, dict(N=63), SHAPE),
    (wgrad, dict(N=60, ld=64), SHAPE), (wgrad, dict(K=64), SHAPE), (wgrad, dict(G=0, off=P), SHAPE),
    (wgrad, dict(G=1025, off=P), SHAPE), (wgrad, dict(G=2), INVALID), (wgrad, dict(R=-1), INVALID),
    (wgrad, dict(X=3), INVALID), (wgrad, dict(X=0, perm=P), INVALID), (wgrad, dict(perm=P, k=0), INVALID),
    (wgrad, dict(ld=56), INVALID), (wgrad, dict(ld=68), INVALID), (wgrad, dict(acc=3), INVALID),
    (wgrad, dict(dw=P + 4), INVALID), (wgrad, dict(dy=P + 2), INVALID), (wgrad, dict(n=ctypes.c_size_t(8)), INVALID),
])
def test_refused(fn, args, status):
    before = moe.moe_launch_count()
    assert fn(**args) == status
    assert moe.binding.last_error() != ""
    assert moe.moe_launch_count() == before


M = (1 << 30) + 1                 # more rows than a call takes
F = [(k + 2) << 36 for k in range(10)]      # pointers 64 GB apart


@pytest.mark.parametrize("fn,args,status", [
    (balance, dict(T=M), SHAPE), (route, dict(T=M), SHAPE), (router, dict(T=M), SHAPE), (pack, dict(T=M), SHAPE),
    (unpack, dict(T=M), SHAPE), (swiglu, dict(T=M), SHAPE), (wgrad, dict(R=M, X=M), SHAPE),
    (wgrad, dict(R=4, X=M), SHAPE), (balance, dict(T=(1 << 31) - 1), SHAPE), (router, dict(H=(1 << 20) + 32), SHAPE),
])
def test_too_large(fn, args, status):
    assert fn(**args) == status


ROUTER = dict(dl=F[0], x=F[1], w=F[2], dx=F[3], dw=F[4], db=F[5], ws=F[6], T=4, H=128, E=16)
SWIGLU = dict(codes=F[0], scales=F[1], dh=F[2], dgu=F[3], h=F[4])
WGRAD = dict(dy=F[0], codes=F[1], scales=F[2], dw=F[3], ws=F[4])


@pytest.mark.parametrize("fn,args", [
    (router, {**ROUTER, "dx": F[1]}), (router, {**ROUTER, "dx": F[1] + 4 * 128 * 2 - 16}),
    (router, {**ROUTER, "dx": F[0]}), (router, {**ROUTER, "dx": F[2]}), (router, {**ROUTER, "dw": F[2]}),
    (router, {**ROUTER, "dw": F[0]}), (router, {**ROUTER, "dw": F[3]}), (router, {**ROUTER, "db": F[0] + 16}),
    (router, {**ROUTER, "x": None, "codes": F[1], "scales": F[7], "dx": F[1]}),
    (pack, dict(x=F[0], codes=F[0], scales=F[1])), (pack, dict(x=F[0], codes=F[1], scales=F[0] + 4 * 256 - 1)),
    (unpack, dict(x=F[0], codes=F[0] + 512, scales=F[1])),
    (unpack, dict(x=F[0], ld=256, codes=F[0] + 1536, scales=F[1])),
    (swiglu, {**SWIGLU, "dgu": F[0]}), (swiglu, {**SWIGLU, "dgu": F[2]}), (swiglu, {**SWIGLU, "h": F[2]}),
    (swiglu, {**SWIGLU, "h": F[3] + 16}), (swiglu, {**SWIGLU, "h": F[0]}),
    (wgrad, {**WGRAD, "dw": F[0]}), (wgrad, {**WGRAD, "dw": F[1] + 496}),
])
def test_overlapping_outputs_refused(fn, args):
    before = moe.moe_launch_count()
    assert fn(**args) == INVALID
    assert "overlap" in moe.binding.last_error()
    assert moe.moe_launch_count() == before


def test_size_queries():
    assert moe.moe_balance_workspace_bytes(0, 1, 1) > 0
    # a workspace for T_max serves every smaller call
    for E, S in ((256, 1), (7, 300)):
        sizes = [moe.moe_balance_workspace_bytes(T, E, S) for T in (0, 1, 8, 4604, 4736, 4737, 16384, 65536)]
        assert sizes == sorted(sizes)
    sizes = [moe.moe_ckpt_wgrad_workspace_bytes(R, 4096, 4096, 16) for R in (0, 1, 63, 64, 5000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    sizes = [moe.moe_router_backward_workspace_bytes(T, 4096, 256) for T in (0, 1, 8, 64, 65, 4604, 16384, 70000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for bad in (lambda: moe.moe_balance_workspace_bytes(4, 1025, 1), lambda: moe.moe_balance_workspace_bytes(4, 8, 0),
                lambda: moe.moe_router_backward_workspace_bytes(4, 100, 8),
                lambda: moe.moe_ckpt_wgrad_workspace_bytes(4, 60, 128, 1),
                lambda: moe.moe_ckpt_wgrad_workspace_bytes(4, 64, 64, 1),
                lambda: moe.moe_balance_workspace_bytes(M, 8, 1),
                lambda: moe.moe_router_backward_workspace_bytes(M, 64, 8),
                lambda: moe.moe_router_backward_workspace_bytes(4, (1 << 20) + 32, 8),
                lambda: moe.moe_ckpt_wgrad_workspace_bytes(M, 64, 128, 1)):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.status == SHAPE


def test_binding_refuses_host_tensors():
    import torch

    z = torch.zeros(4, 16)
    for call in (lambda: moe.moe_balance_loss(z, torch.zeros(4, 2, dtype=torch.int32), 0.1),
                 lambda: moe.moe_route_backward(z, torch.zeros(4, 2, dtype=torch.int32), dgates=z[:, :2]),
                 lambda: moe.moe_router_logits_backward(z, torch.zeros(16, 128)),
                 lambda: moe.moe_ckpt_pack(torch.zeros(4, 128, dtype=torch.bfloat16)),
                 lambda: moe.moe_ckpt_unpack(torch.zeros(4, 128, dtype=torch.uint8),
                                             torch.zeros(4, 1, dtype=torch.uint8)),
                 lambda: moe.moe_ckpt_swiglu_backward(z, z, z), lambda: moe.moe_ckpt_wgrad(z, z, z)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == INVALID
