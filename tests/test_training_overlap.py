"""No output of a training call may lie on an input, another output or the
workspace: refused on the host, before any launch (no GPU: the pointers are
numbers that nothing reads)."""
import ctypes

import pytest

import fp4_routed_mixture_b200 as moe

L = moe.lib
A = [(k + 2) << 36 for k in range(16)]      # 64 GB apart
BIG = ctypes.c_size_t(1 << 40)
T, E, K, S, H, G = 5, 16, 2, 3, 256, 2


def balance(b):
    return L.moe_balance_loss(b["logits"], b["idx"], b["seq"], b["mask"], T, E, K, S, 0.01, b["counts"], b["prob"],
                              b["tokens"], b["loss"], b["ws"], BIG, None)


def route(b):
    return L.moe_route_backward(b["logits"], b["idx"], b["gates"], b["dgates"], b["dloss"], b["counts"], b["tokens"],
                                b["seq"], b["mask"], T, E, K, S, 0.01, b["out"], b["flag"], None)


def router(b):
    return L.moe_router_logits_backward(b["dl"], b.get("x"), b.get("codes"), b.get("scales"), b["w"], T, H, E, b["dx"],
                                        b["dw"], b["db"], 0, b["ws"], BIG, None)


def pack(b):
    return L.moe_ckpt_pack(b["x"], H + 64, T, H, b["codes"], b["scales"], None)


def unpack(b):
    return L.moe_ckpt_unpack(b["codes"], b["scales"], T, H, b["x"], H + 64, None)


def swiglu(b):
    return L.moe_ckpt_swiglu_backward(b["codes"], b["scales"], b["dh"], H, T, H, b["dgu"], b["h"], None)


def wgrad(b):
    return L.moe_ckpt_wgrad(b["dy"], 64, b["codes"], b["scales"], b["off"], b["perm"], 1, T, T, 64, H, G, b["dw"], 0,
                            b["ws"], BIG, None)


BALANCE_WS = moe.moe_balance_workspace_bytes(T, E, S)
ROUTER_WS = moe.moe_router_backward_workspace_bytes(T, H, E)
WGRAD_WS = moe.moe_ckpt_wgrad_workspace_bytes(T, 64, H, G)
ROWS = 2 * ((T - 1) * (H + 64) + H)         # bytes from the first to the last strided row
CALLS = [  # call, outputs and inputs with their bytes
    (balance, dict(counts=4 * S * E, prob=4 * S * E, tokens=4 * (S + 1), loss=4, ws=BALANCE_WS),
     dict(logits=4 * T * E, idx=4 * T * K, seq=4 * (S + 1), mask=T)),
    (route, dict(out=4 * T * E, flag=4),
     dict(logits=4 * T * E, idx=4 * T * K, gates=4 * T * K, dgates=4 * T * K, dloss=4, counts=4 * S * E,
          tokens=4 * (S + 1), seq=4 * (S + 1), mask=T)),
    (router, dict(dx=2 * T * H, dw=4 * E * H, db=4 * E, ws=ROUTER_WS), dict(dl=4 * T * E, x=2 * T * H, w=4 * E * H)),
    (router, dict(dx=2 * T * H, dw=4 * E * H, db=4 * E, ws=ROUTER_WS),
     dict(dl=4 * T * E, codes=T * H, scales=T * H // 128, w=4 * E * H)),
    (pack, dict(codes=T * H, scales=T * H // 128), dict(x=ROWS)),
    (unpack, dict(x=ROWS), dict(codes=T * H, scales=T * H // 128)),
    (swiglu, dict(dgu=4 * T * H, h=2 * T * H), dict(codes=2 * T * H, scales=T * 2 * H // 128, dh=2 * T * H)),
    (wgrad, dict(dw=4 * G * 64 * H, ws=WGRAD_WS),
     dict(dy=2 * T * 64, codes=T * H, scales=T * H // 128, off=4 * (G + 1), perm=4 * T)),
]
PAIRS = [(i, o, n) for i, (_, outs, ins) in enumerate(CALLS) for k, o in enumerate(outs)
         for n in [*ins, *list(outs)[:k]]]


@pytest.mark.parametrize("call,out,other", PAIRS, ids=[f"{CALLS[i][0].__name__}{i}-{o}-{n}" for i, o, n in PAIRS])
def test_refused(call, out, other):
    """At the same place, and where only the last bytes of one lie on the other
    (the larger one in front; its start stays aligned)."""
    fn, outs, ins = CALLS[call]
    base = dict(zip([*outs, *ins], A))
    sizes = {**outs, **ins}
    big, small = (out, other) if sizes[out] >= sizes[other] else (other, out)
    before = moe.moe_launch_count()
    places = [{**base, out: base[other]}]
    if small != "ws" and sizes[big] > 16:
        places.append({**base, small: base[big] + (sizes[big] - 1) // 16 * 16})
    for b in places:
        assert fn(b) == -1
        assert "overlap" in moe.binding.last_error()
    assert moe.moe_launch_count() == before
