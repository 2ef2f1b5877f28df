"""Timed cases of the operators that train the router and the projections
around the routed experts:

  balance     per-expert counts, the load-balance loss and the gradient of the
              logits (balance loss and gates together)
  router      gradients of the router projection: of its input, its weights
              and its bias
  checkpoint  an activation stored in 8 bits (E4M3 codes, one power-of-two
              scale per row and 128 inputs) and restored
  swiglu      the gradient of SwiGLU from an 8-bit checkpoint of its inputs
  wgrad       the weight gradient of a projection from an 8-bit checkpoint of
              its input, dense or grouped by expert

`own` selects what run() calls: False the plain form in torch operations, True
the library.  The sizes are those of the layer (H = 4096, I = 2048, 256 experts,
6 active per token; 8, 64, 4604 and 16384 tokens) and generic ones.
"""
import math

import torch

own = False

BLOCK = 128          # inputs that share one scale of an 8-bit checkpoint


# ---- cases ----------------------------------------------------------------------

def listed():
    return [
        # a decode batch: the launches' latency
        {"name": "balance_T8", "op": "balance", "T": 8, "E": 256, "k": 6, "S": 1, "pad": 0, "mask": False},
        # ragged sequences with padding behind the last one and masked tokens
        {"name": "balance_T4604_S13", "op": "balance", "T": 4604, "E": 256, "k": 6, "S": 13, "pad": 37, "mask": True},
        # a training batch of 16 long sequences
        {"name": "balance_T65536_S16", "op": "balance", "T": 65536, "E": 256, "k": 6, "S": 16, "pad": 0,
         "mask": False},
        # a short fine-tuning batch, the router's input kept in bf16
        {"name": "router_T64", "op": "router", "T": 64, "H": 4096, "E": 256, "ckpt": False},
        # a training batch, the input kept in 8 bits
        {"name": "router_ckpt_T16384", "op": "router", "T": 16384, "H": 4096, "E": 256, "ckpt": True},
        # a small activation: latency
        {"name": "checkpoint_T61", "op": "checkpoint", "T": 61, "K": 4096},
        # the hidden states of a training batch
        {"name": "checkpoint_T16384", "op": "checkpoint", "T": 16384, "K": 4096},
        # a short batch, gradients only
        {"name": "swiglu_T64", "op": "swiglu", "T": 64, "I": 2048, "h": False},
        # a training batch, with the activation recomputed for the next weight gradient
        {"name": "swiglu_h_T16384", "op": "swiglu", "T": 16384, "I": 2048, "h": True},
        # few tokens: bound by writing the gradient
        {"name": "wgrad_T40", "op": "wgrad", "T": 40, "N": 4096, "K": 4096, "G": 0, "k": 1},
        # a dense projection over a training batch
        {"name": "wgrad_T16384", "op": "wgrad", "T": 16384, "N": 4096, "K": 4096, "G": 0, "k": 1},
        # gate and up projections of 16 experts, rows gathered through the sort
        {"name": "wgrad_experts_T4604", "op": "wgrad", "T": 4604, "N": 4096, "K": 4096, "G": 16, "k": 6},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "router", "checkpoint", "swiglu", "wgrad"])
    if op == "balance":
        E = _log_int(rng, 4, 1024)
        T = _log_int(rng, 1, min(65536, 65536 * 256 // E))
        pad = rng.choice([0, rng.randint(0, T - 1)])
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 8)), "S": min(_log_int(rng, 1, 48), T),
                "pad": pad, "mask": rng.random() < 0.5}
    if op == "router":
        E = _log_int(rng, 4, 1024)
        T = _log_int(rng, 1, min(16384, 16384 * 256 // E))
        ckpt = rng.random() < 0.5
        step = 128 if ckpt else 32
        return {"op": op, "T": T, "H": step * _log_int(rng, max(1, 256 // step), 4096 // step), "E": E, "ckpt": ckpt}
    if op == "checkpoint":
        return {"op": op, "T": _log_int(rng, 1, 16384), "K": 128 * _log_int(rng, 1, 32)}
    if op == "swiglu":
        return {"op": op, "T": _log_int(rng, 1, 16384), "I": 128 * _log_int(rng, 1, 16), "h": rng.random() < 0.5}
    if rng.random() < 0.5:
        return {"op": op, "T": _log_int(rng, 1, 16384), "N": 8 * _log_int(rng, 8, 512),
                "K": 128 * _log_int(rng, 1, 32), "G": 0, "k": 1}
    G = rng.randint(4, 16)
    return {"op": op, "T": _log_int(rng, 1, 4604), "N": 8 * _log_int(rng, 8, 512), "K": 128 * _log_int(rng, 1, 32),
            "G": G, "k": rng.randint(1, min(G, 6))}


# ---- inputs ---------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activation(g, T, K):
    """Hidden states: rows of different size, a few channels far above the rest,
    every 61st row zero (padding)."""
    x = _normal(g, T, K)
    x *= torch.exp(0.5 * _normal(g, T, 1))
    x[:, ::97] *= 12.0
    x[60::61] = 0.0
    return x.to(torch.bfloat16)


def _store(x):
    """8-bit checkpoint of x [T, K] bf16: codes [T, K] and scales [T, K/128], uint8."""
    T, K = x.shape
    b = x.float().view(T, K // BLOCK, BLOCK)
    m, e = torch.frexp(b.abs().amax(dim=2))
    s = e - 9 + (m > 0.875).to(e.dtype)             # smallest s with max|x| <= 448 * 2^s
    s = torch.where(m > 0, s.clamp(min=-127), torch.full_like(s, -127))
    codes = torch.ldexp(b, -s.unsqueeze(2)).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(T, K), (s + 127).to(torch.uint8)


def _restore(codes, scales):
    """The fp32 values an 8-bit checkpoint stands for."""
    T, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(T, K // BLOCK, BLOCK)
    return torch.ldexp(v, scales.to(torch.int32).unsqueeze(2) - 127).view(T, K)


def _sequence_bounds(case, seed):
    """S ragged sequences over the first T - pad tokens (some may be empty)."""
    g = torch.Generator()
    g.manual_seed(seed)
    n, S = case["T"] - case["pad"], case["S"]
    cuts = torch.sort(torch.randint(0, n + 1, (S - 1,), generator=g)).values.tolist()
    return [0] + cuts + [n]


def _route(g, T, E, k, skew):
    logits = 1.3 * _normal(g, T, E)
    logits -= skew * torch.log1p(torch.arange(E, device="cuda", dtype=torch.float32))
    top, idx = torch.topk(logits, k, dim=1)
    return logits, idx.to(torch.int32), torch.softmax(top, dim=1)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op, T = case["op"], case["T"]
    if op == "balance":
        st["logits"], st["idx"], st["gates"] = _route(g, T, case["E"], case["k"], 0.5)
        st["dgates"] = 1e-2 * _normal(g, T, case["k"])
        st["dloss"] = torch.full((1,), 0.75, device="cuda")
        st["coef"] = 0.01
        st["bounds"] = _sequence_bounds(case, seed)
        st["seq_offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device="cuda")
        st["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9) if case["mask"] else None
    elif op == "router":
        dl = 1e-4 * _normal(g, T, case["E"]) * torch.exp(_normal(g, T, case["E"]))
        dl[50::51] = 0.0                              # rows without a gradient (padding)
        st["dlogits"] = dl
        st["w"] = 0.02 * _normal(g, case["E"], case["H"])
        x = _activation(g, T, case["H"])
        if case["ckpt"]:
            st["codes"], st["scales"] = _store(x)
        else:
            st["x"] = x
    elif op == "checkpoint":
        st["x"] = _activation(g, T, case["K"])
    elif op == "swiglu":
        st["codes"], st["scales"] = _store(_activation(g, T, 2 * case["I"]))
        st["dh"] = (1e-3 * _normal(g, T, case["I"])).to(torch.bfloat16)
    else:
        st["codes"], st["scales"] = _store(_activation(g, T, case["K"]))
        R = T * case["k"]
        st["dy"] = (1e-3 * _normal(g, R, case["N"])).to(torch.bfloat16)
        if case["G"]:
            _, idx, _ = _route(g, T, case["G"], case["k"], 0.7)
            flat = idx.flatten().long()
            st["perm"] = torch.sort(flat, stable=True).indices.to(torch.int32)
            sizes = torch.bincount(flat, minlength=case["G"])
            st["sizes"] = sizes.tolist()
            st["offsets"] = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32)
    if own:
        _own_buffers(st)
    return st


def _own_buffers(st):
    """Outputs and workspaces that a training program keeps between steps."""
    import fp4_routed_mixture_b200 as moe

    case = st["case"]
    op, T = case["op"], case["T"]

    def buf(n):
        return torch.empty(max(1, n), dtype=torch.uint8, device="cuda")

    def f32(*s):
        return torch.empty(s, dtype=torch.float32, device="cuda")

    def bf16(*s):
        return torch.empty(s, dtype=torch.bfloat16, device="cuda")

    def i32(*s):
        return torch.empty(s, dtype=torch.int32, device="cuda")

    if op == "balance":
        E, S = case["E"], case["S"]
        st["ws"] = buf(moe.moe_balance_workspace_bytes(T, E, S))
        st["out"] = (f32(1), i32(S, E), f32(S, E), i32(S + 1))
        st["dlogits"] = f32(T, E)
    elif op == "router":
        H, E = case["H"], case["E"]
        st["ws"] = buf(moe.moe_router_backward_workspace_bytes(T, H, E))
        st["out"] = (bf16(T, H), f32(E, H), f32(E))
    elif op == "checkpoint":
        K = case["K"]
        st["store"] = (torch.empty((T, K), dtype=torch.uint8, device="cuda"),
                       torch.empty((T, K // BLOCK), dtype=torch.uint8, device="cuda"))
        st["out"] = bf16(T, K)
    elif op == "swiglu":
        st["out"] = (bf16(T, 2 * case["I"]), bf16(T, case["I"]) if case["h"] else None)
    else:
        st["ws"] = buf(moe.moe_ckpt_wgrad_workspace_bytes(T * case["k"], case["N"], case["K"], max(1, case["G"])))
        shape = (case["G"], case["N"], case["K"]) if case["G"] else (case["N"], case["K"])
        st["out"] = f32(*shape)


# ---- one pass -------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import fp4_routed_mixture_b200 as moe

    case = st["case"]
    op = case["op"]
    if op == "balance":
        loss, counts, mean_prob, tokens = moe.moe_balance_loss(
            st["logits"], st["idx"], st["coef"], seq_offsets=st["seq_offsets"], token_mask=st["mask"], ws=st["ws"],
            out=st["out"])
        dlogits = moe.moe_route_backward(
            st["logits"], st["idx"], st["gates"], dgates=st["dgates"], dloss=st["dloss"], coef=st["coef"],
            counts=counts, tokens=tokens, seq_offsets=st["seq_offsets"], token_mask=st["mask"], ws=st["ws"],
            out=st["dlogits"])
        return loss, counts, mean_prob, dlogits
    if op == "router":
        src = dict(codes=st["codes"], scales=st["scales"]) if case["ckpt"] else dict(x=st["x"])
        return moe.moe_router_logits_backward(st["dlogits"], st["w"], ws=st["ws"], out=st["out"], **src)
    if op == "checkpoint":
        codes, scales = moe.moe_ckpt_pack(st["x"], out=st["store"])
        return moe.moe_ckpt_unpack(codes, scales, out=st["out"])
    if op == "swiglu":
        dgu, h = moe.moe_ckpt_swiglu_backward(st["codes"], st["scales"], st["dh"], need_h=case["h"], out=st["out"])
        return (dgu, h) if case["h"] else dgu
    if case["G"]:
        return moe.moe_ckpt_wgrad(st["dy"], st["codes"], st["scales"], offsets=st["offsets"], perm=st["perm"],
                                  k=case["k"], dw=st["out"], ws=st["ws"])
    return moe.moe_ckpt_wgrad(st["dy"], st["codes"], st["scales"], dw=st["out"], ws=st["ws"])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "balance":
        return _plain_balance(st)
    if op == "router":
        dl = st["dlogits"]
        x = _restore(st["codes"], st["scales"]) if case["ckpt"] else st["x"].float()
        return (dl @ st["w"]).to(torch.bfloat16), dl.t() @ x, dl.sum(dim=0)
    if op == "checkpoint":
        return _restore(*_store(st["x"])).to(torch.bfloat16)
    if op == "swiglu":
        I = case["I"]
        gu = _restore(st["codes"], st["scales"])
        g, u, dh = gu[:, :I], gu[:, I:], st["dh"].float()
        s = 1.0 / (1.0 + torch.exp(-g))
        a = g * s
        dgu = torch.cat([dh * u * (s * (1.0 + g * (1.0 - s))), dh * a], dim=1).to(torch.bfloat16)
        return (dgu, (a * u).to(torch.bfloat16)) if case["h"] else dgu
    x, dy = _restore(st["codes"], st["scales"]), st["dy"].float()
    if not case["G"]:
        return dy.t() @ x
    x = x[torch.div(st["perm"], case["k"], rounding_mode="floor").long()]
    dw, r = [], 0
    for n in st["sizes"]:
        dw.append(dy[r:r + n].t() @ x[r:r + n])
        r += n
    return torch.stack(dw)


def _plain_balance(st):
    case, idx, bounds = st["case"], st["idx"].long(), st["bounds"]
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    p = torch.softmax(st["logits"], dim=1)
    on = st["seq_offsets"].new_zeros(T).float()
    on[:bounds[-1]] = 1.0
    if st["mask"] is not None:
        on = on * st["mask"].float()
    pm = p * on.unsqueeze(1)
    ones = on.unsqueeze(1).expand(T, k)
    prob, hits, n = [], [], []
    for a, b in zip(bounds[:-1], bounds[1:]):
        prob.append(pm[a:b].sum(dim=0))
        hits.append(pm.new_zeros(E).scatter_add_(0, idx[a:b].flatten(), ones[a:b].flatten()))
        n.append(on[a:b].sum())
    prob, hits, n = torch.stack(prob), torch.stack(hits), torch.stack(n).unsqueeze(1)
    used = (n > 0).float().sum().clamp(min=1.0)
    inv = 1.0 / n.clamp(min=1.0)
    f = hits * (inv * (E / k))
    mean_prob = prob * inv
    loss = st["coef"] * (f * mean_prob).sum() / used
    # gradient of the loss through the probabilities, and of the gates
    seq = torch.bucketize(torch.arange(T, device=p.device), st["seq_offsets"], right=True) - 1
    seq = seq.clamp(max=S - 1)
    ft = f[seq]
    w = st["dloss"] * (st["coef"] / used) * inv[seq, 0] * on
    dl = w.unsqueeze(1) * p * (ft - (p * ft).sum(dim=1, keepdim=True))
    gates, dg = st["gates"], st["dgates"]
    dl.scatter_add_(1, idx, gates * (dg - (gates * dg).sum(dim=1, keepdim=True)))
    return loss.view(1), hits.to(torch.int32), mean_prob, dl


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        return {"bytes": 8 * T * E + 12 * T * k + 8 * S * E + (T if case["mask"] else 0), "flops": 12 * T * E}
    if op == "router":
        H, E = case["H"], case["E"]
        xb = T * H + T * H // BLOCK if case["ckpt"] else 2 * T * H
        return {"bytes": 4 * T * E + 8 * E * H + xb + 2 * T * H + 4 * E, "flops": 4 * T * E * H}
    if op == "checkpoint":
        K = case["K"]
        return {"bytes": 6 * T * K + 2 * T * K // BLOCK, "flops": 4 * T * K}
    if op == "swiglu":
        I = case["I"]
        return {"bytes": (8 + (2 if case["h"] else 0)) * T * I + 2 * T * I // BLOCK, "flops": 20 * T * I}
    N, K, R = case["N"], case["K"], T * case["k"]
    return {"bytes": 2 * R * N + T * K + T * K // BLOCK + 4 * max(1, case["G"]) * N * K + (4 * R if case["G"] else 0),
            "flops": 2 * R * N * K}


# ---- the definitions in 64 bits ---------------------------------------------------

def _value64(codes, scales):
    """E4M3 codes and scale bytes as float64, from the bits."""
    c = codes.to(torch.int64)
    sign = 1.0 - 2.0 * (c >> 7).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8.0 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    return sign * mag * torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "balance":
        return _exact_balance(st)
    if op == "router":
        dl = st["dlogits"].double()
        x = _value64(st["codes"], st["scales"]) if case["ckpt"] else st["x"].double()
        return torch.einsum("te,eh->th", dl, st["w"].double()), torch.einsum("te,th->eh", dl, x), dl.sum(dim=0)
    if op == "checkpoint":
        # the nearest E4M3 multiple of the block's power of two, ties to even
        x = st["x"].double().view(T, -1, BLOCK)
        a = x.abs().amax(dim=2, keepdim=True)
        s = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448.0)).clamp(min=-127.0)
        v = x / torch.exp2(s)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
        return (torch.round(v / step) * step * torch.exp2(s)).view(T, -1)
    if op == "swiglu":
        I = case["I"]
        gu = _value64(st["codes"], st["scales"])
        g, u, dh = gu[:, :I], gu[:, I:], st["dh"].double()
        e = torch.exp(-g.abs())
        s = torch.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
        dgu = torch.cat([dh * u * (s + g * s * (1.0 - s)), dh * g * s], dim=1)
        return (dgu, g * s * u) if case["h"] else dgu
    dy = st["dy"].double()
    if not case["G"]:
        return torch.einsum("tn,tk->nk", dy, _value64(st["codes"], st["scales"]))
    x = _value64(st["codes"], st["scales"])
    dw = torch.zeros((case["G"], case["N"], case["K"]), dtype=torch.float64, device="cuda")
    off = st["offsets"].tolist()
    for e in range(case["G"]):
        rows = torch.arange(off[e], off[e + 1], device="cuda")
        dw[e] = torch.einsum("tn,tk->nk", dy[rows], x[st["perm"][rows].long() // case["k"]])
    return dw


def _exact_balance(st):
    case = st["case"]
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    z = st["logits"].double()
    p = torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True))
    dl = torch.zeros_like(p)
    counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    mean_prob = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    keep = [torch.arange(a, b, device="cuda") for a, b in zip(st["bounds"][:-1], st["bounds"][1:])]
    if st["mask"] is not None:
        keep = [r[st["mask"][r]] for r in keep]
    used = max(1, sum(len(r) > 0 for r in keep))
    for s, r in enumerate(keep):
        if len(r) == 0:
            continue
        hits = torch.bincount(st["idx"][r].flatten().long(), minlength=E)
        counts[s] = hits.to(torch.int32)
        mean_prob[s] = p[r].mean(dim=0)
        f = hits.double() * E / (k * len(r))
        loss += st["coef"] / used * (f @ mean_prob[s])
        q = p[r]
        dl[r] = float(st["dloss"]) * st["coef"] / (used * len(r)) * q * (f - (q @ f).unsqueeze(1))
    gates, dg = st["gates"].double(), st["dgates"].double()
    dl.scatter_add_(1, st["idx"].long(), gates * dg - gates * (gates * dg).sum(dim=1, keepdim=True))
    return loss, counts, mean_prob, dl
