"""Cases of the routing operators and of the quantized linear product, with their plain forms.

Operators: moe_route (scores, group-limited top-K, weights, load statistics), moe_route_backward (gradient of the
logits), moe_slot_weight_grad (gradient of the routing weights from the experts' outputs) and moe_linear (int4 / int8
codes times fp32, bf16 or fp16 activations with bias, activation and residual).

`own` selects what `run` computes: False, elementary torch operations; True, the framework's kernels.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BIG = torch.finfo(torch.float32).max


# ------------------------------------------------------------------------------------------------------ cases

def _route(name, T, E, K, G=1, KG=1, score="sigmoid", group_score="top2", renorm=True, bias=True, dtype="f32",
           scale=2.5, valid=False, stats=False):
    return dict(name=name, op="route", T=T, E=E, K=K, G=G, KG=KG, score=score, group_score=group_score,
                renorm=renorm, bias=bias, dtype=dtype, scale=scale, valid=valid, stats=stats)


def _backward(name, T, E, K, score, renorm, dtype, scale, valid, balance):
    return dict(name=name, op="route_backward", T=T, E=E, K=K, G=1, KG=1, score=score, group_score="max",
                renorm=renorm, bias=False, dtype=dtype, scale=scale, valid=valid, balance=balance)


def _slot(name, T, K, H, drop):
    return dict(name=name, op="slot_weight_grad", T=T, K=K, H=H, drop=drop)


def _linear(name, T, N, K, bits=4, group=0, act="none", dtype="bf16", bias=False, residual=False):
    return dict(name=name, op="linear", T=T, N=N, K=K, bits=bits, group=group, act=act, dtype=dtype, bias=bias,
                residual=residual)


def listed():
    return [
        # one token of the 256-expert layer in 8 groups while it answers: latency only
        _route("route_1", 1, 256, 8, 8, 4),
        # positions checked together by a draft model, a softmax router without groups, bf16 logits
        _route("route_192_softmax", 192, 128, 6, score="softmax", bias=False, dtype="bf16", scale=1.0),
        # a training batch of packed sequences with padding: balance statistics for the bias and the auxiliary loss
        _route("route_32768_stats", 32768, 256, 8, 8, 4, valid=True, stats=True),
        # a small fine-tuning batch of odd length, softmax before the choice, weights as they are, balance term
        _backward("route_grad_381_softmax", 381, 128, 6, "softmax", False, "bf16", 1.0, False, True),
        # the training batch above: sigmoid scores renormalised over the chosen, balance term, padding
        _backward("route_grad_32768", 32768, 256, 8, "sigmoid", True, "f32", 2.5, True, True),
        # tuning the router against a handful of tokens, some slots dropped
        _slot("weight_grad_33", 33, 8, 6144, 0.1),
        # the same over a prefill-sized batch
        _slot("weight_grad_2048", 2048, 8, 6144, 0.0),
        # one token through an output projection with the residual stream: reading the weights is all
        _linear("linear_1_int4", 1, 6144, 6144, residual=True),
        # a decode batch through the gate and up rows of a dense layer, scales by groups
        _linear("linear_32_swiglu_g64", 32, 4096, 6144, group=64, act="swiglu"),
        # a verify batch of odd length through int8 codes, the precision a draft head needs
        _linear("linear_191_int8_gelu", 191, 6144, 2048, bits=8, act="gelu_tanh", dtype="f16", bias=True),
        # prefill through the gate and up rows of a dense layer
        _linear("linear_2048_swiglu", 2048, 12288, 6144, act="swiglu"),
        # calibration in fp32 over a ragged batch, down projection into the residual stream
        _linear("linear_1001_f32", 1001, 6144, 4096, dtype="f32", bias=True, residual=True),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "slot_weight_grad", "linear", "linear"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("route", "route_backward"):
        score = rng.choice(["sigmoid", "softmax"])
        renorm = rng.random() < 0.5
        scale = rng.choice([1.0, 2.5])
        valid = rng.random() < 0.4
        T = _logint(rng, 1, 32768)
        if op == "route_backward":
            E = rng.randint(8, 256)
            return _backward(None, T, E, rng.randint(1, min(E, 12)), score, renorm, dtype, scale, valid,
                             rng.random() < 0.5)
        G = rng.choice([1, 1, 2, 4, 8])
        KG = rng.randint(max(1, G // 2), G)
        E = G * rng.randint(2, 256 // G)
        return _route(None, T, E, rng.randint(1, min(KG * (E // G), 12)), G, KG, score,
                      rng.choice(["top2", "max"]), renorm, rng.random() < 0.6, dtype, scale, valid,
                      rng.random() < 0.4)
    if op == "slot_weight_grad":
        return _slot(None, _logint(rng, 1, 2048), rng.randint(1, 8), 64 * rng.randint(1, 96),
                     rng.choice([0.0, 0.1, 0.5]))
    bits, group = rng.choice([(4, 0), (4, 0), (8, 0), (4, 32), (4, 64), (4, 128)])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
    T, N, K = _logint(rng, 1, 2048), 128 * rng.randint(1, 48), max(group, 32) * rng.randint(1, 6144 // max(group, 32))
    return _linear(None, T, N, K, bits, group, act, dtype, rng.random() < 0.5, rng.random() < 0.5)


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "route":
        E, z = case["E"], SIZE[case["dtype"]]
        b = T * E * z + 8 * T * K + (4 * E if case["bias"] else 0) + (T if case["valid"] else 0)
        return {"bytes": b + (8 * E if case["stats"] else 0), "flops": 4 * T * E}
    if case["op"] == "route_backward":
        E, z = case["E"], SIZE[case["dtype"]]
        dense = case["balance"] or (case["score"] == "softmax" and not case["renorm"])
        b = T * E * z + (T * E if dense else T * K) * z + 8 * T * K + (T if case["valid"] else 0)
        return {"bytes": b + (4 * E if case["balance"] else 0), "flops": (6 * T * E if dense else 6 * T * K)}
    if case["op"] == "slot_weight_grad":
        H = case["H"]
        return {"bytes": 4 * (T * K * H + T * H + 2 * T * K), "flops": 2 * T * K * H}
    N, s = case["N"], SIZE[case["dtype"]]
    out = N // 2 if case["act"] == "swiglu" else N
    b = N * K * case["bits"] // 8 + 4 * N * (K // case["group"] if case["group"] else 1) + T * K * s + T * out * s
    b += (4 * N if case["bias"] else 0) + (T * out * s if case["residual"] else 0)
    return {"bytes": b, "flops": 2 * T * N * K}


# ----------------------------------------------------------------------------------------------------- inputs

def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + tag)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _valid(case, seed):
    """Padded batch: runs of real tokens, each followed by padding."""
    if not case["valid"]:
        return None
    T = case["T"]
    run = torch.randint(3, 60, (T // 16 + 2,), generator=_gen(seed, 7), device="cuda")
    edge = torch.cumsum(run, 0)
    at = torch.searchsorted(edge, torch.arange(T, device="cuda"), right=True)
    return (at % 4 != 3).to(torch.uint8)


def _logits(case, seed):
    """Router logits: a common preference per expert and the token's own part."""
    T, E = case["T"], case["E"]
    z = 1.5 * _randn((T, E), _gen(seed, 1)) + 0.7 * _randn((1, E), _gen(seed, 2))
    return z.to(DT[case["dtype"]])


def _choose(case, seed):
    """Ids of the K largest logits (a routing that the backward pass is given)."""
    ids = torch.topk(_logits(case, seed).float() + 1e-3 * _randn((case["T"], case["E"]), _gen(seed, 3)),
                     case["K"], dim=1).indices.to(torch.int32)
    v = _valid(case, seed)
    return ids if v is None else torch.where(v[:, None] != 0, ids, -1).contiguous()


def _codes(case, seed):
    """Weights quantized by rows or groups: signed codes [N][K] (int8) and scales [N][groups]."""
    N, K, G = case["N"], case["K"], case["group"] or case["K"]
    top = 7.0 if case["bits"] == 4 else 127.0
    w = (0.02 * _randn((N, K), _gen(seed, 11))).view(N, K // G, G)
    s = w.abs().amax(dim=2) / top
    q = torch.round(w / s[:, :, None]).clamp(-top, top).to(torch.int8)
    return q.view(N, K), s.contiguous()


def _pack4(q):
    """Two codes a byte, element 2j in the low half of byte j."""
    u = (q.to(torch.int16) & 15).to(torch.uint8)
    return (u[:, 0::2] | (u[:, 1::2] << 4)).contiguous()


def _linear_inputs(case, seed):
    T, N, K, dt = case["T"], case["N"], case["K"], DT[case["dtype"]]
    x = _randn((T, K), _gen(seed, 12))
    x[:, :: max(1, K // 7)] *= 20.0  # a few channels far above the rest, as hidden states have
    out = N // 2 if case["act"] == "swiglu" else N
    bias = 0.1 * _randn((N,), _gen(seed, 13)) if case["bias"] else None
    res = _randn((T, out), _gen(seed, 14)).to(dt) if case["residual"] else None
    return x.to(dt), bias, res


def prepare(case, seed):
    st = dict(case)
    T, K = case["T"], case["K"]
    if case["op"] == "route":
        E = case["E"]
        st["z"] = _logits(case, seed)
        st["b"] = 0.1 * (torch.rand((E,), generator=_gen(seed, 4), device="cuda") - 0.5) if case["bias"] else None
        st["v"] = _valid(case, seed)
        if own:
            import int4_quantized_expert_amd as moe
            st["cfg"] = _route_config(case)
            st["ids"] = torch.empty((T, K), dtype=torch.int32, device="cuda")
            st["w"] = torch.empty((T, K), dtype=torch.float32, device="cuda")
            if case["stats"]:
                st["load"] = torch.empty((E,), dtype=torch.int32, device="cuda")
                st["imp"] = torch.empty((E,), dtype=torch.float32, device="cuda")
                st["ws"] = torch.empty((moe.moe_route_workspace_bytes(st["cfg"], T),), dtype=torch.uint8,
                                       device="cuda")
    elif case["op"] == "route_backward":
        E = case["E"]
        st["z"] = _logits(case, seed)
        st["v"] = _valid(case, seed)
        st["ids"] = _choose(case, seed)
        st["dw"] = _randn((T, K), _gen(seed, 5))
        st["dimp"] = _randn((E,), _gen(seed, 6)) if case["balance"] else None
        if own:
            st["cfg"] = _route_config(case)
            st["dz"] = torch.empty((T, E), dtype=DT[case["dtype"]], device="cuda")
    elif case["op"] == "slot_weight_grad":
        st["eout"], st["dy"], st["ids"] = _slot_inputs(case, seed)
        if own:
            st["dw"] = torch.empty((T, K), dtype=torch.float32, device="cuda")
    else:
        q, s = _codes(case, seed)
        codes = _pack4(q) if case["bits"] == 4 else q.contiguous()
        st["x"], st["b"], st["r"] = _linear_inputs(case, seed)
        if own:
            import int4_quantized_expert_amd as moe
            N, G = case["N"], case["group"]
            tiled = torch.empty((codes.numel(),), dtype=torch.uint8, device="cuda")
            (moe.moe_tile_int4 if case["bits"] == 4 else moe.moe_tile_int8)(codes, tiled)
            scales = s.view(-1)
            if G:
                scales = torch.empty_like(scales)
                moe.moe_tile_group_scales(s, scales)
            st["codes"], st["scales"] = tiled, scales
            st["cfg"] = moe.LinearConfig(rows=N, cols=K, weight_bits=case["bits"], group_size=G,
                                         act=getattr(moe, "MOE_ACT_" + case["act"].upper()))
            st["y"] = torch.empty((T, N // 2 if case["act"] == "swiglu" else N), dtype=DT[case["dtype"]],
                                  device="cuda")
            st["ws"] = torch.empty((moe.moe_linear_workspace_bytes(st["cfg"], T),), dtype=torch.uint8, device="cuda")
        else:
            st["codes"], st["scales"] = codes, s
    return st


def _slot_inputs(case, seed):
    T, K, H = case["T"], case["K"], case["H"]
    eout = 0.1 * _randn((T * K, H), _gen(seed, 21))
    dy = _randn((T, H), _gen(seed, 22)) / math.sqrt(H)
    ids = torch.randint(0, 256, (T, K), generator=_gen(seed, 23), device="cuda", dtype=torch.int32)
    if case["drop"] > 0:  # a dropped slot's output row is never written: whatever the buffer held
        gone = torch.rand((T, K), generator=_gen(seed, 24), device="cuda") < case["drop"]
        ids = torch.where(gone, -1, ids).contiguous()
        eout[gone.view(-1)] = float("nan")
    return eout, dy, ids


def _route_config(case):
    import int4_quantized_expert_amd as moe
    return moe.RouteConfig(n_experts=case["E"], n_group=case["G"], topk_group=case["KG"], top_k=case["K"],
                           score=moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                           group_score=moe.MOE_GROUP_TOP2 if case["group_score"] == "top2" else moe.MOE_GROUP_MAX,
                           renorm=case["renorm"], scale=case["scale"])


# -------------------------------------------------------------------------------------------------------- run

def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "route_backward": _plain_backward, "slot_weight_grad": _plain_slot,
            "linear": _plain_linear}[state["op"]](state)


def _run_own(st):
    import int4_quantized_expert_amd as moe
    if st["op"] == "route":
        if st["stats"]:
            moe.moe_route(st["cfg"], st["z"], st["ids"], st["w"], bias=st["b"], valid=st["v"], load=st["load"],
                          importance=st["imp"], ws=st["ws"])
            return st["ids"], st["w"], st["load"], st["imp"]
        moe.moe_route(st["cfg"], st["z"], st["ids"], st["w"], bias=st["b"], valid=st["v"])
        return st["ids"], st["w"]
    if st["op"] == "route_backward":
        moe.moe_route_backward(st["cfg"], st["z"], st["ids"], st["dz"], d_w=st["dw"], d_importance=st["dimp"],
                               valid=st["v"])
        return st["dz"]
    if st["op"] == "slot_weight_grad":
        moe.moe_slot_weight_grad(st["eout"], st["ids"], st["dy"], st["dw"])
        return st["dw"]
    moe.moe_linear(st["cfg"], st["codes"], st["scales"], st["x"], st["y"], st["ws"], bias=st["b"],
                   residual=st["r"])
    return st["y"]


def _live(z):
    """fp32 logits and which of them take part: not masked by NaN, -inf or the lowest value of the type."""
    live = z > torch.finfo(z.dtype).min
    return z.float().clamp(max=BIG), live


def _scores(zf, live, kind, wide):
    """Scores (0 where masked); wide: in 64 bits, for values that are compared with each other."""
    z = zf.double() if wide else zf
    if kind == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
        return torch.where(live, s, torch.zeros_like(s))
    z = torch.where(live, z, torch.full_like(z, -math.inf))
    m = z.amax(dim=1, keepdim=True)
    e = torch.where(live, torch.exp(z - torch.where(m > -math.inf, m, torch.zeros_like(m))), torch.zeros_like(z))
    t = e.sum(dim=1, keepdim=True)
    return e / torch.where(t > 0, t, torch.ones_like(t))


def _relative(z, on, kind):
    """Scores relative to the largest of the entries that are on (0 elsewhere), so that no sum underflows."""
    low = torch.full_like(z, -math.inf)
    m = torch.where(on, z, low).amax(dim=1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    if kind == "sigmoid":
        m = m.clamp(max=0.0)
        t = torch.where(z < 0, torch.exp(torch.minimum(z, m) - m) / (1.0 + torch.exp(z.clamp(max=0.0))),
                        1.0 / (1.0 + torch.exp(-z)))
    else:
        t = torch.exp(z - m)
    return torch.where(on, t, torch.zeros_like(t))


def _share(t):
    s = t.sum(dim=1, keepdim=True)
    return t / torch.where(s > 0, s, torch.ones_like(s))


def _plain_route(st):
    T, E, K, G, KG = st["T"], st["E"], st["K"], st["G"], st["KG"]
    zf, live = _live(st["z"])
    if st["v"] is not None:
        live = live & (st["v"] != 0)[:, None]
    low = torch.full_like(zf, -math.inf)
    s = None
    if st["bias"] or (G > 1 and st["group_score"] == "top2"):
        s = _scores(zf, live, st["score"], True).float()
    c = s + st["b"][None, :] if st["bias"] else zf
    c = torch.where(live, c, low)
    if G > 1:
        g = c if st["bias"] or st["group_score"] == "max" else torch.where(live, s, low)
        g = g.view(T, G, E // G)
        if st["group_score"] == "max":
            g = g.amax(dim=2)
        else:
            top = g.topk(2, dim=2).values
            g = torch.where(top[:, :, 1] > -math.inf, top[:, :, 0] + top[:, :, 1], top[:, :, 0])
        order = torch.sort(g, dim=1, descending=True, stable=True).indices[:, :KG]
        keep = torch.zeros((T, G), dtype=torch.bool, device=zf.device).scatter_(1, order, True)
        c = torch.where(keep.repeat_interleave(E // G, dim=1), c, low)
    val, idx = torch.sort(c, dim=1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    on = val > -math.inf
    zk = torch.gather(zf, 1, idx)
    if st["renorm"]:
        w = _share(_relative(zk, on, st["score"]))
    else:
        w = torch.gather(_scores(zf, live, st["score"], False), 1, idx)
    w = torch.where(on, w * st["scale"], torch.zeros_like(w))
    ids = torch.where(on, idx, -1).to(torch.int32)
    if not st["stats"]:
        return ids, w
    load = torch.zeros(E + 1, dtype=torch.int32, device=zf.device)
    load.scatter_add_(0, torch.where(on, idx, E).view(-1), torch.ones(T * K, dtype=torch.int32, device=zf.device))
    imp = _share(_relative(zf, live, st["score"])).double().sum(dim=0).float()
    return ids, w, load[:E].contiguous(), imp


def _plain_backward(st):
    zf, live = _live(st["z"])
    if st["v"] is not None:
        live = live & (st["v"] != 0)[:, None]
    ids = st["ids"].long()
    at = ids.clamp(min=0)
    on = (ids >= 0) & torch.gather(live, 1, at)
    u = torch.where(on, st["dw"] * st["scale"], torch.zeros_like(st["dw"]))
    zk = torch.gather(zf, 1, at)
    miss = 1.0 / (1.0 + torch.exp(zf))  # 1 - sigmoid(z)
    if st["renorm"]:
        r = _share(_relative(zk, on, st["score"]))
        dk = r * (u - (r * u).sum(dim=1, keepdim=True))
        if st["score"] == "sigmoid":
            dk = dk * torch.gather(miss, 1, at)
        dz = torch.zeros_like(zf).scatter_add_(1, at, torch.where(on, dk, torch.zeros_like(dk)))
    elif st["score"] == "sigmoid":
        dk = u * torch.gather(_scores(zf, live, "sigmoid", False) * miss, 1, at)
        dz = torch.zeros_like(zf).scatter_add_(1, at, torch.where(on, dk, torch.zeros_like(dk)))
    else:
        p = _scores(zf, live, "softmax", False)
        full = torch.zeros_like(zf).scatter_add_(1, at, u)
        dz = p * (full - (p * full).sum(dim=1, keepdim=True))
    if st["dimp"] is not None:
        p = _share(_relative(zf, live, st["score"]))
        d = p * (st["dimp"][None, :] - (p * st["dimp"][None, :]).sum(dim=1, keepdim=True))
        dz = dz + (d * miss if st["score"] == "sigmoid" else d)
    return torch.where(live, dz, torch.zeros_like(dz)).to(st["z"].dtype)


def _plain_slot(st):
    T, K, H = st["T"], st["K"], st["H"]
    d = (st["eout"].view(T, K, H) * st["dy"][:, None, :]).sum(dim=2)
    return torch.where(st["ids"] >= 0, d, torch.zeros_like(d))


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(st):
    N, K, G = st["N"], st["K"], st["group"] or st["K"]
    q = st["codes"]
    if st["bits"] == 4:
        lo, hi = q & 15, q >> 4
        q = torch.stack([lo, hi], dim=2).view(N, K).to(torch.int8)
        q = torch.where(q > 7, q - 16, q)
    w = (q.float().view(N, K // G, G) * st["scales"][:, :, None]).view(N, K)
    v = st["x"].float() @ w.t()
    if st["b"] is not None:
        v = v + st["b"][None, :]
    v = _act(v[:, : N // 2], "silu") * v[:, N // 2:] if st["act"] == "swiglu" else _act(v, st["act"])
    if st["r"] is not None:
        v = v + st["r"].float()
    return v.to(st["x"].dtype)


# ------------------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """The operators' definitions in 64 bits, written without the plain forms: the choice by rounds of a largest
    entry, gradients by differentiating the weights."""
    if case["op"] == "route":
        return _exact_route(case, seed)
    if case["op"] == "route_backward":
        return _exact_backward(case, seed)
    if case["op"] == "slot_weight_grad":
        eout, dy, ids = _slot_inputs(case, seed)
        on = ids >= 0
        rows = torch.nan_to_num(eout).double().view(case["T"], case["K"], case["H"])
        return (torch.bmm(rows, dy.double()[:, :, None]).squeeze(2)) * on
    q, s = _codes(case, seed)
    x, bias, res = _linear_inputs(case, seed)
    N, K, G = case["N"], case["K"], case["group"] or case["K"]
    v = torch.zeros((case["T"], N), dtype=torch.float64, device="cuda")
    step = max(G, 2048 // G * G)
    for k0 in range(0, K, step):
        k1 = min(K, k0 + step)
        wk = q[:, k0:k1].double() * s[:, k0 // G:(k1 + G - 1) // G].double().repeat_interleave(min(G, k1 - k0), dim=1)
        v += torch.mm(x[:, k0:k1].double(), wk.t().contiguous())
    if bias is not None:
        v += bias.double()
    act = case["act"]
    if act == "swiglu":
        g, u = v.chunk(2, dim=1)
        v = g * u * torch.special.expit(g)
    elif act == "relu":
        v = v.clamp(min=0)
    elif act == "silu":
        v = v * torch.special.expit(v)
    elif act == "gelu":
        v = v * torch.special.ndtr(v)
    elif act == "gelu_tanh":
        v = v * torch.special.expit(2 * math.sqrt(2 / math.pi) * v * (1 + 0.044715 * v * v))
    return v if res is None else v + res.double()


def _score64(z, kind):
    """log of the scores of all experts (none of the listed inputs masks an expert)."""
    return -torch.nn.functional.softplus(-z) if kind == "sigmoid" else z - torch.logsumexp(z, dim=1, keepdim=True)


def _exact_route(case, seed):
    T, E, K, G, KG = case["T"], case["E"], case["K"], case["G"], case["KG"]
    st_z = _logits(case, seed)
    v = _valid(case, seed)
    z = st_z.double()
    ls = _score64(z, case["score"])
    s32 = torch.exp(ls).float()
    if case["bias"]:
        b = 0.1 * (torch.rand((E,), generator=_gen(seed, 4), device="cuda") - 0.5)
        c = s32 + b
    else:
        c = st_z.float()
    dead = torch.finfo(torch.float32).min
    if G > 1:
        by = c if case["bias"] or case["group_score"] == "max" else s32
        by = by.reshape(T, G, E // G).clone()
        first, at = by.max(dim=2)
        if case["group_score"] == "top2":
            by.scatter_(2, at[:, :, None], -math.inf)
            first = first + by.max(dim=2).values
        rank = (first[:, None, :] > first[:, :, None]).sum(dim=2)
        rank += ((first[:, None, :] == first[:, :, None])
                 & (torch.arange(G, device="cuda")[None, None, :] < torch.arange(G, device="cuda")[None, :, None])
                 ).sum(dim=2)
        c = torch.where((rank < KG)[:, :, None], c.reshape(T, G, E // G), dead).reshape(T, E)
    c = c.clone()
    number = torch.arange(E, device="cuda")[None, :]
    picks = []
    for _ in range(K):
        top = c.amax(dim=1, keepdim=True)
        i = torch.where(c == top, number, E).amin(dim=1)
        picks.append(i)
        c.scatter_(1, i[:, None], dead)
    ids = torch.stack(picks, dim=1)
    lk = torch.gather(ls, 1, ids)
    w = (torch.softmax(lk, dim=1) if case["renorm"] else torch.exp(lk)) * case["scale"]
    on = torch.ones((T, 1), dtype=torch.bool, device="cuda") if v is None else (v != 0)[:, None]
    out = [torch.where(on, ids, -1).to(torch.int32), w * on]
    if case["stats"]:
        load = torch.bincount(ids[on.expand(T, K)], minlength=E).to(torch.int32)
        out += [load, (torch.softmax(ls, dim=1) * on).sum(dim=0)]
    return tuple(out)


def _exact_backward(case, seed):
    T, K, E = case["T"], case["K"], case["E"]
    z = _logits(case, seed).double().requires_grad_(True)
    v, ids = _valid(case, seed), _choose(case, seed).long()
    dw = _randn((T, K), _gen(seed, 5)).double()
    on = torch.ones((T, 1), dtype=torch.float64, device="cuda") if v is None else (v != 0)[:, None].double()
    ls = _score64(z, case["score"])
    lk = torch.gather(ls, 1, ids.clamp(min=0))
    w = torch.softmax(lk, dim=1) if case["renorm"] else torch.exp(lk)
    loss = (w * dw * on).sum() * case["scale"]
    if case["balance"]:
        dimp = _randn((E,), _gen(seed, 6)).double()
        loss = loss + ((torch.softmax(ls, dim=1) * on).sum(dim=0) * dimp).sum()
    return torch.autograd.grad(loss, z)[0]
