"""Cases of the adapted linear product, of its gradients and of gradient clipping, with their plain forms.

Operators: moe_linear_adapted (int4 / int8 codes times activations with low-rank adapters by token, bias, activation and
residual), moe_linear_backward (gradients of its activations and adapters; without adapters the backward pass of a frozen
or gated projection) and moe_grad_clip (norm over many gradients, and the gradients scaled by it).

`own` selects what `run` computes: False, elementary torch operations; True, the framework's kernels.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------------------------ cases

def _adapted(name, T, N, K, R, n, mix, bits=4, group=0, act="none", dtype="bf16", bias=False, residual=False, pre=False):
    return dict(name=name, op="adapted", T=T, N=N, K=K, R=R, n=n, mix=mix, bits=bits, group=group, act=act, dtype=dtype,
                bias=bias, residual=residual, pre=pre)


def _backward(name, T, N, K, R, n, mix, bits=4, group=0, act="none", dtype="bf16"):
    return dict(name=name, op="backward", T=T, N=N, K=K, R=R, n=n, mix=mix, bits=bits, group=group, act=act, dtype=dtype)


def _clip(name, count, total, dtype, clipped):
    return dict(name=name, op="clip", count=count, total=total, dtype=dtype, clipped=clipped)


def listed():
    return [
        # one token of one request with its adapter through an output projection: latency
        _adapted("adapted_1", 1, 6144, 6144, 16, 32, "token", residual=True),
        # a decode batch, each request with an adapter of its own or none, gate and up rows with group scales
        _adapted("adapted_32_swiglu_g64", 32, 4096, 6144, 16, 64, "token", group=64, act="swiglu"),
        # positions of a few requests checked together, int8 codes
        _adapted("adapted_191_int8_gelu", 191, 6144, 2048, 8, 4, "runs", bits=8, act="gelu_tanh", dtype="f16", bias=True),
        # prefill of several requests through the gate and up rows of a dense layer
        _adapted("adapted_2048_swiglu", 2048, 12288, 6144, 32, 8, "runs", act="swiglu"),
        # a training step's forward in fp32 over a ragged batch, pre-activations kept for the gradients
        _adapted("adapted_1001_f32", 1001, 6144, 4096, 64, 2, "runs", act="silu", dtype="f32", bias=True, residual=True,
                 pre=True),
        # tuning on a handful of tokens: the weights' codes are nearly all there is to read
        _backward("backward_33", 33, 6144, 6144, 16, 3, "token"),
        # calibration through fp32 activations and group scales, one adapter
        _backward("backward_381_f32_g128", 381, 6144, 2048, 8, 1, "all", group=128, act="silu", dtype="f32"),
        # a fine-tuning batch of several adapters through gate and up rows, some tokens without one
        _backward("backward_2000_adapters", 2000, 4096, 6144, 32, 4, "runs", act="swiglu"),
        # the frozen gated projection of a dense layer: only the activations' gradient goes on
        _backward("backward_2048_swiglu", 2048, 12288, 6144, 0, 0, "none", act="swiglu"),
        # the gradients of one routed layer's router and adapters
        _clip("clip_12", 12, 1 << 20, "f32", True),
        # the adapters' gradients of a whole model, ragged sizes
        _clip("clip_640", 640, 100_000_007, "f32", True),
        # gradients in 16 bits, below the limit
        _clip("clip_180_bf16", 180, 300_000_011, "bf16", False),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adapted", "adapted", "backward", "backward", "clip"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "clip":
        count = _logint(rng, 1, 640)
        return _clip(None, count, _logint(rng, 64 * count, 100_000_000), dtype, rng.random() < 0.6)
    bits, group = rng.choice([(4, 0), (4, 0), (8, 0), (4, 32), (4, 64), (4, 128)])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
    T, N, K = _logint(rng, 1, 2048), 128 * rng.randint(1, 48), max(group, 32) * rng.randint(1, 6144 // max(group, 32))
    R = 8 * _logint(rng, 1, 16)
    n = _logint(rng, 1, max(1, min(64, 1024 // R)))
    mix = rng.choice(["token", "runs", "all"])
    if op == "adapted":
        return _adapted(None, T, N, K, R, n, mix, bits, group, act, dtype, rng.random() < 0.5, rng.random() < 0.5,
                        rng.random() < 0.3)
    if rng.random() < 0.3:
        R, n, mix = 0, 0, "none"
    return _backward(None, T, N, K, R, n, mix, bits, group, act, dtype)


def work(case):
    if case["op"] == "clip":
        return {"bytes": 2 * case["total"] * SIZE[case["dtype"]], "flops": 3 * case["total"]}
    T, N, K, R, s = case["T"], case["N"], case["K"], case["R"], SIZE[case["dtype"]]
    out = N // 2 if case["act"] == "swiglu" else N
    used = min(case["n"], T)
    b = N * K * case["bits"] // 8 + 4 * N * (K // case["group"] if case["group"] else 1)
    b += used * R * (N + K) * s + 4 * T * (case["n"] > 0)
    if case["op"] == "adapted":
        b += T * (K + out) * s + (4 * N if case["bias"] else 0)
        b += (T * out * s if case["residual"] else 0) + (T * N * s if case["pre"] else 0)
        return {"bytes": b, "flops": 2 * T * N * K + 2 * T * R * (N + K)}
    b += T * (K + out) * s + (T * N * s if case["act"] != "none" else 0)
    b += (T * K * s if R else 0) + s * case["n"] * R * (N + K)
    return {"bytes": b, "flops": 2 * T * N * K + 2 * T * R * (2 * N + 3 * K)}


# ----------------------------------------------------------------------------------------------------- inputs

def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + tag)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


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


def _hidden(case, seed):
    T, K = case["T"], case["K"]
    x = _randn((T, K), _gen(seed, 12))
    x[:, :: max(1, K // 7)] *= 20.0  # a few channels far above the rest, as hidden states have
    return x.to(DT[case["dtype"]])


def _ids(case, seed):
    """Adapter of each token: its own, one by runs of tokens (about an eighth of them without one), or one for all."""
    T, n = case["T"], case["n"]
    if case["mix"] == "all":
        return torch.randint(0, n, (1,), generator=_gen(seed, 31), device="cuda").to(torch.int32).expand(T).contiguous()
    if case["mix"] == "token":
        at = torch.arange(T, device="cuda")
    else:
        run = torch.randint(1, max(2, T // 4), (T + 1,), generator=_gen(seed, 32), device="cuda")
        at = torch.searchsorted(torch.cumsum(run, 0), torch.arange(T, device="cuda"), right=True)
    pick = torch.randint(0, 8 * n, (T + 1,), generator=_gen(seed, 33), device="cuda")
    pick = torch.where(pick < 7 * n, pick % n, -1) if T > 1 else pick % n
    return pick[at].to(torch.int32).contiguous()


def _adapters(case, seed):
    """A [n][R][K], B [n][N][R] and the adapters' scales."""
    n, R, N, K, dt = case["n"], case["R"], case["N"], case["K"], DT[case["dtype"]]
    a = _randn((n, R, K), _gen(seed, 34)) / math.sqrt(K)
    b = 0.05 * _randn((n, N, R), _gen(seed, 35))
    s = 0.5 + 1.5 * torch.rand((n,), generator=_gen(seed, 36), device="cuda")
    return a.to(dt), b.to(dt), s


def _forward_extras(case, seed):
    T, N, dt = case["T"], case["N"], DT[case["dtype"]]
    out = N // 2 if case["act"] == "swiglu" else N
    bias = 0.1 * _randn((N,), _gen(seed, 13)) if case["bias"] else None
    return bias, (_randn((T, out), _gen(seed, 14)).to(dt) if case["residual"] else None)


def _gradient_inputs(case, seed):
    """Gradient of the output, and the pre-activations that the forward pass kept."""
    T, N, dt = case["T"], case["N"], DT[case["dtype"]]
    out = N // 2 if case["act"] == "swiglu" else N
    dy = (_randn((T, out), _gen(seed, 15)) / math.sqrt(out)).to(dt)
    return dy, (1.5 * _randn((T, N), _gen(seed, 16))).to(dt) if case["act"] != "none" else None


def _sizes(case, seed):
    """Elements of each gradient: ragged, some of them tiny, all of them together `total`."""
    count, total = case["count"], case["total"]
    g = torch.Generator()
    g.manual_seed(7919 * seed + 41)
    share = torch.exp(3.0 * torch.randn((count,), generator=g, dtype=torch.float64))
    size = (share / share.sum() * (total - count)).long() + 1
    size[size.argmax()] += total - int(size.sum())
    return size.tolist()


def _gradients(case, seed):
    """All gradients, one behind the other: [total] values of one type (each tensor is a part of it)."""
    g = _gen(seed, 42)
    flat = torch.empty((case["total"],), dtype=DT[case["dtype"]], device="cuda")
    step = 1 << 26
    for at in range(0, case["total"], step):
        part = flat[at:at + step]
        part.copy_(1e-3 * torch.randn((part.numel(),), generator=g, device="cuda", dtype=torch.float32))
    norm = 1e-3 * math.sqrt(case["total"])
    return flat, (0.25 if case["clipped"] else 4.0) * norm


def prepare(case, seed):
    st = dict(case)
    if case["op"] == "clip":
        flat, st["max_norm"] = _gradients(case, seed)
        sizes = _sizes(case, seed)
        st["grads"] = list(torch.split(flat, sizes))
        st["out"] = torch.empty_like(flat)
        if own:
            import int4_quantized_expert_amd as moe
            st["norm"] = torch.empty((1,), dtype=torch.float32, device="cuda")
            st["table"] = moe.GradTable(st["grads"], list(torch.split(st["out"], sizes)))
        return st
    T, N, K, dt = case["T"], case["N"], case["K"], DT[case["dtype"]]
    out = N // 2 if case["act"] == "swiglu" else N
    q, s = _codes(case, seed)
    codes = _pack4(q) if case["bits"] == 4 else q.contiguous()
    st["x"] = _hidden(case, seed)
    if case["n"]:
        st["ids"] = _ids(case, seed)
        st["a"], st["b"], st["s"] = _adapters(case, seed)
    if case["op"] == "adapted":
        st["bias"], st["res"] = _forward_extras(case, seed)
    else:
        st["dy"], st["z"] = _gradient_inputs(case, seed)
    if not own:
        st["codes"], st["scales"] = codes, s
        return st
    import int4_quantized_expert_amd as moe
    tiled = torch.empty((codes.numel(),), dtype=torch.uint8, device="cuda")
    (moe.moe_tile_int4 if case["bits"] == 4 else moe.moe_tile_int8)(codes, tiled)
    scales = s.view(-1)
    if case["group"]:
        scales = torch.empty_like(scales)
        moe.moe_tile_group_scales(s, scales)
    st["codes"], st["scales"] = tiled, scales
    st["cfg"] = moe.LinearConfig(rows=N, cols=K, weight_bits=case["bits"], group_size=case["group"],
                                 act=getattr(moe, "MOE_ACT_" + case["act"].upper()))
    st["ad"] = moe.Adapters(st["a"], st["b"], st["s"]) if case["n"] else None
    if case["op"] == "adapted":
        st["y"] = torch.empty((T, out), dtype=dt, device="cuda")
        st["z"] = torch.empty((T, N), dtype=dt, device="cuda") if case["pre"] else None
        size = moe.moe_linear_adapted_workspace_bytes(st["cfg"], st["ad"], T)
    else:
        st["dx"] = torch.empty((T, K), dtype=dt, device="cuda")
        st["da"] = torch.empty_like(st["a"]) if case["n"] else None
        st["db"] = torch.empty_like(st["b"]) if case["n"] else None
        size = moe.moe_linear_backward_workspace_bytes(st["cfg"], st["ad"], T)
    st["ws"] = torch.empty((size,), dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------------------------------------------------- run

def run(state):
    if own:
        return _run_own(state)
    return {"adapted": _plain_adapted, "backward": _plain_backward, "clip": _plain_clip}[state["op"]](state)


def _run_own(st):
    import int4_quantized_expert_amd as moe
    if st["op"] == "clip":
        moe.moe_grad_clip(st["table"], st["max_norm"], st["norm"])
        return st["norm"], st["out"]
    if st["op"] == "adapted":
        moe.moe_linear_adapted(st["cfg"], st["codes"], st["scales"], st["ad"], st["ids"], st["x"], st["y"], st["ws"],
                               bias=st["bias"], residual=st["res"], pre=st["z"])
        return (st["y"], st["z"]) if st["pre"] else st["y"]
    if st["n"]:
        moe.moe_linear_backward(st["cfg"], st["codes"], st["scales"], st["dy"], st["dx"], st["ws"], pre=st["z"],
                                adapters=st["ad"], ids=st["ids"], x=st["x"], d_a=st["da"], d_b=st["db"])
        return st["dx"], st["da"], st["db"]
    moe.moe_linear_backward(st["cfg"], st["codes"], st["scales"], st["dy"], st["dx"], st["ws"], pre=st["z"])
    return st["dx"]


def _plain_weights(st):
    N, K, G = st["N"], st["K"], st["group"] or st["K"]
    q = st["codes"]
    if st["bits"] == 4:
        lo, hi = q & 15, q >> 4
        q = torch.stack([lo, hi], dim=2).view(N, K).to(torch.int8)
        q = torch.where(q > 7, q - 16, q)
    return (q.float().view(N, K // G, G) * st["scales"][:, :, None]).view(N, K)


def _chosen(st):
    """[T][n * R]: the scale of the token's adapter in the adapter's columns, 0 in the others'."""
    one = st["ids"].long()[:, None] == torch.arange(st["n"], device="cuda")[None, :]
    return torch.where(one, st["s"][None, :], torch.zeros_like(st["s"])[None, :]).repeat_interleave(st["R"], dim=1)


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


def _slope(v, act):
    """Derivative of the activation."""
    if act == "relu":
        return torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 + v * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(v / math.sqrt(2.0))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * v * v)


def _plain_adapted(st):
    N, K, n, R = st["N"], st["K"], st["n"], st["R"]
    x = st["x"].float()
    h = (x @ st["a"].float().view(n * R, K).t()) * _chosen(st)
    v = x @ _plain_weights(st).t() + h @ st["b"].float().transpose(1, 2).reshape(n * R, N)
    if st["bias"] is not None:
        v = v + st["bias"][None, :]
    y = _act(v[:, : N // 2], "silu") * v[:, N // 2:] if st["act"] == "swiglu" else _act(v, st["act"])
    if st["res"] is not None:
        y = y + st["res"].float()
    y = y.to(st["x"].dtype)
    return (y, v.to(st["x"].dtype)) if st["pre"] else y


def _plain_backward(st):
    N, K, n, R = st["N"], st["K"], st["n"], st["R"]
    d = st["dy"].float()
    if st["act"] == "swiglu":
        g, u = st["z"].float().chunk(2, dim=1)
        d = torch.cat([d * u * _slope(g, "silu"), d * _act(g, "silu")], dim=1)
    elif st["act"] != "none":
        d = d * _slope(st["z"].float(), st["act"])
    dx = d @ _plain_weights(st)
    if not n:
        return dx.to(st["dy"].dtype)
    x, on = st["x"].float(), _chosen(st)
    a, b = st["a"].float().view(n * R, K), st["b"].float().transpose(1, 2).reshape(n * R, N)
    h = (x @ a.t()) * on
    u = (d @ b.t()) * on
    dx = dx + u @ a
    da, db = (u.t() @ x).view(n, R, K), (h.t() @ d).view(n, R, N).transpose(1, 2).contiguous()
    return dx.to(st["dy"].dtype), da.to(st["a"].dtype), db.to(st["b"].dtype)


def _plain_clip(st):
    g = torch.cat(st["grads"])
    norm = torch.sqrt((g.double() * g.double()).sum())
    return norm.float().view(1), (g.float() * (st["max_norm"] / norm).clamp(max=1.0).float()).to(g.dtype)


# ------------------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """The operators' definitions in 64 bits, written without the plain forms: adapters one after another over their own
    tokens, gradients by differentiation."""
    if case["op"] == "clip":
        g = _gradients(case, seed)
        norm = torch.linalg.vector_norm(g[0].double())
        return norm.view(1), g[0].double() * min(1.0, g[1] / float(norm))
    N, K, G = case["N"], case["K"], case["group"] or case["K"]
    q, s = _codes(case, seed)
    w = q.double().view(N, K // G, G).mul_(s.double()[:, :, None]).view(N, K)
    x = _hidden(case, seed).double()
    if case["op"] == "adapted":
        bias, res = _forward_extras(case, seed)
        v = torch.mm(x, w.t())
        v = _with_adapters(case, seed, x, v, *[t.double() for t in _adapters(case, seed)])
        v = v if bias is None else v + bias.double()
        y = _act64(v, case["act"])
        y = y if res is None else y + res.double()
        return (y, v) if case["pre"] else y
    dy, z = _gradient_inputs(case, seed)
    dz = dy.double()
    if z is not None:
        z = z.double().requires_grad_(True)
        dz = torch.autograd.grad(_act64(z, case["act"]), z, dz)[0]
    dx = torch.mm(dz, w)
    if not case["n"]:
        return dx
    x = x.requires_grad_(True)
    a, b, sc = (t.double() for t in _adapters(case, seed))
    a, b = a.requires_grad_(True), b.requires_grad_(True)
    v = _with_adapters(case, seed, x, torch.zeros((case["T"], N), dtype=torch.float64, device="cuda"), a, b, sc)
    if not v.requires_grad:  # no token has an adapter
        return dx, torch.zeros_like(a), torch.zeros_like(b)
    gx, ga, gb = torch.autograd.grad(v, (x, a, b), dz)
    return dx + gx, ga, gb


def _with_adapters(case, seed, x, v, a, b, sc):
    ids = _ids(case, seed).long()
    for k in range(case["n"]):
        rows = torch.nonzero(ids == k).view(-1)
        if rows.numel():
            v = v.index_add(0, rows, torch.mm(torch.mm(x[rows], a[k].t()), b[k].t()) * sc[k])
    return v


def _act64(v, act):
    if act == "swiglu":
        g, u = v.chunk(2, dim=1)
        return g * u * torch.special.expit(g)
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * v * (1 + 0.044715 * v * v))
    return v
