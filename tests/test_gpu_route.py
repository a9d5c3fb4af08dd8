"""moe_route, moe_route_backward, moe_slot_weight_grad and moe_layer_forward_routed on the GPU, against plain 64-bit
implementations.

Tolerances. Weights: two exponentials (1.5 units of 2^-23 each), the subtraction of the reference logit (|z - ref|
2^-24, below 60 of them for weights that matter; smaller ones are below 1e-26), a sum of 32, a reciprocal: 64 units
of 2^-23. Importance: the same per token, and T additions. Gradients: 64 units of the terms that cancel in them.
"""
import numpy as np
import pytest

from synth import synth
from tests import ops_reference as R
from tests.harness import GpuLayer, config_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import int4_quantized_expert_amd as moe  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -23


def _cfg(E, K, G=1, KG=1, softmax=False, group_max=False, renorm=True, scale=1.0):
    return moe.RouteConfig(E, K, G, KG, moe.MOE_SCORE_SOFTMAX if softmax else moe.MOE_SCORE_SIGMOID,
                           moe.MOE_GROUP_MAX if group_max else moe.MOE_GROUP_TOP2, renorm, scale)


def _logits(rng, T, E, dtype, pad=0, shift=0, sigma=2.0):
    """Device logits [T][E] with rows E + pad apart, starting `shift` elements into the buffer; their exact values."""
    z = torch.from_numpy(rng.normal(0.0, sigma, (T, E)).astype(np.float32)).to(DT[dtype])
    buf = torch.full((T * (E + pad) + shift,), float("nan"), dtype=DT[dtype], device=DEV)
    d = buf[shift:].as_strided((T, E), (E + pad, 1))
    d.copy_(z)
    return d, z.double().numpy()


def _run(cfg, z, K, bias=None, valid=None, stats=True):
    T, E = z.shape
    ids = torch.full((T + 1, K), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, K), float("nan"), device=DEV)
    load = torch.full((E,), -9, dtype=torch.int32, device=DEV) if stats else None
    imp = torch.full((E,), float("nan"), device=DEV) if stats else None
    ws = torch.full((moe.moe_route_workspace_bytes(cfg, T),), 0xA5, dtype=torch.uint8, device=DEV) if stats else None
    moe.moe_route(cfg, z, ids, w, bias=bias, valid=valid, load=load, importance=imp, ws=ws)
    torch.cuda.synchronize()
    assert bool((ids[T] == -7).all()) and bool(w[T].isnan().all())  # nothing behind the last token
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy(), load, imp


def _check(cfg, zd, z64, dtype, kw, bias=None, valid=None):
    K = cfg.top_k
    T = z64.shape[0]
    db = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).to(DEV)
    dv = None if valid is None else torch.from_numpy(np.asarray(valid, np.uint8)).to(DEV)
    ids, w, load, imp = R.route(z64, dtype, K, bias=bias, valid=valid, **kw)
    for stats in (True, False):
        gi, gw, gl, gm = _run(cfg, zd, K, db, dv, stats)
        assert np.array_equal(gi, ids)
        assert np.all(np.abs(gw - w) <= 64 * U * np.abs(w) + 1e-30)
        assert np.all(gw[ids < 0] == 0)
        if stats:
            assert np.array_equal(gl.cpu().numpy(), load)
            assert np.all(np.abs(gm.cpu().numpy() - imp) <= (64 + T) * U * imp + 1e-30)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,K,G,KG", [(1, 1, 1, 1), (5, 5, 1, 1), (16, 4, 4, 2), (64, 8, 1, 1), (65, 3, 1, 1),
                                      (96, 6, 6, 2), (128, 8, 8, 3), (200, 12, 5, 5), (256, 8, 8, 4), (300, 7, 1, 1),
                                      (512, 32, 64, 8), (1000, 9, 10, 4), (1024, 32, 64, 9)])
def test_route_forms(E, K, G, KG, dtype):
    rng = np.random.default_rng(E * 7 + K)
    T = 9
    z, z64 = _logits(rng, T, E, dtype)
    bias = rng.uniform(-0.1, 0.1, E).astype(np.float32)
    for softmax in (False, True):
        for renorm in (False, True):
            for b in (None, bias):
                gm = bool(renorm) != bool(softmax)
                kw = dict(G=G, KG=KG, softmax=softmax, group_max=gm, renorm=renorm, scale=2.5)
                _check(_cfg(E, K, **kw), z, z64, dtype, kw, b)


@pytest.mark.parametrize("dtype,pad,shift", [("f32", 3, 1), ("bf16", 8, 0), ("bf16", 0, 1), ("f16", 5, 4), ("f32", 4, 4)])
@pytest.mark.parametrize("T", [1, 4, 67])
def test_route_strides_and_padding(T, dtype, pad, shift):
    rng = np.random.default_rng(T + pad)
    z, z64 = _logits(rng, T, 256, dtype, pad, shift)
    valid = (rng.random(T) < 0.6).astype(np.uint8) * 3
    kw = dict(G=8, KG=4, scale=2.5)
    _check(_cfg(256, 8, **kw), z, z64, dtype, kw, rng.uniform(-0.1, 0.1, 256).astype(np.float32), valid)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_masks(dtype, renorm, softmax):
    """NaN, -inf and the lowest value mask an expert; +inf is a very large logit; rows with fewer live experts than
    slots, with one and with none; a bias of -inf or NaN; logits so low that every score underflows."""
    rng = np.random.default_rng(3)
    E, K = 24, 4
    z = rng.normal(0, 1, (12, E))
    low = R.LOWEST[dtype]
    z[0, 1:] = -np.inf
    z[1, :] = -np.inf
    z[2, :] = np.nan
    z[3, :] = low
    z[4, 3:] = low
    z[5, 0:20:2] = np.nan
    z[6, 7] = np.inf
    z[7, [2, 9]] = np.inf
    z[8, :] = -3000.0 - np.arange(E) * 0.5 * (4 if dtype == "f16" else 16 if dtype == "bf16" else 1)
    z[9, :] = 60.0
    z[10, 6:] = np.nan  # one live group of 6, others empty
    zt = torch.from_numpy(z.astype(np.float32)).to(DT[dtype])
    if dtype != "f32":
        zt[3, :] = low
        zt[4, 3:] = low
    z64 = zt.double().numpy()
    bias = rng.uniform(-0.1, 0.1, E).astype(np.float32)
    bias[[5, 11]] = -np.inf
    bias[17] = np.nan
    for G, KG in ((1, 1), (4, 2)):
        for b in (None, bias):
            for gm in (False, True):
                kw = dict(G=G, KG=KG, softmax=softmax, group_max=gm, renorm=renorm, scale=1.0)
                _check(_cfg(E, K, **kw), zt.to(DEV), z64, dtype, kw, b)


@pytest.mark.parametrize("softmax", [False, True])
def test_route_close_scores(softmax):
    """Biased scores that differ by a few units of the last place, or not at all: the order is the definition's."""
    rng = np.random.default_rng(11)
    E, K, T = 256, 8, 24
    z = rng.normal(0, 1.5, (1, E)).astype(np.float32).repeat(T, 0)
    s = R.scores(z[0].astype(np.float64), np.ones(E, bool), softmax).astype(np.float32)
    bias = (np.float32(0.5) - s + rng.integers(-3, 4, E).astype(np.float32) * np.float32(2.0 ** -24)).astype(np.float32)
    z[1:] += (rng.integers(-2, 3, (T - 1, E)) * 2.0 ** -22).astype(np.float32)
    zd = torch.from_numpy(z).to(DEV)
    for G, KG in ((1, 1), (8, 4)):
        kw = dict(G=G, KG=KG, softmax=softmax, scale=2.5)
        _check(_cfg(E, K, **kw), zd, z.astype(np.float64), "f32", kw, bias)


def test_route_ties_take_the_lower_index():
    z = np.zeros((3, 128))
    z[1] = np.repeat([1.0, 2.0], 64)
    z[2, ::3] = 5.0
    zd = torch.from_numpy(z.astype(np.float32)).to(DEV)
    for kw in (dict(), dict(G=8, KG=3), dict(softmax=True, renorm=False), dict(G=8, KG=3, group_max=True)):
        _check(_cfg(128, 8, **kw), zd, z, "f32", kw)
        _check(_cfg(128, 8, **kw), zd, z, "f32", kw, np.zeros(128, np.float32))


def test_route_many_tokens_equal_single_ones():
    """A token gets the same result in any batch (9,001 tokens: several per wavefront), and sums repeat bit for bit."""
    rng = np.random.default_rng(5)
    z, _ = _logits(rng, 9001, 64, "bf16")
    cfg = _cfg(64, 6, softmax=True)
    ids, w, load, imp = _run(cfg, z, 6)
    for t in (0, 1, 4095, 8191, 8192, 9000):
        i1, w1, _, _ = _run(cfg, z[t:t + 1], 6, stats=False)
        assert np.array_equal(i1[0], ids[t]) and np.array_equal(w1[0], w[t])
    assert np.array_equal(load.cpu().numpy(), np.bincount(ids.ravel(), minlength=64))
    _, _, load2, imp2 = _run(cfg, z, 6)
    assert torch.equal(imp, imp2) and torch.equal(load, load2)
    assert abs(float(imp.double().sum()) - 9001) < 9001 * 64 * U


@pytest.mark.parametrize("E,K,G,KG,dtype", [(1024, 32, 64, 9, "f32"), (500, 16, 1, 1, "bf16"), (256, 8, 8, 4, "f16")])
def test_route_statistics_of_long_batches(E, K, G, KG, dtype):
    """2,500 tokens, with padding: the workgroups of 16 wavefronts, every expert width; sums against 64 bits."""
    rng = np.random.default_rng(E)
    T = 2500
    z, z64 = _logits(rng, T, E, dtype)
    bias = rng.uniform(-0.1, 0.1, E).astype(np.float32)
    valid = (rng.random(T) < 0.8).astype(np.uint8)
    for softmax in (False, True):
        cfg = _cfg(E, K, G, KG, softmax=softmax)
        gi, gw, gl, gm = _run(cfg, z, K, torch.from_numpy(bias).to(DEV), torch.from_numpy(valid).to(DEV))
        pick = rng.permutation(T)[:60]
        ids, w, _, _ = R.route(z64[pick], dtype, K, G=G, KG=KG, softmax=softmax, bias=bias, valid=valid[pick])
        assert np.array_equal(gi[pick], ids)
        assert np.all(np.abs(gw[pick] - w) <= 64 * U * np.abs(w) + 1e-30)
        assert np.array_equal(gl.cpu().numpy(), np.bincount(gi[gi >= 0], minlength=E))
        s = np.exp(z64 - z64.max(1, keepdims=True)) if softmax else 1 / (1 + np.exp(-z64))
        imp = ((s / s.sum(1, keepdims=True)) * valid[:, None]).sum(0)
        assert np.all(np.abs(gm.cpu().numpy() - imp) <= (64 + T) * U * imp)


def _grad_case(rng, T, E, K, dtype, pad=0):
    z, z64 = _logits(rng, T, E, dtype, pad)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, K)) < 0.15] = -1
    if E > 4:
        z[0, :3] = float("nan")
        z[0, 3] = float("-inf")
        z64 = z.double().cpu().numpy()
    dw = rng.normal(0, 1, (T, K)).astype(np.float32)
    dimp = rng.normal(0, 1, E).astype(np.float32)
    return z, z64, ids, dw, dimp


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,K,pad", [(1, 1, 1, 0), (3, 16, 4, 0), (7, 65, 6, 3), (5, 128, 8, 8), (4, 256, 8, 0),
                                       (3, 300, 5, 1), (2, 1024, 32, 0)])
def test_route_backward(T, E, K, pad, dtype):
    rng = np.random.default_rng(E + T)
    z, z64, ids, dw, dimp = _grad_case(rng, T, E, K, dtype, pad)
    valid = np.ones(T, np.uint8)
    if T > 2:
        valid[1] = 0
    for softmax in (False, True):
        for renorm in (False, True):
            for a, b in ((dw, None), (None, dimp), (dw, dimp)):
                cfg = _cfg(E, K, softmax=softmax, renorm=renorm, scale=2.5)
                out = torch.full((T + 1, E + pad), 7.0, dtype=DT[dtype], device=DEV)
                d = out[:T, :E]
                moe.moe_route_backward(cfg, z, torch.from_numpy(ids).to(DEV), d,
                                       d_w=None if a is None else torch.from_numpy(a).to(DEV),
                                       d_importance=None if b is None else torch.from_numpy(b).to(DEV),
                                       valid=torch.from_numpy(valid).to(DEV))
                torch.cuda.synchronize()
                assert bool((out[T] == 7).all()) and bool((out[:, E:] == 7).all())
                ref, size = R.route_grad(z64, dtype, ids, a, b, softmax, renorm, 2.5, valid)
                tiny = {"f32": 1e-30, "bf16": 1e-30, "f16": 2.0 ** -25}[dtype]  # half the smallest step
                tol = R.HALF_STEP[dtype] * (1 + 64 * U) * np.abs(ref) + 64 * U * size + tiny
                assert np.all(np.abs(d.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(renorm, softmax):
    rng = np.random.default_rng(2)
    T, E, K = 3, 24, 4
    z, z64, ids, dw, dimp = _grad_case(rng, T, E, K, "f32")
    cfg = _cfg(E, K, softmax=softmax, renorm=renorm, scale=1.5)
    d = torch.empty((T, E), device=DEV)
    moe.moe_route_backward(cfg, z, torch.from_numpy(ids).to(DEV), d, d_w=torch.from_numpy(dw).to(DEV),
                           d_importance=torch.from_numpy(dimp).to(DEV))
    g = d.double().cpu().numpy()
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(z64[t, e]):
                assert g[t, e] == 0
                continue
            v = []
            for sg in (h, -h):
                zz = z64.copy()
                zz[t, e] += sg
                v.append(R.route_value(zz, "f32", ids, dw, dimp, softmax, renorm, 1.5))
            # central difference: h^2 of a third derivative below 10, and 1e-15 / h of rounding
            assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) < 10 * h * h + 1e-9 + 64 * U * 10


@pytest.mark.parametrize("T,K,H", [(1, 1, 4), (1, 8, 6144), (3, 2, 260), (7, 8, 1000), (33, 5, 16384), (2, 32, 64)])
def test_slot_weight_grad(T, K, H):
    rng = np.random.default_rng(H)
    e = rng.normal(0, 1, (T * K, H)).astype(np.float32)
    dy = rng.normal(0, 1, (T, H)).astype(np.float32)
    ids = rng.integers(0, 9, (T, K)).astype(np.int32)
    ids[rng.random((T, K)) < 0.2] = -1
    ref = np.einsum("tkh,th->tk", e.reshape(T, K, H).astype(np.float64), dy.astype(np.float64)) * (ids >= 0)
    mag = np.einsum("tkh,th->tk", np.abs(e.reshape(T, K, H)).astype(np.float64), np.abs(dy).astype(np.float64))
    e[(ids < 0).ravel()] = np.nan  # never written by the layer
    out = torch.full((T * K + 1,), 5.0, device=DEV)
    moe.moe_slot_weight_grad(torch.from_numpy(e).to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(dy).to(DEV), out)
    got = out.cpu().numpy()
    assert got[-1] == 5.0
    assert np.all(np.abs(got[:-1].reshape(T, K) - ref) <= (H + 8) * 2.0 ** -24 * mag)
    assert np.all(got[:-1].reshape(T, K)[ids < 0] == 0)


@pytest.mark.parametrize("T,K,H", [(1, 1, 4), (5, 8, 1000), (9, 3, 6144)])
def test_slot_weight_grad_of_ids_beyond_the_experts(T, K, H):
    """With the number of experts, ids from it on drop their slot as negative ones do; their rows hold NaN."""
    rng = np.random.default_rng(H + T)
    E = 16
    e = rng.normal(0, 1, (T * K, H)).astype(np.float32)
    dy = rng.normal(0, 1, (T, H)).astype(np.float32)
    ids = rng.choice([0, 3, E - 1, E, E + 3, 2 ** 31 - 1, -1, -2 ** 31], (T, K)).astype(np.int32)
    on = (ids >= 0) & (ids < E)
    ref = np.einsum("tkh,th->tk", e.reshape(T, K, H).astype(np.float64), dy.astype(np.float64)) * on
    mag = np.einsum("tkh,th->tk", np.abs(e.reshape(T, K, H)).astype(np.float64), np.abs(dy).astype(np.float64))
    e[~on.ravel()] = np.nan
    out = torch.full((T, K), 5.0, device=DEV)
    moe.moe_slot_weight_grad(torch.from_numpy(e).to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(dy).to(DEV),
                             out, n_experts=E)
    got = out.cpu().numpy()
    assert np.all(np.abs(got - ref) <= (H + 8) * 2.0 ** -24 * mag) and np.all(got[~on] == 0)


# ------------------------------------------------------------------------------------------- with the layer

_LAYER = {}


def _layer():
    if "l" not in _LAYER:
        _LAYER["l"] = GpuLayer(synth.TINY)
    return _LAYER["l"]


def _buffers(sh, T):
    H, K = sh.hidden, sh.top_k
    ws = torch.empty(moe.moe_workspace_bytes(config_of(sh), T), dtype=torch.uint8, device=DEV)
    return ws, torch.empty((T, H), device=DEV), torch.empty((T * K + sh.n_shared * T, H), device=DEV)


@pytest.mark.parametrize("gemm_min", [0, 1, 4, 1 << 20])
@pytest.mark.parametrize("T", [1, 2, 7, 40, 300])
def test_routed_layer_equals_the_layer(T, gemm_min):
    """Given the ids and weights of the layer's own router, the routed layer gives its output bit for bit."""
    sh = synth.TINY
    cfg = config_of(sh, gemm_min)
    layer = _layer()
    x = torch.from_numpy(synth.hidden_states(sh, T)).to(DEV)
    ws = torch.empty(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV)
    y, y2 = torch.empty((T, sh.hidden), device=DEV), torch.empty((T, sh.hidden), device=DEV)
    ids = torch.empty((T, sh.top_k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, sh.top_k), device=DEV)
    moe.moe_layer_forward(cfg, layer.weights(), x, y, ws, moe.taps(topk_ids=ids, topk_w=w))
    ws.fill_(0xA5)
    moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, w, y2, ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("gemm_min", [0, 1, 3])
@pytest.mark.parametrize("T", [1, 2, 3, 9])
def test_routed_layer_with_repeated_and_dropped_experts(T, gemm_min):
    """The same expert in several slots of a token (buckets above T positions) and dropped slots: every slot's expert
    output equals the one that the expert gives alone, and the sum runs over the slots in order."""
    sh = synth.TINY
    cfg = config_of(sh, gemm_min)
    layer = _layer()
    K, H, E = sh.top_k, sh.hidden, sh.n_experts
    x = torch.from_numpy(synth.hidden_states(sh, T)).to(DEV)
    ws, y, e_out = _buffers(sh, T)
    alone = {}
    for e0 in range(0, 8, K):
        ids = torch.arange(e0, e0 + K, dtype=torch.int32, device=DEV).repeat(T, 1).contiguous()
        moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, torch.ones((T, K), device=DEV), y, ws,
                                     moe.taps(e_out=e_out))
        for k in range(K):
            alone[e0 + k] = e_out[:T * K].view(T, K, H)[:, k].clone()
    shared = e_out[T * K:].clone()
    rng = np.random.default_rng(T)
    for ids_np in (np.full((T, K), 5), rng.integers(0, 3, (T, K)), np.full((T, K), -1),
                   np.where(rng.random((T, K)) < 0.5, 7, E + 3)):
        ids = torch.from_numpy(ids_np.astype(np.int32)).to(DEV)
        w = torch.from_numpy(rng.uniform(0.1, 1, (T, K)).astype(np.float32)).to(DEV)
        moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, w, y, ws, moe.taps(e_out=e_out))
        got = e_out[:T * K].view(T, K, H)
        acc = shared.double()
        for t in range(T):
            for k in range(K):
                e = int(ids_np[t, k])
                if 0 <= e < E:
                    assert torch.equal(got[t, k], alone[e][t]), (t, k, e)
                    acc[t] += w[t, k].double() * alone[e][t].double()
        assert bool(((y.double() - acc).abs() <= 16 * 2.0 ** -24 * (acc.abs() + 8 * shared.abs().max())).all())


@pytest.mark.parametrize("softmax", [False, True])
def test_router_gradient_through_the_layer(softmax):
    """Router weights tuned through a layer with frozen experts: logits, route, layer, loss, and back. The gradient
    of the logits is compared with differences of the loss in 64 bits over the layer's own expert outputs."""
    sh = synth.TINY
    cfg = config_of(sh)
    layer = _layer()
    T, K, E, H = 6, sh.top_k, sh.n_experts, sh.hidden
    rc = _cfg(E, K, softmax=softmax, renorm=not softmax, scale=2.5)
    x = torch.from_numpy(synth.hidden_states(sh, T)).to(DEV)
    target = torch.from_numpy(np.random.default_rng(1).normal(0, 1, (T, H)).astype(np.float32)).to(DEV)
    logits = (x @ layer.router_w.t()).contiguous()
    ids, w = torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
    load, imp = torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV)
    ws, y, e_out = _buffers(sh, T)
    rws = torch.empty(moe.moe_route_workspace_bytes(rc, T), dtype=torch.uint8, device=DEV)
    moe.moe_route(rc, logits, ids, w, bias=layer.bias, load=load, importance=imp, ws=rws)
    moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, w, y, ws, moe.taps(e_out=e_out))
    dy = y - target
    dw = torch.empty((T, K), device=DEV)
    moe.moe_slot_weight_grad(e_out, ids, dy, dw)
    dimp = 0.01 * E * load.float() / (T * T)  # of the balance term 0.01 E sum_e (load_e / T) (importance_e / T)
    dz = torch.empty_like(logits)
    moe.moe_route_backward(rc, logits, ids, dz, d_w=dw, d_importance=dimp)
    torch.cuda.synchronize()
    z64, e64 = logits.double().cpu().numpy(), e_out.double().cpu().numpy()
    idn, tg, fr = ids.cpu().numpy(), target.double().cpu().numpy(), load.double().cpu().numpy()

    def loss(z):
        out = 0.0
        for t in range(T):
            on = np.zeros(E, bool)
            on[idn[t]] = True
            r = 2.5 * (R.scores(z[t], np.ones(E, bool), True) if softmax else R.shares(z[t], on, False))
            yt = e64[T * K + t] + sum(r[idn[t, k]] * e64[t * K + k] for k in range(K))
            out += 0.5 * ((yt - tg[t]) ** 2).sum()
            out += 0.01 * E / (T * T) * float(fr @ R.shares(z[t], np.ones(E, bool), softmax))
        return out

    g = dz.double().cpu().numpy()
    h = 1e-4
    num = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            zp, zm = z64.copy(), z64.copy()
            zp[t, e] += h
            zm[t, e] -= h
            num[t, e] = (loss(zp) - loss(zm)) / (2 * h)
    # fp32 dot products over H = 256 and the layer's own rounding of y: below 2e-5 of the largest
    assert np.abs(num - g).max() <= 2e-5 * np.abs(num).max()


def test_route_streams_and_graph_replays():
    """On a side stream, and captured: every replay equals the eager call on the same inputs, with eager work and
    synchronizations between the replays."""
    rng = np.random.default_rng(8)
    T, E, K = 130, 256, 8
    cfg = _cfg(E, K, 8, 4, scale=2.5)
    z, _ = _logits(rng, T, E, "f32")
    bias = torch.from_numpy(rng.uniform(-0.1, 0.1, E).astype(np.float32)).to(DEV)
    inputs = [_logits(rng, T, E, "f32")[0] for _ in range(4)]
    dw, dimp = torch.randn((T, K), device=DEV), torch.randn(E, device=DEV)

    def bufs():
        return (torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV),
                torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV),
                torch.empty((T, E), device=DEV),
                torch.empty(moe.moe_route_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV))

    def call(zz, b):
        moe.moe_route(cfg, zz, b[0], b[1], bias=bias, load=b[2], importance=b[3], ws=b[5])
        moe.moe_route_backward(cfg, zz, b[0], b[4], d_w=dw, d_importance=dimp)

    side = torch.cuda.Stream()
    got, want = bufs(), bufs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(z, got)
    torch.cuda.current_stream().wait_stream(side)
    call(z, want)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(z, got)
    for zz in inputs:
        z.copy_(zz)
        call(zz, want)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))


def test_dropped_slots_from_the_layer_to_the_logits():
    """Slots dropped by -1, by the number of experts and by ids beyond it mean the same to the layer, to the gradient
    of its weights and to the gradient of the logits, although the layer writes no expert output for any of them."""
    sh = synth.TINY
    cfg, layer = config_of(sh), _layer()
    T, K, E, H = 6, sh.top_k, sh.n_experts, sh.hidden
    rng = np.random.default_rng(9)
    x = torch.from_numpy(synth.hidden_states(sh, T)).to(DEV)
    kept = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    drop = rng.random((T, K)) < 0.4
    drop[2] = True
    dy = torch.from_numpy(rng.normal(0, 1, (T, H)).astype(np.float32)).to(DEV)
    w = torch.from_numpy(rng.uniform(0.1, 1, (T, K)).astype(np.float32)).to(DEV)
    logits, _ = _logits(rng, T, E, "f32")
    rc = _cfg(E, K)
    results = []
    for away in (-1, E, E + 3):
        ids = torch.from_numpy(np.where(drop, away, kept).astype(np.int32)).to(DEV)
        ws, y, e_out = _buffers(sh, T)
        e_out.fill_(float("nan"))
        moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, w, y, ws, moe.taps(e_out=e_out))
        dw, dz = torch.empty((T, K), device=DEV), torch.empty((T, E), device=DEV)
        moe.moe_slot_weight_grad(e_out, ids, dy, dw, n_experts=E)
        moe.moe_route_backward(rc, logits, ids, dz, d_w=dw)
        assert bool((dw[torch.from_numpy(drop).to(DEV)] == 0).all()) and bool(dz.isfinite().all())
        results.append((y, dw, dz))
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))


@pytest.mark.parametrize("size", [1.0e4, 6.0e4])
def test_route_groups_of_large_opposite_biases(size):
    """Group sums whose two addends are large and of opposite sign: what a score loses by its addition to the bias is
    of the size of the addends, not of the sum. One expert of each group has the bias +size, the others -size, and the
    former's score lies within a few steps of a value where its sum with the bias falls between two floats, so that a
    score off by one step moves the sum by a whole one (2^-10 at 1e4). The groups are the definition's."""
    rng = np.random.default_rng(int(size))
    G, n, T = 8, 4, 400
    step = 2.0 ** (np.floor(np.log2(size)) - 23)
    # scores (k + 1/2) step, which size + score cannot hold, in (0.3, 0.7)
    s = (rng.integers(int(0.3 / step), int(0.7 / step), (T, 1)) + 0.5) * step
    z = np.full((T, G, n), 0.25)
    z[:, :, 0] = np.log(s / (1 - s)) + rng.integers(-3, 4, (T, G)) * 2.0 ** -24
    z = z.reshape(T, G * n).astype(np.float32)
    bias = np.full((G, n), -size)
    bias[:, 0] = size
    for K, KG in ((4, 2), (1, 1), (8, 5)):
        kw = dict(G=G, KG=KG, scale=2.5)
        _check(_cfg(G * n, K, **kw), torch.from_numpy(z).to(DEV), z.astype(np.float64), "f32", kw,
               bias.ravel().astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E", [24, 256])
def test_route_backward_with_infinite_gradients_of_masked_experts(E, softmax, dtype):
    """An expert that is masked in every token has importance 0, where the logarithm of a balance loss has an infinite
    gradient: the tokens do not depend on it, and their gradients are those without it."""
    rng = np.random.default_rng(E)
    T, K = 5, 4
    z, _ = _logits(rng, T, E, dtype)
    z[:, 2], z[:, 9], z[:, E - 1] = float("-inf"), float("nan"), R.LOWEST[dtype]
    z[3, :4] = float("-inf")  # one token with more of them masked
    z[4, :] = float("-inf")  # and one without live experts
    z[1, :] -= 60.0  # scores so low that the sum is taken relative to the largest
    z64 = z.double().cpu().numpy()
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    dw, dimp = rng.normal(0, 1, (T, K)).astype(np.float32), rng.normal(0, 1, E).astype(np.float32)
    dimp[[2, 9, E - 1]] = 0.0
    bad = dimp.copy()
    bad[[2, 9, E - 1]] = np.inf, np.nan, -np.inf
    for renorm in (False, True):
        cfg = _cfg(E, K, softmax=softmax, renorm=renorm, scale=2.5)
        ref, size = R.route_grad(z64, dtype, ids, dw, dimp, softmax, renorm, 2.5)
        d = torch.full((T, E), 7.0, dtype=DT[dtype], device=DEV)
        moe.moe_route_backward(cfg, z, torch.from_numpy(ids).to(DEV), d, d_w=torch.from_numpy(dw).to(DEV),
                               d_importance=torch.from_numpy(bad).to(DEV))
        tiny = {"f32": 1e-30, "bf16": 1e-30, "f16": 2.0 ** -25}[dtype]
        tol = R.HALF_STEP[dtype] * (1 + 64 * U) * np.abs(ref) + 64 * U * size + tiny
        assert np.all(np.abs(d.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("weight_bits,group_size", [(8, 0), (4, 32), (4, 64)])
@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_routed_layer_equals_the_layer_in_other_formats(T, weight_bits, group_size):
    """int8 experts and int4 ones with group scales: the routed layer's output is the layer's, bit for bit."""
    sh = synth.TINY
    key = (weight_bits, group_size)
    if key not in _LAYER:
        _LAYER[key] = GpuLayer(sh, weight_bits=weight_bits, group_size=group_size)
    layer, cfg = _LAYER[key], config_of(sh, 0, weight_bits, group_size)
    x = torch.from_numpy(synth.hidden_states(sh, T)).to(DEV)
    ws = torch.empty(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV)
    y, y2 = torch.empty((T, sh.hidden), device=DEV), torch.empty((T, sh.hidden), device=DEV)
    ids = torch.empty((T, sh.top_k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, sh.top_k), device=DEV)
    moe.moe_layer_forward(cfg, layer.weights(), x, y, ws, moe.taps(topk_ids=ids, topk_w=w))
    ws.fill_(0xA5)
    moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, w, y2, ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("T", [1, 4, 32, 192, 700])
def test_routed_layer_equals_the_layer_at_full_size(T):
    """The same with hidden 6144, 256 experts of 2048 and top 8; and under moe_route's own routing of the logits, with
    a third of the tokens masked, whose rows are the shared expert's output alone."""
    sh = synth.GLM
    if "glm" not in _LAYER:
        _LAYER["glm"] = GpuLayer(sh)
    layer, cfg = _LAYER["glm"], config_of(sh)
    E, K, H = sh.n_experts, sh.top_k, sh.hidden
    x = torch.from_numpy(synth.hidden_states(sh, T)).to(DEV)
    ws = torch.empty(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV)
    y, y2 = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    ids, w = torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
    moe.moe_layer_forward(cfg, layer.weights(), x, y, ws, moe.taps(topk_ids=ids, topk_w=w))
    moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids, w, y2, ws)
    assert torch.equal(y, y2)
    rc = _cfg(E, K, sh.n_group, sh.topk_group, scale=sh.rsf)
    valid = (torch.arange(T, device=DEV) % 3 != 1).to(torch.uint8)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    moe.moe_route(rc, (x @ layer.router_w.t()).contiguous(), ids2, w2, bias=layer.bias, valid=valid)
    e_out = torch.empty((T * K + sh.n_shared * T, H), device=DEV)
    moe.moe_layer_forward_routed(cfg, layer.weights(), x, ids2, w2, y2, ws, moe.taps(e_out=e_out))
    assert torch.equal(y2[valid == 0], e_out[T * K:T * K + T][valid == 0])
    if T == 700:
        del _LAYER["glm"]


@pytest.mark.parametrize("softmax", [False, True])
def test_route_largest_batch(softmax):
    """2^20 tokens, the most that the operators take: tokens at both ends and between as they come out alone, counts
    and sums over all; the gradient and the slots' gradient of the same batch."""
    T, E, K = 1 << 20, 8, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn((T, E), device=DEV, generator=g)
    cfg = _cfg(E, K, softmax=softmax)
    ids, w, load, imp = _run(cfg, z, K)
    assert np.array_equal(load.cpu().numpy(), np.bincount(ids.ravel(), minlength=E))
    assert abs(float(imp.double().sum()) - T) < T * 64 * U
    idd, dw, dimp = torch.from_numpy(ids).to(DEV), torch.randn((T, K), device=DEV, generator=g), torch.randn(E, device=DEV)
    dz = torch.empty_like(z)
    moe.moe_route_backward(cfg, z, idd, dz, d_w=dw, d_importance=dimp)
    for t in (0, 1, 65535, 524288, T - 1):
        i1, w1, _, _ = _run(cfg, z[t:t + 1], K, stats=False)
        assert np.array_equal(i1[0], ids[t]) and np.array_equal(w1[0], w[t])
        d1 = torch.empty((1, E), device=DEV)
        moe.moe_route_backward(cfg, z[t:t + 1], idd[t:t + 1].contiguous(), d1, d_w=dw[t:t + 1].contiguous(), d_importance=dimp)
        assert torch.equal(d1[0], dz[t])
    e_out, dy = torch.randn((T * K, E), device=DEV, generator=g), z
    got = torch.empty((T, K), device=DEV)
    moe.moe_slot_weight_grad(e_out, idd, dy, got)
    ref = (e_out.view(T, K, E).double() * dy.double()[:, None, :]).sum(2)
    mag = (e_out.view(T, K, E).double() * dy.double()[:, None, :]).abs().sum(2)
    assert bool(((got.double() - ref).abs() <= (E + 8) * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("T", [1, 7, 200])
def test_router_tuning_step_captured(T):
    """Route, layer, both gradients, on a captured stream: every replay, with other inputs and eager work between the
    replays, equals the eager chain. Weights of dropped slots are NaN for the layer, which does not use them."""
    sh = synth.TINY
    cfg, layer = config_of(sh), _layer()
    K, E, H = sh.top_k, sh.n_experts, sh.hidden
    rc = _cfg(E, K, sh.n_group, sh.topk_group, scale=2.5)
    valid = (torch.arange(T, device=DEV) % 5 != 3).to(torch.uint8)
    target = torch.randn((T, H), device=DEV)
    rws = [torch.empty(moe.moe_route_workspace_bytes(rc, T), dtype=torch.uint8, device=DEV) for _ in range(2)]

    def bufs():
        ws, y, e_out = _buffers(sh, T)
        return dict(ws=ws, y=y, e_out=e_out, ids=torch.empty((T, K), dtype=torch.int32, device=DEV),
                    w=torch.empty((T, K), device=DEV), load=torch.empty(E, dtype=torch.int32, device=DEV),
                    imp=torch.empty(E, device=DEV), dw=torch.empty((T, K), device=DEV), dz=torch.empty((T, E), device=DEV),
                    dy=torch.empty((T, H), device=DEV))

    def step(x, z, b, rw):
        moe.moe_route(rc, z, b["ids"], b["w"], bias=layer.bias, valid=valid, load=b["load"], importance=b["imp"], ws=rw)
        b["w"].masked_fill_(b["ids"] < 0, float("nan"))
        moe.moe_layer_forward_routed(cfg, layer.weights(), x, b["ids"], b["w"], b["y"], b["ws"], moe.taps(e_out=b["e_out"]))
        torch.sub(b["y"], target, out=b["dy"])
        moe.moe_slot_weight_grad(b["e_out"], b["ids"], b["dy"], b["dw"], n_experts=E)
        moe.moe_route_backward(rc, z, b["ids"], b["dz"], d_w=b["dw"], d_importance=b["imp"], valid=valid)

    xs = [torch.from_numpy(synth.hidden_states(sh, T, step=i)).to(DEV) for i in range(4)]
    zs = [(x @ layer.router_w.t()).contiguous() for x in xs]
    x, z, got, want = xs[0].clone(), zs[0].clone(), bufs(), bufs()
    step(x, z, got, rws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(x, z, got, rws[0])
    for xx, zz in zip(xs, zs):
        x.copy_(xx)
        z.copy_(zz)
        step(xx, zz, want, rws[1])
        g.replay()
        torch.cuda.synchronize()
        assert bool(want["y"].isfinite().all()) and bool(want["dz"].isfinite().all())
        for k in ("ids", "load", "imp", "y", "dw", "dz"):
            assert torch.equal(got[k], want[k]), k
        assert torch.equal(got["w"][got["ids"] >= 0], want["w"][want["ids"] >= 0])


@pytest.mark.parametrize("T", [3, 2500])
def test_route_load_or_importance_alone(T):
    """Each of the two sums without the other, with the same bits as together; and without live experts or tokens."""
    rng = np.random.default_rng(T)
    E, K = 96, 6
    z, _ = _logits(rng, T, E, "bf16")
    cfg = _cfg(E, K, 6, 2)
    ids, w, load, imp = _run(cfg, z, K)
    ws = torch.empty(moe.moe_route_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV)
    i2, w2 = torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
    l2, m2 = torch.full_like(load, -1), torch.full_like(imp, -1.0)
    moe.moe_route(cfg, z, i2, w2, load=l2, ws=ws)
    moe.moe_route(cfg, z, i2, w2, importance=m2, ws=ws)
    assert torch.equal(l2, load) and torch.equal(m2, imp) and np.array_equal(i2.cpu().numpy(), ids)
    moe.moe_route(cfg, z, i2, w2, valid=torch.zeros(T, dtype=torch.uint8, device=DEV), load=l2, importance=m2, ws=ws)
    assert bool((i2 == -1).all()) and not bool(w2.any()) and not bool(l2.any()) and not bool(m2.any())
    moe.moe_route(cfg, torch.full_like(z, float("-inf")), i2, w2, load=l2, importance=m2, ws=ws)
    assert bool((i2 == -1).all()) and not bool(w2.any()) and not bool(l2.any()) and not bool(m2.any())
