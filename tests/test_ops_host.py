"""Host-side checks of the routing and linear entry points (no GPU needed): bad arguments are refused before any
device work, by the library and by the binding; the plain references of the GPU tests on hand-worked values."""
import ctypes

import numpy as np
import pytest

import int4_quantized_expert_amd as moe
from int4_quantized_expert_amd import _lib as L
from tests import ops_reference as R

P = ctypes.c_void_p
A, WS = P(4096), P(65536)


def _route(cfg, logits=A, dtype=0, ld=256, T=4, bias=None, valid=None, ids=A, w=A, load=None, imp=None, ws=None, n=0):
    c = cfg.c()
    return L._lib.moe_route(ctypes.byref(c), logits, dtype, ld, T, bias, valid, ids, w, load, imp, ws, n, None)


def _back(cfg, logits=A, dtype=0, ld=256, T=4, valid=None, ids=A, dw=A, dimp=None, dz=P(8192), ldd=256):
    c = cfg.c()
    return L._lib.moe_route_backward(ctypes.byref(c), logits, dtype, ld, T, valid, ids, dw, dimp, dz, ldd, None)


@pytest.mark.parametrize("bad,code", [(dict(n_experts=0), "SHAPE"), (dict(n_experts=1025), "SHAPE"),
                                      (dict(top_k=0), "SHAPE"), (dict(top_k=33), "SHAPE"),
                                      (dict(n_group=7), "SHAPE"), (dict(n_group=128), "SHAPE"),
                                      (dict(n_group=64, topk_group=1, top_k=5), "SHAPE"),
                                      (dict(topk_group=2), "SHAPE"), (dict(topk_group=0), "SHAPE"),
                                      (dict(score=2), "ARG"), (dict(group_score=-1), "ARG"), (dict(renorm=2), "ARG"),
                                      (dict(scale=float("nan")), "ARG"), (dict(scale=0.0), "ARG"),
                                      (dict(scale=float("inf")), "ARG")])
def test_route_configs_refused(bad, code):
    cfg = moe.RouteConfig(256, 8)
    for k, v in bad.items():
        setattr(cfg, k, v)
    rc = getattr(L, "MOE_E_" + code)
    assert _route(cfg) == rc
    assert _back(cfg) == rc
    assert moe.moe_route_workspace_bytes(cfg, 4) == 0


def test_route_arguments_refused():
    cfg = moe.RouteConfig(256, 8)
    assert _route(cfg, logits=None) == _route(cfg, ids=None) == _route(cfg, w=None) == L.MOE_E_NULL
    assert L._lib.moe_route(None, A, 0, 256, 4, None, None, A, A, None, None, None, 0, None) == L.MOE_E_NULL
    assert _route(cfg, T=0) == _route(cfg, T=(1 << 20) + 1) == L.MOE_E_SHAPE
    assert _route(cfg, dtype=3) == _route(cfg, ld=255) == _route(cfg, logits=P(4098)) == L.MOE_E_ARG
    assert _route(cfg, dtype=1, logits=P(4097)) == _route(cfg, ids=P(4097)) == _route(cfg, bias=P(4098)) == L.MOE_E_ARG
    need = moe.moe_route_workspace_bytes(cfg, 4)
    assert need > 0 and moe.moe_route_workspace_bytes(cfg, 0) == 0
    for kw in (dict(load=A), dict(imp=A)):
        assert _route(cfg, ws=None, n=need, **kw) == L.MOE_E_WORKSPACE
        assert _route(cfg, ws=WS, n=need - 1, **kw) == L.MOE_E_WORKSPACE
        assert _route(cfg, ws=P(65536 + 128), n=need, **kw) == L.MOE_E_WORKSPACE
    assert _back(cfg, logits=None) == _back(cfg, ids=None) == _back(cfg, dz=None) == _back(cfg, dw=None) == L.MOE_E_NULL
    assert _back(cfg, T=0) == L.MOE_E_SHAPE
    assert _back(cfg, ldd=255) == _back(cfg, ld=1) == _back(cfg, dtype=-1) == _back(cfg, dz=P(8194)) == L.MOE_E_ARG


def test_slot_weight_grad_arguments_refused():
    f = L._lib.moe_slot_weight_grad
    assert f(None, A, A, 1, 1, 4, A, None) == f(A, None, A, 1, 1, 4, A, None) == L.MOE_E_NULL
    assert f(A, A, None, 1, 1, 4, A, None) == f(A, A, A, 1, 1, 4, None, None) == L.MOE_E_NULL
    for T, K, H in ((0, 1, 4), (1, 0, 4), (1, 33, 4), (1, 1, 0), (1, 1, 6), (1, 1, 16388)):
        assert f(A, A, A, T, K, H, A, None) == L.MOE_E_SHAPE
    assert f(P(4104), A, A, 1, 1, 4, A, None) == f(A, A, P(4104), 1, 1, 4, A, None) == L.MOE_E_ARG


def test_slot_weight_grad_experts_arguments_refused():
    f = L._lib.moe_slot_weight_grad_experts
    assert f(None, A, A, 1, 1, 4, 8, A, None) == f(A, A, A, 1, 1, 4, 8, None, None) == L.MOE_E_NULL
    for T, K, H, E in ((0, 1, 4, 8), (1, 33, 4, 8), (1, 1, 6, 8), (1, 1, 4, 0), (1, 1, 4, -1), (1, 1, 4, 1025)):
        assert f(A, A, A, T, K, H, E, A, None) == L.MOE_E_SHAPE
    assert f(P(4104), A, A, 1, 1, 4, 8, A, None) == f(A, P(4098), A, 1, 1, 4, 8, A, None) == L.MOE_E_ARG


def _linear(cfg, codes=A, scales=A, bias=None, x=A, ldx=256, T=2, dtype=0, res=None, ldr=0, y=P(1 << 20), ldy=128, ws=WS,
            n=1 << 30):
    c = cfg.c()
    return L._lib.moe_linear(ctypes.byref(c), codes, scales, bias, x, ldx, T, dtype, res, ldr, y, ldy, ws, n, None)


@pytest.mark.parametrize("bad,code", [(dict(rows=0), "SHAPE"), (dict(rows=96), "SHAPE"), (dict(rows=(1 << 20) + 64), "SHAPE"),
                                      (dict(cols=0), "SHAPE"), (dict(cols=48), "SHAPE"), (dict(cols=65536 + 32), "SHAPE"),
                                      (dict(weight_bits=3), "ARG"), (dict(act=6), "ARG"), (dict(act=-1), "ARG"),
                                      (dict(group_size=48), "ARG"), (dict(group_size=96), "ARG"),
                                      (dict(group_size=32, weight_bits=8), "ARG"), (dict(group_size=512), "SHAPE")])
def test_linear_configs_refused(bad, code):
    cfg = moe.LinearConfig(128, 256)
    for k, v in bad.items():
        setattr(cfg, k, v)
    assert _linear(cfg) == getattr(L, "MOE_E_" + code)
    assert moe.moe_linear_workspace_bytes(cfg, 2) == 0


def test_linear_arguments_refused():
    cfg = moe.LinearConfig(128, 256)
    for k in ("codes", "scales", "x", "y"):
        assert _linear(cfg, **{k: None}) == L.MOE_E_NULL
    assert _linear(cfg, T=0) == _linear(cfg, T=(1 << 20) + 1) == L.MOE_E_SHAPE
    assert _linear(cfg, dtype=7) == _linear(cfg, ldx=255) == _linear(cfg, ldy=127) == L.MOE_E_ARG
    assert _linear(cfg, res=A, ldr=127) == _linear(cfg, codes=P(4104)) == _linear(cfg, x=P(4098)) == L.MOE_E_ARG
    assert _linear(cfg, res=P(4098), ldr=128) == _linear(cfg, bias=P(4098)) == L.MOE_E_ARG
    need = moe.moe_linear_workspace_bytes(cfg, 2)
    assert need > 0
    assert _linear(cfg, ws=None) == _linear(cfg, n=need - 1) == _linear(cfg, ws=P(65536 + 8)) == L.MOE_E_WORKSPACE


def test_routed_layer_arguments_refused():
    cfg = moe.Config(6144, 256, 8, 4, 8, 2048, 1, 2.5)
    c = cfg.c()
    w = L.moe_layer_weights(None, None, *([4096] * 8))
    f = L._lib.moe_layer_forward_routed

    def call(x=A, T=4, ids=A, wt=A, y=A, ws=WS, n=1 << 40, taps=None, wts=w):
        return f(ctypes.byref(c), ctypes.byref(wts), x, T, ids, wt, y, ws, n, taps, None)

    assert call(ids=None) == call(wt=None) == call(x=None) == call(y=None) == L.MOE_E_NULL
    assert call(wts=L.moe_layer_weights()) == L.MOE_E_NULL
    assert call(T=0) == L.MOE_E_SHAPE
    assert call(x=P(4100)) == call(ids=P(4098)) == call(wt=P(4097)) == L.MOE_E_ARG
    assert call(n=16) == call(ws=P(65536 + 4)) == L.MOE_E_WORKSPACE
    for name in ("topk_ids", "topk_w", "near_tie"):
        t = L.moe_taps()
        t.sum_slot = -1
        setattr(t, name, 4096)
        assert call(taps=ctypes.byref(t)) == L.MOE_E_ARG


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros((4, 256))
    i = torch.zeros((4, 8), dtype=torch.int32)
    rc, lc = moe.RouteConfig(256, 8), moe.LinearConfig(128, 256)
    with pytest.raises(moe.ArgError):
        moe.moe_route(rc, z, i, z)
    with pytest.raises(moe.ArgError):
        moe.moe_route_backward(rc, z, i, z, d_w=z)
    with pytest.raises(moe.ArgError):
        moe.moe_slot_weight_grad(z, i, z, z)
    with pytest.raises(moe.ArgError):
        moe.moe_linear(lc, z, z, z, z, z)
    with pytest.raises(moe.ArgError):
        moe.moe_layer_forward_routed(moe.Config(256, 16, 4, 2, 4, 128, 1, 2.5), L.moe_layer_weights(), z, i, z, z, z)


def test_reference_route_by_hand():
    z = np.array([[0.0, 2.0, 1.0, -1.0]])
    ids, w, load, imp = R.route(z, "f32", 2, softmax=True, renorm=False)
    p = np.exp(z[0]) / np.exp(z[0]).sum()
    assert ids.tolist() == [[1, 2]] and np.allclose(w[0], p[[1, 2]]) and np.allclose(imp, p)
    assert load.tolist() == [0, 1, 1, 0]
    # the bias moves the choice, not the weight; groups (0, 1) and (2, 3) by their two largest
    ids, w, _, _ = R.route(z, "f32", 1, G=2, KG=1, bias=np.array([0, 0, 1, 1.0]), scale=3.0)
    assert ids.tolist() == [[2]] and np.allclose(w, 3.0)
    # a masked row has no slots
    ids, w, load, imp = R.route(np.full((1, 4), -np.inf), "f32", 2)
    assert ids.tolist() == [[-1, -1]] and not w.any() and not load.any() and not imp.any()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(renorm, softmax):
    rng = np.random.default_rng(4)
    z = rng.normal(0, 1, (3, 6))
    z[0, 2] = -np.inf
    ids = np.array([[1, 2], [5, 0], [-1, 3]], np.int32)
    dw, dimp = rng.normal(0, 1, (3, 2)), rng.normal(0, 1, 6)
    g, _ = R.route_grad(z, "f32", ids, dw, dimp, softmax, renorm, 1.5)
    h = 1e-6
    for t in range(3):
        for e in range(6):
            if not np.isfinite(z[t, e]):
                assert g[t, e] == 0
                continue
            v = []
            for sg in (h, -h):
                zz = z.copy()
                zz[t, e] += sg
                v.append(R.route_value(zz, "f32", ids, dw, dimp, softmax, renorm, 1.5))
            assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) < 1e-8


def test_configs_keep_their_struct_until_a_field_changes():
    import copy
    import pickle
    for cfg, field in ((moe.RouteConfig(256, 8), "top_k"), (moe.LinearConfig(128, 256), "act")):
        a = cfg.ref()
        assert cfg.ref() is a
        for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
            assert other == cfg and getattr(other.ref()._obj, field) == getattr(cfg, field)
        setattr(cfg, field, 2)
        assert getattr(cfg.ref()._obj, field) == 2 and getattr(a._obj, field) != 2


@pytest.mark.parametrize("rows,cols,act", [(64, 32, 0), (64, 65536, 0), (192, 6144, 5), (2048, 2048, 0), (6144, 6144, 5),
                                           (12352, 8320, 0), (131072, 6144, 0), (1 << 20, 32, 0)])
def test_a_workspace_serves_every_smaller_batch(rows, cols, act):
    """A workspace sized for the largest batch is large enough for any other: its size never falls with the tokens."""
    cfg = moe.LinearConfig(rows, cols, act=act)
    last = 0
    for T in (*range(1, 70), *range(70, 7000, 31), 1 << 14, 1 << 17, 1 << 20):
        need = moe.moe_linear_workspace_bytes(cfg, T)
        assert need >= last
        last = need
    assert last >= (1 << 20) * cols * 2
    for E in (1, 64, 100, 256, 512, 1024):
        route, last = moe.RouteConfig(E, 1), 0
        for T in (*range(1, 200), *range(200, 9000, 61), 1 << 20):
            need = moe.moe_route_workspace_bytes(route, T)
            assert need >= last
            last = need
