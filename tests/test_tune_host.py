"""Host-side checks of the adapted product, its gradients and gradient clipping (no GPU needed): bad arguments are refused
before any device work, workspaces, and the plain references of the GPU tests by hand and by differences."""
import ctypes

import numpy as np
import pytest

import int4_quantized_expert_amd as moe
from int4_quantized_expert_amd import _lib as L
from tests import tune_reference as R

P = ctypes.c_void_p
A, B2, WS = P(4096), P(1 << 20), P(65536)


def _ad(n=2, rank=16, a=4096, b=4096, scale=4096):
    return L.moe_adapters(n, rank, a, b, scale)


def _forward(cfg, ad=None, ids=None, codes=A, scales=A, bias=None, x=A, ldx=256, T=2, dtype=0, res=None, ldr=0, y=B2, ldy=128,
             pre=None, ldp=0, ws=WS, n=1 << 40):
    c = cfg.c()
    return L._lib.moe_linear_adapted(ctypes.byref(c), codes, scales, bias, None if ad is None else ctypes.byref(ad), ids, x,
                                     ldx, T, dtype, res, ldr, y, ldy, pre, ldp, ws, n, None)


def _backward(cfg, ad=None, ids=None, codes=A, scales=A, x=A, ldx=256, T=2, dtype=0, pre=A, ldp=128, dy=A, ldd=128, res=None,
              ldr=256, dx=B2, ldg=256, da=None, db=None, ws=WS, n=1 << 40):
    c = cfg.c()
    return L._lib.moe_linear_backward(ctypes.byref(c), codes, scales, None if ad is None else ctypes.byref(ad), ids, x, ldx, T,
                                      dtype, pre, ldp, dy, ldd, res, ldr, dx, ldg, da, db, ws, n, None)


@pytest.mark.parametrize("bad,code", [(dict(rows=96), "SHAPE"), (dict(cols=48), "SHAPE"), (dict(weight_bits=3), "ARG"),
                                      (dict(act=6), "ARG"), (dict(group_size=48), "ARG"),
                                      (dict(group_size=32, weight_bits=8), "ARG"), (dict(group_size=512), "SHAPE")])
def test_configs_refused(bad, code):
    cfg = moe.LinearConfig(128, 256)
    for k, v in bad.items():
        setattr(cfg, k, v)
    assert _forward(cfg) == _backward(cfg) == getattr(L, "MOE_E_" + code)
    assert moe.moe_linear_adapted_workspace_bytes(cfg, None, 2) == moe.moe_linear_backward_workspace_bytes(cfg, None, 2) == 0


@pytest.mark.parametrize("bad", [dict(n=0), dict(n=1025), dict(rank=0), dict(rank=4), dict(rank=20), dict(rank=136)])
def test_adapter_sizes_refused(bad):
    cfg, ad = moe.LinearConfig(128, 256), _ad(**bad)
    assert _forward(cfg, ad) == _backward(cfg, ad) == L.MOE_E_SHAPE
    for f in (L._lib.moe_linear_adapted_workspace_bytes, L._lib.moe_linear_backward_workspace_bytes):
        assert f(cfg.ref(), ctypes.byref(ad), 2) == 0


def test_adapter_arrays_refused():
    cfg = moe.LinearConfig(128, 256)
    for bad in (dict(a=None), dict(b=None), dict(scale=None)):
        assert _forward(cfg, _ad(**bad)) == _backward(cfg, _ad(**bad)) == L.MOE_E_NULL
    for bad in (dict(a=4104), dict(b=4100), dict(scale=4098)):
        assert _forward(cfg, _ad(**bad)) == _backward(cfg, _ad(**bad)) == L.MOE_E_ARG
    assert _forward(cfg, _ad(), ids=P(4098)) == _backward(cfg, _ad(), ids=P(4098)) == L.MOE_E_ARG


def test_forward_arguments_refused():
    cfg, ad = moe.LinearConfig(128, 256), _ad()
    for k in ("codes", "scales", "x", "y"):
        assert _forward(cfg, ad, **{k: None}) == L.MOE_E_NULL
    assert _forward(cfg, ad, T=0) == _forward(cfg, ad, T=(1 << 20) + 1) == L.MOE_E_SHAPE
    assert _forward(cfg, ad, dtype=3) == _forward(cfg, ad, ldx=255) == _forward(cfg, ad, ldy=127) == L.MOE_E_ARG
    assert _forward(cfg, ad, pre=A, ldp=127) == _forward(cfg, ad, pre=P(4098), ldp=128) == L.MOE_E_ARG
    assert _forward(cfg, ad, res=A, ldr=127) == _forward(cfg, ad, codes=P(4104)) == L.MOE_E_ARG
    need = L._lib.moe_linear_adapted_workspace_bytes(cfg.ref(), ctypes.byref(ad), 2)
    assert need > moe.moe_linear_workspace_bytes(cfg, 2)
    assert _forward(cfg, ad, ws=None) == _forward(cfg, ad, n=need - 1) == _forward(cfg, ad, ws=P(65536 + 8)) == L.MOE_E_WORKSPACE
    swiglu = moe.LinearConfig(128, 256, act=moe.MOE_ACT_SWIGLU)
    assert _forward(swiglu, ad, ldy=63) == _forward(swiglu, ad, ldy=64, pre=A, ldp=127) == L.MOE_E_ARG


def test_backward_arguments_refused():
    cfg, ad = moe.LinearConfig(128, 256, act=moe.MOE_ACT_SILU), _ad()
    for k in ("codes", "scales", "dy", "pre", "dx"):
        assert _backward(cfg, **{k: None}) == L.MOE_E_NULL
    assert _backward(cfg, da=A) == _backward(cfg, db=A) == L.MOE_E_NULL          # gradients of no adapters
    assert _backward(cfg, ad, da=A, x=None) == _backward(cfg, dx=None, res=A, da=A, ad=ad) == L.MOE_E_NULL
    assert _backward(cfg, T=0) == L.MOE_E_SHAPE
    assert _backward(cfg, ldd=127) == _backward(cfg, ldp=127) == _backward(cfg, ldg=255) == L.MOE_E_ARG
    assert _backward(cfg, ad, da=B2, ldx=255) == _backward(cfg, res=A, ldr=255) == _backward(cfg, dtype=-1) == L.MOE_E_ARG
    assert _backward(cfg, ad, da=P(4104)) == _backward(cfg, ad, db=P(4104)) == _backward(cfg, dy=P(4098)) == L.MOE_E_ARG
    for bad in (dict(x=P(4098), da=B2), dict(pre=P(4098)), dict(dx=P(4098)), dict(res=P(4098))):
        assert _backward(cfg, ad, **bad) == L.MOE_E_ARG
    need = L._lib.moe_linear_backward_workspace_bytes(cfg.ref(), ctypes.byref(ad), 2)
    assert _backward(cfg, ad, ws=None) == _backward(cfg, ad, n=need - 1) == _backward(cfg, ad, ws=P(65536 + 8)) == L.MOE_E_WORKSPACE


def _grad(g=4096, out=4096, n=16, dtype=0):
    return L.moe_grad(g, out, n, dtype)


def _table(grads, table=WS, size=1 << 40):
    c = (L.moe_grad * len(grads))(*grads)
    return L._lib.moe_grad_table(c, len(grads), table, size, ctypes.byref(L.moe_grads()), None)


def test_grad_tables_refused():
    assert _table([_grad(g=None)]) == _table([_grad(out=None)]) == L.MOE_E_NULL
    assert L._lib.moe_grad_table(None, 1, WS, 1 << 40, ctypes.byref(L.moe_grads()), None) == L.MOE_E_NULL
    c = (L.moe_grad * 1)(_grad())
    assert L._lib.moe_grad_table(c, 1, WS, 1 << 40, None, None) == L.MOE_E_NULL
    assert L._lib.moe_grad_table(c, 0, WS, 1 << 40, ctypes.byref(L.moe_grads()), None) == L.MOE_E_SHAPE
    assert _table([_grad(n=-1)]) == _table([_grad(n=(1 << 40) + 1)]) == L.MOE_E_SHAPE
    assert _table([_grad(dtype=3)]) == _table([_grad(g=4098, out=4098)]) == _table([_grad(g=4097, out=4097, dtype=1)]) == L.MOE_E_ARG
    # the same tensor twice, an output in another's gradient, in another's output, half in its own gradient
    assert _table([_grad(), _grad()]) == _table([_grad(), _grad(g=8192, out=4096 + 32)]) == L.MOE_E_ARG
    assert _table([_grad(out=8192), _grad(g=16384, out=8192 + 60)]) == _table([_grad(out=4096 + 32)]) == L.MOE_E_ARG
    assert _table([_grad(out=8192), _grad(g=8192 + 60, out=16384)]) == L.MOE_E_ARG
    # in place, elsewhere, one gradient read twice, and side by side: only the table is missing
    ok = [_grad(), _grad(4096 + 64, 4096 + 64), _grad(1 << 20, 1 << 21), _grad(1 << 20, 1 << 22), _grad(None, None, 0)]
    c = (L.moe_grad * len(ok))(*ok)
    need = L._lib.moe_grad_table_bytes(c, len(ok))
    assert need > 0
    assert _table(ok, None) == _table(ok, WS, need - 1) == _table(ok, P(65536 + 8)) == L.MOE_E_WORKSPACE
    assert L._lib.moe_grad_table_bytes(c, 0) == 0


def test_clip_arguments_refused():
    f = L._lib.moe_grad_clip
    t = L.moe_grads(1, 1, 65536)
    assert f(None, 1.0, A, None) == f(ctypes.byref(t), 1.0, None, None) == L.MOE_E_NULL
    for bad in (0.0, -1.0, float("nan")):
        assert f(ctypes.byref(t), bad, A, None) == L.MOE_E_ARG
    assert f(ctypes.byref(t), 1.0, P(4098), None) == L.MOE_E_ARG
    assert f(ctypes.byref(L.moe_grads(0, 0, 65536)), 1.0, A, None) == L.MOE_E_SHAPE
    assert f(ctypes.byref(L.moe_grads(1, 1, None)), 1.0, A, None) == L.MOE_E_WORKSPACE


def test_binding_refuses_host_tensors():
    import torch
    z, cfg = torch.zeros((4, 256)), moe.LinearConfig(128, 256)
    with pytest.raises(moe.ArgError):
        moe.Adapters(torch.zeros((1, 8, 256)), torch.zeros((1, 128, 8)), torch.zeros(1))
    with pytest.raises(moe.ArgError):
        moe.moe_linear_adapted(cfg, z, z, None, None, z, z, z)
    with pytest.raises(moe.ArgError):
        moe.moe_linear_backward(cfg, z, z, z, z, z)
    with pytest.raises(moe.ArgError):
        moe.GradTable([z])
    with pytest.raises(moe.ArgError):
        moe.GradTable([])


@pytest.mark.parametrize("rows,cols,act,rank", [(64, 32, 0, 8), (192, 6144, 5, 16), (6144, 6144, 5, 128), (12352, 8320, 0, 64),
                                                (131072, 6144, 2, 8)])
def test_a_workspace_serves_every_smaller_batch(rows, cols, act, rank):
    cfg, ad = moe.LinearConfig(rows, cols, act=act), _ad(64, rank)
    for f in (L._lib.moe_linear_adapted_workspace_bytes, L._lib.moe_linear_backward_workspace_bytes):
        for adapters in (None, ctypes.byref(ad)):
            last = 0
            for T in (*range(1, 70), *range(70, 9000, 31), 1 << 14, 1 << 17, 1 << 20):
                need = f(cfg.ref(), adapters, T)
                assert need >= last
                last = need


def test_reference_by_hand():
    q, s = np.array([[1.0, 2.0], [0.0, -1.0]]), np.array([[0.5], [2.0]])
    x, a, b = np.array([[1.0, 1.0], [2.0, 0.0]]), np.array([[[1.0, -1.0]], [[0.0, 3.0]]]), np.array([[[1.0], [2.0]], [[1.0], [0.0]]])
    y, _, z, _ = R.adapted(q, s, x, a, b, np.array([1.0, 0.5]), [1, 0], "f32", "relu", np.array([0.0, 1.0]))
    # token 0: W x = (1.5, -2), adapter 1: 0.5 * 3 * (1, 0); token 1: (1, 0), adapter 0: 2 * (1, 2)
    assert np.allclose(z, [[3.0, -1.0], [3.0, 5.0]]) and np.allclose(y, [[3.0, 0.0], [3.0, 5.0]])
    y, _, z, _ = R.adapted(q, s, x, a, b, np.array([1.0, 0.5]), [-1, 2], "f32")
    assert np.allclose(y, [[1.5, -2.0], [1.0, 0.0]])
    (dx, _), (da, _), (db, _) = R.backward(q, s, x, a, b, np.array([1.0, 0.5]), [1, -1], np.array([[1.0, 1.0], [1.0, 0.0]]), None, "f32")
    assert np.allclose(dx, [[0.5, -1.0 + 1.5], [0.5, 1.0]])
    assert not da[0].any() and np.allclose(da[1], [[0.5, 0.5]]) and np.allclose(db[1], [[1.5], [1.5]]) and not db[0].any()


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_reference_gradient_against_differences(act):
    rng = np.random.default_rng(7)
    T, N, K, Rk, n = 5, 6, 4, 2, 2
    q, s, x = rng.integers(-7, 8, (N, K)).astype(float), rng.uniform(0.1, 0.4, (N, 2)), rng.normal(0, 1, (T, K))
    a, b, sc = rng.normal(0, 0.5, (n, Rk, K)), rng.normal(0, 0.5, (n, N, Rk)), np.array([1.5, 0.7])
    ids = np.array([0, 1, -1, 1, 9])
    dy = rng.normal(0, 1, (T, N // 2 if act == "swiglu" else N))
    z = x @ R.weights(q, s).T + R.low_rank(x, a, b, sc, ids, False)[0]
    grads = [g for g, _ in R.backward(q, s, x, a, b, sc, ids, dy, z, "f32", act)]
    h = 1e-6
    for k, base in enumerate((x, a, b)):
        for i in np.ndindex(base.shape):
            keep, v = base[i], []
            for sg in (h, -h):
                base[i] = keep + sg
                v.append(R.value(q, s, x, a, b, sc, ids, dy, act))
            base[i] = keep
            assert abs((v[0] - v[1]) / (2 * h) - grads[k][i]) < 1e-7
