"""moe_linear_backward on the GPU against a plain 64-bit implementation (tests/tune_reference.py, which derives the bounds),
bit for bit where every sum is a whole number, and in a training step of a gated block with adapters."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import int4_quantized_expert_amd as moe  # noqa: E402
from tests import tune_harness as H  # noqa: E402
from tests import tune_reference as R  # noqa: E402
from tests.tune_harness import ACT, DEV, DT  # noqa: E402


def _call(cfg, codes, scales, dy, ad=None, ids=None, x=None, z=None, res=None, dtype="f32", want=("dx", "da", "db")):
    T = dy.shape[0]
    dx, full = H.guarded(T, cfg.cols, dtype) if "dx" in want else (None, None)
    da, db = ((torch.full_like(t, float("nan")) if ad is not None and k in want else None)
              for k, t in zip(("da", "db"), ad._keep[:2] if ad is not None else (None, None)))
    ws = H.space(moe.moe_linear_backward_workspace_bytes(cfg, ad, T))
    moe.moe_linear_backward(cfg, codes, scales, dy, dx, ws, pre=z, adapters=ad, ids=ids, x=x, d_a=da, d_b=db, residual=res)
    torch.cuda.synchronize()
    assert dx is None or H.untouched(full, T, cfg.cols)
    return dx, da, db


SHAPES = [(1, 64, 32), (100, 64, 32), (2, 128, 2080), (5, 320, 96), (16, 64, 160), (31, 512, 64), (33, 576, 224), (64, 192, 544),
          (129, 320, 1088), (200, 1088, 4160), (300, 128, 8192), (191, 704, 6080), (600, 64, 8128), (1024, 64, 16384)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_whole_numbers_are_exact(T, N, K, bits, group, dtype):
    """Small whole gradients and scales of 1/2, 1 and 2: dz times a scale is exact in fp16, as is a code times what is left
    of a group scale, and every partial sum is a multiple of 1/2 below 2^22."""
    K = (K + group - 1) // group * group if group else K
    rng = np.random.default_rng(T * 1000 + N + K)
    q, s, codes, scales = H.weights(rng, N, K, bits, group, whole=True)
    dy, dy64 = H.matrix(rng, T, N, dtype, whole=8)
    dx, _, _ = _call(moe.LinearConfig(N, K, bits, group), codes, scales, dy, dtype=dtype)
    w = torch.from_numpy(R.weights(q, s)).to(DEV)
    want = torch.mm(torch.from_numpy(dy64).to(DEV), w)
    assert torch.equal(dx, want.float().to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K,bits,group,Rk,n,how", [(1, 64, 32, 4, 0, 8, 1, "all"), (3, 192, 96, 8, 0, 24, 2, "mix"),
                                                       (33, 320, 160, 4, 32, 16, 5, "mix"), (130, 704, 1088, 4, 0, 40, 3, "runs"),
                                                       (300, 1088, 544, 8, 0, 128, 2, "mix"), (300, 128, 4160, 4, 64, 32, 60, "mix"),
                                                       (777, 192, 256, 4, 0, 16, 2, "runs"), (600, 320, 96, 4, 0, 64, 3, "one")])
def test_adapters_of_whole_numbers_are_exact(T, N, K, bits, group, Rk, n, how, dtype):
    """Gradients and activations of -1, 0 and 1 and sparse adapters: scale (A x) and scale (B^T dz) are multiples of 1/2 with
    at most 15 bits, all sums multiples of 1/4 below 2^22."""
    rng = np.random.default_rng(T + N + K)
    q, s, codes, scales = H.weights(rng, N, K, bits, group, whole=True)
    a, b = (torch.from_numpy((rng.integers(-1, 2, sh) * (rng.random(sh) < 0.3)).astype(np.float32)).to(DT[dtype])
            for sh in ((n, Rk, K), (n, N, Rk)))
    sc = torch.from_numpy(rng.choice([0.5, 1.0, 2.0], n).astype(np.float32))
    ad = moe.Adapters(a.to(DEV), b.to(DEV), sc.to(DEV))
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, whole=1)
    dy, dy64 = H.matrix(rng, T, N, dtype, whole=1)
    got = _call(moe.LinearConfig(N, K, bits, group), codes, scales, dy, ad, ids, x, dtype=dtype)
    want = R.backward(q, s, x64, a.double().numpy(), b.double().numpy(), sc.double().numpy(), i, dy64, None, dtype)
    for g, (v, _) in zip(got, want):
        assert np.abs(v).max() < 2 ** 20
        assert torch.equal(g.cpu(), torch.from_numpy(v.astype(np.float32)).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("T,N,K,bits,group,Rk,n,how", [(1, 256, 544, 4, 0, 16, 4, "all"), (9, 64, 256, 4, 32, 8, 2, "mix"),
                                                       (40, 192, 96, 8, 0, 24, 3, "runs"), (140, 1024, 320, 4, 64, 48, 5, "mix"),
                                                       (310, 8256, 160, 4, 0, 16, 2, "runs")])
def test_against_64_bits(T, N, K, bits, group, Rk, n, how, act, dtype):
    rng = np.random.default_rng(T + N + Rk)
    q, s, codes, scales = H.weights(rng, N, K, bits, group)
    ad, a, b, sc = H.adapters(rng, n, Rk, N, K, dtype)
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, pad=5, shift=1)
    dy, dy64 = H.matrix(rng, T, N // 2 if act == "swiglu" else N, dtype, pad=1)
    z, z64 = H.matrix(rng, T, N, dtype, pad=8, shift=8, spread=False)
    z.mul_(2)
    z64 = 2 * z64
    res, res64 = H.matrix(rng, T, K, dtype, pad=3)
    got = _call(moe.LinearConfig(N, K, bits, group, ACT[act]), codes, scales, dy, ad, ids, x, z if act != "none" else None, res,
                dtype)
    want = R.backward(q, s, x64, a, b, sc, i, dy64, z64, dtype, act, res64)
    for name, g, (v, err) in zip(("dx", "da", "db"), got, want):
        ok = R.within(g.double().cpu().numpy(), v, err, dtype)
        assert ok.all(), (name, g.double().cpu().numpy()[~ok][:4], v[~ok][:4], err[~ok][:4])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K,Rk,n,how", [(64, 128, 288, 16, 70, "mix"), (65, 128, 288, 16, 70, "mix"), (64, 64, 96, 128, 1, "all"),
                                            (2500, 64, 224, 8, 1024, "mix"), (4500, 128, 96, 24, 3, "runs"), (300, 128, 32, 16, 2, "all"),
                                            (9000, 64, 160, 8, 2, "runs"), (1024, 64, 16384, 16, 2, "runs")])
def test_many_tokens_and_adapters_of_whole_numbers(T, N, K, Rk, n, how, dtype):
    """The borders between the forms for few and many tokens, adapters' sums in one run and in several, 1024 adapters."""
    rng = np.random.default_rng(T + N + K)
    q, s, codes, scales = H.weights(rng, N, K, 4, 0, whole=True)
    a, b = (torch.from_numpy((rng.integers(-1, 2, sh) * (rng.random(sh) < 0.2)).astype(np.float32)).to(DT[dtype])
            for sh in ((n, Rk, K), (n, N, Rk)))
    sc = torch.from_numpy(rng.choice([0.5, 1.0], n).astype(np.float32))
    ad = moe.Adapters(a.to(DEV), b.to(DEV), sc.to(DEV))
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, whole=1)
    dy, dy64 = H.matrix(rng, T, N, dtype, whole=1)
    got = _call(moe.LinearConfig(N, K), codes, scales, dy, ad, ids, x, dtype=dtype)
    want = R.backward(q, s, x64, a.double().numpy(), b.double().numpy(), sc.double().numpy(), i, dy64, None, dtype)
    for g, (v, _) in zip(got, want):
        assert np.abs(v).max() < 2 ** 20
        assert torch.equal(g.cpu(), torch.from_numpy(v.astype(np.float32)).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("group", [32, 64])
def test_group_scales_far_apart(group, T, dtype):
    """Scales of a row from 1 down to 2^-20 of it, rows of sizes from 2^-30 to 2^10, columns with small scales only."""
    rng = np.random.default_rng(T + group)
    N, K = 192, 256
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    s = 2.0 ** rng.uniform(-20, 0, (N, K // group)) * 2.0 ** rng.uniform(-30, 10, (N, 1))
    s[:, 1] = s.max(axis=1) * 2.0 ** -18
    s = s.astype(np.float32)
    u = (q & 15).astype(np.uint8)
    codes = torch.empty(N * K // 2, dtype=torch.uint8, device=DEV)
    moe.moe_tile_int4(torch.from_numpy(u[:, 0::2] | (u[:, 1::2] << 4)).to(DEV), codes)
    scales = torch.empty(s.size, device=DEV)
    moe.moe_tile_group_scales(torch.from_numpy(s).to(DEV), scales)
    dy, dy64 = H.matrix(rng, T, N, dtype)
    dx, _, _ = _call(moe.LinearConfig(N, K, 4, group), codes, scales, dy, dtype=dtype)
    (v, err), _, _ = R.backward(q.astype(np.float64), s.astype(np.float64), None, None, None, None, None, dy64, None, dtype)
    assert R.within(dx.double().cpu().numpy(), v, err, dtype).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -40, 2.0 ** 40])
def test_scales_far_from_one(size, T, dtype):
    """Row scales of 2^-110 leave the adapters' part as it is; others are exact powers of two of the same sums."""
    rng = np.random.default_rng(T)
    N, K, n = 128, 96, 2
    q, s, codes, scales = H.weights(rng, N, K, 4, 0, whole=True)
    scales.mul_(size)
    ad, a, b, sc = H.adapters(rng, n, 8, N, K, dtype)
    ids, i = H.ids_of(rng, T, n, "one")
    x, x64 = H.matrix(rng, T, K, dtype)
    dy, dy64 = H.matrix(rng, T, N, dtype)
    got = _call(moe.LinearConfig(N, K), codes, scales, dy, ad, ids, x, dtype=dtype)
    want = R.backward(q, s * size, x64, a, b, sc, i, dy64, None, dtype)
    for g, (v, err) in zip(got, want):
        assert R.within(g.double().cpu().numpy(), v, err, dtype).all()


@pytest.mark.parametrize("T", [3, 70])
def test_rows_far_apart(T):
    """Rows whose offsets pass 2^31 elements, of every matrix of the call."""
    rng = np.random.default_rng(T)
    N, K = 128, 96
    far = (1 << 31) // (T - 1) // 8 * 8 + 64
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, 2, 8, N, K, "bf16")
    ids, _ = H.ids_of(rng, T, 2, "mix")
    cfg = moe.LinearConfig(N, K, act=ACT["silu"])
    x, _ = H.matrix(rng, T, K, "bf16")
    z, _ = H.matrix(rng, T, N, "bf16", spread=False)
    dy, _ = H.matrix(rng, T, N, "bf16")
    want = _call(cfg, codes, scales, dy, ad, ids, x, z, x, dtype="bf16")
    sx, sz, sdy, sdx = (torch.empty((T - 1) * far + N, dtype=torch.bfloat16, device=DEV).as_strided((T, c), (far, 1))
                        for c in (K, N, N, K))
    for to, of in ((sx, x), (sz, z), (sdy, dy)):
        to.copy_(of)
    da, db = torch.empty_like(ad._keep[0]), torch.empty_like(ad._keep[1])
    ws = H.space(moe.moe_linear_backward_workspace_bytes(cfg, ad, T))
    moe.moe_linear_backward(cfg, codes, scales, sdy, sdx, ws, pre=sz, adapters=ad, ids=ids, x=sx, d_a=da, d_b=db, residual=sx)
    assert all(torch.equal(p, q) for p, q in zip((sdx, da, db), want))


def test_two_streams_with_a_workspace_each():
    rng = np.random.default_rng(8)
    T, N, K, n = 300, 256, 192, 3
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, n, 16, N, K, "bf16")
    cfg = moe.LinearConfig(N, K)
    x = [H.matrix(rng, T, K, "bf16")[0] for _ in range(2)]
    dy = [H.matrix(rng, T, N, "bf16")[0] for _ in range(2)]
    ids = [H.ids_of(rng, T, n, "mix")[0] for _ in range(2)]
    want = [_call(cfg, codes, scales, dy[k], ad, ids[k], x[k], dtype="bf16") for k in range(2)]
    got = [[torch.empty_like(t) for t in want[k]] for k in range(2)]
    ws = [H.space(moe.moe_linear_backward_workspace_bytes(cfg, ad, T)) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k in range(2):
            moe.moe_linear_backward(cfg, codes, scales, dy[k], got[k][0], ws[k], adapters=ad, ids=ids[k], x=x[k],
                                    d_a=got[k][1], d_b=got[k][2], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(p, q) for p, q in zip(got[k], want[k]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_alone_and_equal_calls(dtype):
    """Each gradient alone is what all of them together give, and a call gives the same bits again."""
    rng = np.random.default_rng(9)
    T, N, K = 700, 448, 288
    _, _, codes, scales = H.weights(rng, N, K, 4, 32)
    ad, *_ = H.adapters(rng, 3, 16, N, K, dtype)
    ids, _ = H.ids_of(rng, T, 3, "runs")
    x, _ = H.matrix(rng, T, K, dtype)
    z, _ = H.matrix(rng, T, N, dtype, spread=False)
    for act in ("none", "swiglu"):
        dy, _ = H.matrix(rng, T, N // 2 if act == "swiglu" else N, dtype)
        cfg, zz = moe.LinearConfig(N, K, 4, 32, ACT[act]), z if act != "none" else None
        every = _call(cfg, codes, scales, dy, ad, ids, x, zz, dtype=dtype)
        again = _call(cfg, codes, scales, dy, ad, ids, x, zz, dtype=dtype)
        assert all(torch.equal(p, q) for p, q in zip(every, again))
        for k, name in enumerate(("dx", "da", "db")):
            one = _call(cfg, codes, scales, dy, ad, ids, None if name == "dx" else x, zz, dtype=dtype, want=(name,))
            assert torch.equal(one[k], every[k])
        # gradients of another projection of the same x are added in place
        acc = torch.full((T, K), 0.5, dtype=DT[dtype], device=DEV)
        ws = H.space(moe.moe_linear_backward_workspace_bytes(cfg, ad, T))
        moe.moe_linear_backward(cfg, codes, scales, dy, acc, ws, pre=zz, adapters=ad, ids=ids, residual=acc)
        half = torch.full((T, K), 0.5, dtype=DT[dtype], device=DEV)
        assert torch.equal(acc, _call(cfg, codes, scales, dy, ad, ids, None, zz, half, dtype, ("dx",))[0])


@pytest.mark.parametrize("how", ["none", "one", "mix"])
def test_adapters_without_tokens_get_zeros(how):
    rng = np.random.default_rng(2)
    T, N, K, n = 50, 128, 96, 300
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, n, 8, N, K, "bf16")
    ids, i = H.ids_of(rng, T, n, how)
    x, _ = H.matrix(rng, T, K, "bf16")
    dy, _ = H.matrix(rng, T, N, "bf16")
    _, da, db = _call(moe.LinearConfig(N, K), codes, scales, dy, ad, ids, x, dtype="bf16")
    have = np.zeros(n, bool)
    have[R.chosen(i, n, T)[R.chosen(i, n, T) >= 0]] = True
    for g in (da, db):
        flat = g.view(n, -1).float().cpu()
        assert not bool(flat[torch.from_numpy(~have)].any())
        assert bool((flat[torch.from_numpy(have)] != 0).any(dim=1).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_no_number_stays_with_its_token_and_adapter(dtype):
    rng = np.random.default_rng(6)
    T, N, K = 300, 320, 160
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, 4, 16, N, K, dtype)
    ids, i = H.ids_of(rng, T, 4, "mix")
    i[:2] = 1, -1
    ids.copy_(torch.from_numpy(i))
    x, _ = H.matrix(rng, T, K, dtype)
    dy, _ = H.matrix(rng, T, N, dtype)
    cfg = moe.LinearConfig(N, K)
    clean = _call(cfg, codes, scales, dy, ad, ids, x, dtype=dtype)
    dy[0, 5], dy[1, 9] = float("nan"), float("inf")  # tokens of adapter 1 and of none
    a, b, _ = ad._keep
    b[2, 7] = float("nan")
    got = _call(cfg, codes, scales, dy, ad, ids, x, dtype=dtype)
    bad = (i == 2)
    bad[:2] = True
    assert torch.equal(got[0][torch.from_numpy(~bad)], clean[0][torch.from_numpy(~bad)])
    assert bool((~torch.isfinite(got[0][torch.from_numpy(bad)])).all())
    for k in (1, 2):
        for e in (0, 3):
            assert torch.equal(got[k][e], clean[k][e])
        assert not bool(torch.isfinite(got[k][1]).all())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "swiglu"])
def test_limits_of_the_derivatives(act):
    """Pre-activations from very far below to very far above: the derivative's limits, no NaN from an infinity times 0."""
    far = [-math.inf, -3e38, -1e20, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e20, 3e38, math.inf]
    N, K = 64, 64
    z = torch.zeros((len(far), 64), device=DEV)
    z[:, 0] = torch.tensor(far, device=DEV)
    if act == "swiglu":
        z[:, 32:] = 1.0
    rng = np.random.default_rng(0)
    q, s, codes, scales = H.weights(rng, N, K, 8, 0, whole=True)
    dy = torch.zeros((len(far), N // 2 if act == "swiglu" else N), device=DEV)
    dy[:, 0] = 1.0
    up = act == "swiglu"
    dx, _, _ = _call(moe.LinearConfig(N, K, 8, 0, ACT[act]), codes, scales, dy, z=z)
    w = R.weights(q, s)
    for t, v in enumerate(far):
        g = min(max(v, -1e4), 1e4)
        d = R.slope(np.array([[g]]), "silu" if up else act)[0, 0]
        want = d * w[0]
        if up and v < 1e30:  # beyond, silu(gate) of the up row is all that counts
            want = want + max(v, -1e4) * R._sig(g) * w[32]
        elif up:
            assert bool(torch.isinf(dx[t]).any()) if math.isinf(v) else bool(torch.isfinite(dx[t] / 3e38).any())
            continue
        size = abs(d) * np.abs(w[0]) + (abs(max(v, -1e4) * R._sig(g)) * np.abs(w[32]) if up else 0.0)
        assert np.all(np.abs(dx[t].double().cpu().numpy() - want) <= 2.0 ** -19 * size + 1e-30), v


@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_and_replayed_on_changing_inputs(T):
    rng = np.random.default_rng(T)
    N, K, n = 192, 96, 5
    _, _, codes, scales = H.weights(rng, N, K, 4, 32)
    ad, *_ = H.adapters(rng, n, 16, N, K, "bf16")
    cfg = moe.LinearConfig(N, K, 4, 32, ACT["swiglu"])
    x, _ = H.matrix(rng, T, K, "bf16")
    z, _ = H.matrix(rng, T, N, "bf16", spread=False)
    dy, _ = H.matrix(rng, T, N // 2, "bf16")
    ids, _ = H.ids_of(rng, T, n, "mix")
    dx = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    da, db = torch.empty_like(ad._keep[0]), torch.empty_like(ad._keep[1])
    ws = H.space(moe.moe_linear_backward_workspace_bytes(cfg, ad, T))

    def step():
        moe.moe_linear_backward(cfg, codes, scales, dy, dx, ws, pre=z, adapters=ad, ids=ids, x=x, d_a=da, d_b=db)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(H.matrix(rng, T, K, "bf16")[0])
        dy.copy_(H.matrix(rng, T, N // 2, "bf16")[0])
        ids.copy_(H.ids_of(rng, T, n, "mix" if k % 2 else "runs")[0])
        graph.replay()
        got = [t.clone() for t in (dx, da, db)]
        want = _call(cfg, codes, scales, dy, ad, ids, x, z, dtype="bf16")
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_binding_refuses_what_does_not_fit():
    rng = np.random.default_rng(0)
    _, _, codes, scales = H.weights(rng, 128, 64, 4, 0)
    cfg = moe.LinearConfig(128, 64, act=ACT["silu"])
    ad, *_ = H.adapters(rng, 2, 8, 128, 64, "bf16")
    x, dy = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    z, dx, ids = dy.clone(), x.clone(), torch.zeros(4, dtype=torch.int32, device=DEV)
    da, db = torch.empty_like(ad._keep[0]), torch.empty_like(ad._keep[1])
    ws = H.space(moe.moe_linear_backward_workspace_bytes(cfg, ad, 4))
    ok = dict(cfg=cfg, codes=codes, scales=scales, dy=dy, dx=dx, ws=ws, pre=z, adapters=ad, ids=ids, x=x, d_a=da, d_b=db)
    moe.moe_linear_backward(**ok)
    for kw in (dict(adapters=None), dict(d_a=da.float()), dict(d_b=db[:1]), dict(dx=dx[:3]), dict(dx=dx.float()),
               dict(pre=z[:, :64]), dict(x=x[:2]), dict(ids=ids[:1]), dict(residual=z), dict(dy=dy[:, :64])):
        with pytest.raises(moe.ArgError):
            moe.moe_linear_backward(**(ok | kw))
    for kw in (dict(pre=None), dict(x=None), dict(ws=ws[:-1]), dict(dx=None, d_a=None, d_b=None), dict(dx=None, residual=dx)):
        with pytest.raises(moe.MoeError):
            moe.moe_linear_backward(**(ok | kw))


def test_a_training_step_of_a_gated_block():
    """Gate and up rows with SwiGLU, down rows into the residual stream, adapters on both, their gradients and the clipping of
    all of them, against the same in 64 bits by automatic differentiation. bf16 between the products: each of the four
    roundings on the way to a gradient (h, z, dh, the gradient) is 2^-8 of a value at most, about 2^-9.6 in the mean
    square, so the 2-norm of a difference stays below 2^-7 of the gradient's."""
    rng = np.random.default_rng(11)
    T, D, F, n, Rk = 150, 256, 320, 3, 16
    q1, s1, c1, t1 = H.weights(rng, 2 * F, D, 4, 0)
    q2, s2, c2, t2 = H.weights(rng, D, F, 4, 32)
    ad1, a1, b1, k1 = H.adapters(rng, n, Rk, 2 * F, D, "bf16")
    ad2, a2, b2, k2 = H.adapters(rng, n, Rk, D, F, "bf16")
    ids, i = H.ids_of(rng, T, n, "mix")
    x, x64 = H.matrix(rng, T, D, "bf16", spread=False)
    dy, dy64 = H.matrix(rng, T, D, "bf16", spread=False)
    up, down = moe.LinearConfig(2 * F, D, act=ACT["swiglu"]), moe.LinearConfig(D, F, 4, 32)
    new = lambda *sh: torch.empty(sh, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    h, z, y, dh, dx = new(T, F), new(T, 2 * F), new(T, D), new(T, F), new(T, D)
    grads = [torch.empty_like(t) for ad in (ad1, ad2) for t in ad._keep[:2]]
    ws = H.space(max(moe.moe_linear_adapted_workspace_bytes(up, ad1, T), moe.moe_linear_adapted_workspace_bytes(down, ad2, T),
                     moe.moe_linear_backward_workspace_bytes(up, ad1, T), moe.moe_linear_backward_workspace_bytes(down, ad2, T)))
    table, norm = moe.GradTable(grads), torch.zeros(1, device=DEV)

    def step(limit):
        moe.moe_linear_adapted(up, c1, t1, ad1, ids, x, h, ws, pre=z)
        moe.moe_linear_adapted(down, c2, t2, ad2, ids, h, y, ws, residual=x)
        moe.moe_linear_backward(down, c2, t2, dy, dh, ws, adapters=ad2, ids=ids, x=h, d_a=grads[2], d_b=grads[3])
        moe.moe_linear_backward(up, c1, t1, dh, dx, ws, pre=z, adapters=ad1, ids=ids, x=x, d_a=grads[0], d_b=grads[1],
                                residual=dy)
        moe.moe_grad_clip(table, limit, norm)

    step(math.inf)
    torch.cuda.synchronize()
    leaves = [torch.from_numpy(v).requires_grad_(True) for v in (a1, b1, a2, b2, x64)]

    def product(v, q, s, a, b, k):
        r = v @ torch.from_numpy(R.weights(q, s)).t()
        at = torch.from_numpy(R.chosen(i, n, T))
        for e in range(n):
            m = (at == e).double()[:, None]
            r = r + m * k[e] * ((v @ a[e].t()) @ b[e].t())
        return r

    zz = product(leaves[4], q1, s1, leaves[0], leaves[1], k1)
    hh = torch.nn.functional.silu(zz[:, :F]) * zz[:, F:]
    yy = leaves[4] + product(hh, q2, s2, leaves[2], leaves[3], k2)
    want = torch.autograd.grad(yy, leaves, torch.from_numpy(dy64))
    close = lambda g, w: float((g.double().cpu() - w).norm() / w.norm()) < 2.0 ** -7  # noqa: E731
    assert close(y, yy.detach())
    for g, w in zip((*grads, dx), want):
        assert close(g, w)
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    assert abs(float(norm) - total) <= 2.0 ** -22 * total
    before = [g.clone() for g in grads]
    step(0.5 * total)
    for g, b in zip(grads, before):
        assert bool(((g.double() - 0.5 * b.double()).abs() <= (2.0 ** -8 + 2.0 ** -22) * b.double().abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [3, 100, 1100])
@pytest.mark.parametrize("size", [3e-3, 1e-5, 1e-8])
@pytest.mark.parametrize("group", [32, 64])
def test_rows_whose_group_scales_are_zero(group, size, T, dtype):
    """A quarter of the rows, as padding and pruning leave them, and single groups of live rows: what their codes hold and
    how large their dz is changes nothing, however small the live rows' scales are."""
    rng = np.random.default_rng(T + group)
    N, K = 256, 256
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    s = (size * rng.uniform(0.3, 1.0, (N, K // group))).astype(np.float32)
    dead = rng.permutation(N)[: N // 4]
    s[dead] = 0.0
    s[np.setdiff1d(np.arange(N), dead)[::5], 1] = 0.0
    u = (q & 15).astype(np.uint8)
    codes = torch.empty(N * K // 2, dtype=torch.uint8, device=DEV)
    moe.moe_tile_int4(torch.from_numpy(u[:, 0::2] | (u[:, 1::2] << 4)).to(DEV), codes)
    scales = torch.empty(s.size, device=DEV)
    moe.moe_tile_group_scales(torch.from_numpy(s).to(DEV), scales)
    dy, dy64 = H.matrix(rng, T, N, dtype, spread=False)
    dy.mul_(1024)  # fp16 results stay above its smallest
    dx, _, _ = _call(moe.LinearConfig(N, K, 4, group), codes, scales, dy, dtype=dtype)
    rows = np.sort(rng.permutation(T)[:64])
    (v, err), _, _ = R.backward(q.astype(np.float64), s.astype(np.float64), None, None, None, None, None, 1024 * dy64[rows], None,
                                dtype)
    assert R.within(dx.double().cpu().numpy()[rows], v, err, dtype).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -141])
def test_group_scales_below_the_normal_range(size, T, dtype):
    """Rows whose largest group scale is a subnormal, with gradients that make up for it."""
    rng = np.random.default_rng(T)
    N, K, group = 128, 128, 32
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    s = (size * rng.uniform(0.25, 1.0, (N, K // group))).astype(np.float32)
    u = (q & 15).astype(np.uint8)
    codes = torch.empty(N * K // 2, dtype=torch.uint8, device=DEV)
    moe.moe_tile_int4(torch.from_numpy(u[:, 0::2] | (u[:, 1::2] << 4)).to(DEV), codes)
    scales = torch.empty(s.size, device=DEV)
    moe.moe_tile_group_scales(torch.from_numpy(s).to(DEV), scales)
    dy, dy64 = H.matrix(rng, T, N, dtype, spread=False)
    dy.mul_(2.0 ** 100)
    dx, _, _ = _call(moe.LinearConfig(N, K, 4, group), codes, scales, dy, dtype=dtype)
    (v, err), _, _ = R.backward(q.astype(np.float64), s.astype(np.float64), None, None, None, None, None, 2.0 ** 100 * dy64, None, dtype)
    assert R.within(dx.double().cpu().numpy(), v, err, dtype).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 100])
def test_a_large_gradient_times_a_large_up_part_of_a_closed_gate(T, dtype):
    """dy up is beyond fp32, its product with the gate's derivative is not."""
    rng = np.random.default_rng(T)
    N, K = 128, 64
    q, s, codes, scales = H.weights(rng, N, K, 8, 0)
    dy, z = rng.uniform(0.5, 1.0, (T, N // 2)) * 2.0 ** 84, np.empty((T, N))
    z[:, : N // 2], z[:, N // 2:] = rng.uniform(-40.0, -30.0, (T, N // 2)), rng.uniform(0.5, 1.0, (T, N // 2)) * 2.0 ** 68
    dy, z = (torch.from_numpy(v.astype(np.float32)).to(DT[dtype]) for v in (dy, z))
    dx, _, _ = _call(moe.LinearConfig(N, K, 8, 0, ACT["swiglu"]), codes, scales, dy.to(DEV), z=z.to(DEV), dtype=dtype)
    dy64, z64 = dy.double().numpy(), z.double().numpy()
    dz, _ = R.grad_in(dy64, z64, "swiglu")
    # exp in fp32 at 40 is off by 40 2^-24 of it beside the roundings; the derivative is (1 + gate) exp(gate) there
    size = np.abs(dz) * 128 * R.UNIT
    (v, err), _, _ = R.backward(q, s, None, None, None, None, None, dz, None, dtype)
    assert R.within(dx.double().cpu().numpy(), v, err + size @ np.abs(R.weights(q, s)), dtype).all()


def _unrounded(q, s, x64, a, b, sc, i, dy64, z64, dtype, act):
    """R.backward's results and bounds for adapters' sums over dz as it is: a few fp32 roundings of the derivative, none to the
    type."""
    dz, size = R.grad_in(dy64, z64, act)
    dx, (da, ea), (db, eb) = R.backward(q, s, x64, a, b, sc, i, dz, None, dtype)
    ez = 32 * R.UNIT * size
    ex = dx[1] + ez @ np.abs(R.weights(q, s))
    at = R.chosen(i, a.shape[0], dy64.shape[0])
    for e in np.unique(at[at >= 0]):
        t = np.nonzero(at == e)[0]
        eu = ez[t] @ np.abs(b[e]) * abs(sc[e])
        ea[e] += eu.T @ np.abs(x64[t])
        eb[e] += ez[t].T @ np.abs(x64[t] @ a[e].T * sc[e])
        ex[t] += eu @ np.abs(a[e])
    return (dx[0], ex), (da, ea), (db, eb)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("T,N,K,Rk,n,how", [(5, 256, 96, 16, 2, "mix"), (40, 128, 160, 8, 3, "mix"), (64, 192, 64, 128, 2, "one"),
                                            (300, 448, 288, 16, 3, "runs"), (700, 320, 96, 40, 2, "one"), (2100, 128, 64, 24, 5, "mix")])
def test_adapters_gradients_are_rounded_once(T, N, K, Rk, n, how, act, dtype):
    """Between the activation's derivative and the adapters' sums nothing is rounded to the type: each gradient is off by its
    own rounding and by what fp32 sums and 16 bits of scale (A x) and scale (B^T dz) leave."""
    rng = np.random.default_rng(T + N + Rk)
    q, s, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, a, b, sc = H.adapters(rng, n, Rk, N, K, dtype)
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, pad=3)
    dy, dy64 = H.matrix(rng, T, N // 2 if act == "swiglu" else N, dtype, pad=1)
    z, z64 = H.matrix(rng, T, N, dtype, pad=8, spread=False)
    got = _call(moe.LinearConfig(N, K, 4, 0, ACT[act]), codes, scales, dy, ad, ids, x, z, dtype=dtype)
    want = _unrounded(q, s, x64, a, b, sc, i, dy64, z64, dtype, act)
    for name, g, (v, err) in zip(("dx", "da", "db"), got, want):
        assert R.within(g.double().cpu().numpy(), v, err, dtype).all(), name


@pytest.mark.parametrize("T", [3, 40, 300, 1100])
@pytest.mark.parametrize("big", [True, False])
def test_half_precision_dz_outside_its_range(big, T):
    """fp16 calls whose dz is beyond 65504, or below 2^-24: with adapters dx is finite as it is without, and the gradients are
    the formula's."""
    rng = np.random.default_rng(T)
    N, K, n, Rk = 128, 96, 3, 8
    half = lambda v: torch.from_numpy(v.astype(np.float32)).half()  # noqa: E731
    q, s, codes, scales = H.weights(rng, N, K, 4, 0)
    a, b = rng.normal(0, 1 / np.sqrt(K), (n, Rk, K)), rng.normal(0, 1e-4 if big else 1.0, (n, N, Rk))
    x, dy, z = rng.normal(0, 1e-3 if big else 1e4, (T, K)), rng.normal(0, 500 if big else 3e-6, (T, N // 2)), rng.normal(0, 1, (T, N))
    z[:, N // 2:] *= 500 if big else 3e-3
    z[:, : N // 2] += 2 if big else -5
    a, b, x, dy, z = (half(v) for v in (a, b, x, dy, z))
    sc = torch.from_numpy(rng.uniform(0.5, 2.0, n).astype(np.float32))
    scale = 2.0 ** (-10 if big else 10)
    scales.mul_(scale)
    ad = moe.Adapters(a.to(DEV), b.to(DEV), sc.to(DEV))
    ids, i = H.ids_of(rng, T, n, "mix")
    i[0] = 0
    ids.copy_(torch.from_numpy(i))
    args = (moe.LinearConfig(N, K, 4, 0, ACT["swiglu"]), codes, scales, dy.to(DEV))
    f64 = [t.double().numpy() for t in (x, a, b, sc, dy, z)]
    dz = np.abs(R.grad_in(f64[4], f64[5], "swiglu")[0])
    assert dz.max() > 2 * 65504 if big else np.median(dz) < 2.0 ** -24
    alone = _call(*args, z=z.to(DEV), dtype="f16")[0]
    got = _call(*args, ad, ids, x.to(DEV), z.to(DEV), dtype="f16")
    want = _unrounded(q, s * scale, *f64[:4], i, *f64[4:], "f16", "swiglu")
    assert all(bool(torch.isfinite(t).all()) for t in (alone, *got))
    for name, g, (v, err) in zip(("dx", "da", "db"), got, want):
        assert np.abs(v).max() > 2.0 ** -16
        assert R.within(g.double().cpu().numpy(), v, err, "f16").all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("T", [3, 33, 64, 300, 1100])
def test_no_number_reaches_another_token_or_adapter(T, group, act, dtype):
    """NaN and infinity in dy, in x and in an adapter, for few tokens and for many: other tokens' dx and other adapters'
    gradients keep their bits; so do d_b's rows of an adapter whose token has an infinity in another row of dz."""
    rng = np.random.default_rng(T)
    N, K = 320, 160
    _, _, codes, scales = H.weights(rng, N, K, 4, group)
    ad, *_ = H.adapters(rng, 5, 16, N, K, dtype)
    _, i = H.ids_of(rng, T, 5, "mix")
    i[:3] = 1, -1, 3
    ids = torch.from_numpy(i).to(DEV)
    x, _ = H.matrix(rng, T, K, dtype)
    dy, _ = H.matrix(rng, T, N // 2 if act == "swiglu" else N, dtype)
    z, _ = H.matrix(rng, T, N, dtype, spread=False)
    z = z.abs_().add_(0.5) if act != "none" else None  # no derivative of zero beside an infinity
    cfg = moe.LinearConfig(N, K, 4, group, ACT[act])
    clean = _call(cfg, codes, scales, dy, ad, ids, x, z, dtype=dtype)
    dy[0, 5], dy[1, 9] = float("inf"), float("nan")  # tokens of adapter 1 and of none
    x[2, 7] = float("nan")                           # a token of adapter 3: in its d_a and, by A x, its d_b
    ad._keep[1][2, 7] = float("nan")
    got = _call(cfg, codes, scales, dy, ad, ids, x, z, dtype=dtype)
    bad = i == 2
    bad[:2] = True
    ok = torch.from_numpy(~bad)
    assert torch.equal(got[0].cpu()[ok], clean[0].cpu()[ok])
    assert bool((~torch.isfinite(got[0].cpu()[~ok])).all())
    for k in (1, 2):
        for e in (0, 4):
            assert torch.equal(got[k][e], clean[k][e])
        for e in (1, 3):
            assert not bool(torch.isfinite(got[k][e]).all())
    rows = [r for r in range(N) if r != 5 and not (act == "swiglu" and r == 5 + N // 2)]
    assert torch.equal(got[2][1][rows], clean[2][1][rows])
    assert torch.equal(got[1][3][:, :7], clean[1][3][:, :7]) and torch.equal(got[1][3][:, 8:], clean[1][3][:, 8:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 80])
def test_a_gate_near_the_largest_number(T, dtype):
    """An open gate of 3e38: its derivative is 1, and silu(gate) is the gate; the results go beyond fp32 where W takes them."""
    N, K = 64, 64
    rng = np.random.default_rng(3)
    q, s, codes, scales = H.weights(rng, N, K, 8, 0, whole=True)
    z = torch.zeros((T, N), device=DEV)
    z[:, 0], z[:, 32:] = 3e38, 1.0
    z = z.to(DT[dtype])
    dy = torch.zeros((T, N // 2), dtype=DT[dtype], device=DEV)
    dy[:, 0] = 2.0 ** -5
    dx, _, _ = _call(moe.LinearConfig(N, K, 8, 0, ACT["swiglu"]), codes, scales, dy, z=z, dtype=dtype)
    w = R.weights(q, s)
    gate = float(z[0, 0].double())
    want = 2.0 ** -5 * (w[0] + gate * w[32])
    top, got = float(torch.finfo(DT[dtype]).max), dx.double().cpu().numpy()
    assert (np.abs(want) > 1.01 * top).any() and (np.abs(want) < 0.99 * top).any()
    near = np.abs(np.abs(want) / top - 1.0) < 0.01  # either is right next to the border
    for t in range(T):
        far = np.abs(want) > top
        assert np.array_equal(got[t][far & ~near], np.sign(want[far & ~near]) * math.inf)
        fin = ~far & ~near
        # one rounding to fp16 of dz, in two halves for fp32, and one to the type
        step = 2.0 ** -21 if dtype == "f32" else 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -19
        low = 2.0 ** -38 * 2.0 * gate * (np.abs(q[0]) + np.abs(q[32]))  # of the token's largest dz times scale
        assert np.all(np.abs(got[t] - want)[fin] <= (2.0 ** -5 * (step * (np.abs(gate * w[32]) + np.abs(w[0])) + low))[fin])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 100])
def test_a_small_gradient_times_a_large_up_part_of_a_closed_gate(T, dtype):
    """dy times the gate's derivative is below fp32's normal range, dy up times it is not."""
    rng = np.random.default_rng(T)
    N, K = 128, 64
    q, s, codes, scales = H.weights(rng, N, K, 8, 0)
    dy, z = rng.uniform(0.5, 1.0, (T, N // 2)) * 2.0 ** -96, np.empty((T, N))
    z[:, : N // 2], z[:, N // 2:] = rng.uniform(-40.0, -30.0, (T, N // 2)), rng.uniform(0.5, 1.0, (T, N // 2)) * 2.0 ** 68
    dy, z = (torch.from_numpy(v.astype(np.float32)).to(DT[dtype]) for v in (dy, z))
    dx, _, _ = _call(moe.LinearConfig(N, K, 8, 0, ACT["swiglu"]), codes, scales, dy.to(DEV), z=z.to(DEV), dtype=dtype)
    dz, _ = R.grad_in(dy.double().numpy(), z.double().numpy(), "swiglu")
    size = np.abs(dz) * 128 * R.UNIT  # as above
    (v, err), _, _ = R.backward(q, s, None, None, None, None, None, dz, None, dtype)
    assert R.within(dx.double().cpu().numpy(), v, err + size @ np.abs(R.weights(q, s)), dtype).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("how", ["none", "one", "mix"])
@pytest.mark.parametrize("T,n,Rk", [(40, 70, 40), (300, 90, 8), (300, 3, 40)])
def test_adapters_without_tokens_get_zeros_behind_an_activation(T, n, Rk, how, dtype):
    rng = np.random.default_rng(T + n)
    N, K = 192, 160
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, n, Rk, N, K, dtype)
    ids, i = H.ids_of(rng, T, n, how)
    x, _ = H.matrix(rng, T, K, dtype)
    dy, _ = H.matrix(rng, T, N // 2, dtype)
    z, _ = H.matrix(rng, T, N, dtype, spread=False)
    _, da, db = _call(moe.LinearConfig(N, K, act=ACT["swiglu"]), codes, scales, dy, ad, ids, x, z, dtype=dtype)
    at = R.chosen(i, n, T)
    have = torch.zeros(n, dtype=torch.bool)
    have[torch.from_numpy(at[at >= 0])] = True
    for g in (da, db):
        flat = g.view(n, -1).float().cpu()
        assert not bool(flat[~have].any()) and bool((flat[have] != 0).any(dim=1).all())
