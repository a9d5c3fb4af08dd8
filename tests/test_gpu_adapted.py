"""moe_linear_adapted on the GPU against a plain 64-bit implementation (tests/tune_reference.py, which derives the bounds),
and bit for bit where every sum is a whole number that fp32 holds."""
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


def _call(cfg, codes, scales, ad, ids, x, bias=None, res=None, keep=False, dtype="f32"):
    T, out = x.shape[0], cfg.rows // 2 if cfg.act == ACT["swiglu"] else cfg.rows
    y, fy = H.guarded(T, out, dtype)
    z, fz = H.guarded(T, cfg.rows, dtype) if keep else (None, None)
    ws = H.space(moe.moe_linear_adapted_workspace_bytes(cfg, ad, T))
    moe.moe_linear_adapted(cfg, codes, scales, ad, ids, x, y, ws, bias=bias, residual=res, pre=z)
    torch.cuda.synchronize()
    assert H.untouched(fy, T, out) and (z is None or H.untouched(fz, T, cfg.rows))
    return y, z


# one to four tokens, few, and each way in which tiles of larger batches are cut
SHAPES = [(1, 64, 32, 8, 1), (1, 192, 96, 24, 3), (3, 320, 64, 16, 2), (16, 64, 160, 8, 5), (17, 448, 224, 40, 4),
          (32, 1024, 128, 128, 9), (300, 1088, 64, 16, 3), (129, 4160, 160, 24, 40), (191, 6080, 96, 64, 2),
          (600, 8128, 64, 8, 7), (1024, 16384, 64, 32, 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 32), (4, 64)])
@pytest.mark.parametrize("how", ["mix", "runs", "all"])
@pytest.mark.parametrize("T,N,K,Rk,n", SHAPES)
def test_whole_numbers_are_exact(T, N, K, Rk, n, how, bits, group, dtype):
    """Small whole numbers and scales of 1/2, 1 and 2: every sum is a multiple of 1/4 below 2^21, so any order of additions
    gives the same fp32 value; scale (A x) is a multiple of 1/2 below 2^12, which two bf16 parts hold."""
    K = (K + group - 1) // group * group if group else K
    rng = np.random.default_rng(T * 1000 + N + K)
    q, s, codes, scales = H.weights(rng, N, K, bits, group, whole=True)
    ad, a, b, sc = H.adapters(rng, n, Rk, N, K, dtype, whole=True)
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, whole=4)
    y, z = _call(moe.LinearConfig(N, K, bits, group), codes, scales, ad, ids, x, keep=True, dtype=dtype)
    rows = np.sort(rng.permutation(T)[:200])
    at = R.chosen(i, n, T)[rows]
    want = x64[rows] @ R.weights(q, s).T + R.low_rank(x64[rows], a, b, sc, at, False)[0]
    want = torch.from_numpy(want.astype(np.float32)).to(DT[dtype])
    assert torch.equal(y.cpu()[rows], want) and torch.equal(z.cpu()[rows], want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K,Rk,n,how", [(2000, 64, 96, 8, 1024, "mix"), (6000, 64, 64, 16, 3, "mix"), (2500, 640, 64, 24, 1024, "mix"),
                                            (500, 1024, 96, 8, 4, "mix"), (500, 1024, 96, 8, 5, "mix"), (70, 8192, 32, 128, 33, "mix"),
                                            (100, 64, 96, 64, 1, "all"), (700, 1088, 96, 40, 2, "all")])
def test_many_tokens_and_adapters_of_whole_numbers(T, N, K, Rk, n, how, dtype):
    """Few rows for many tokens, 1024 adapters, tokens with and without an order."""
    rng = np.random.default_rng(T + N)
    q, s, codes, scales = H.weights(rng, N, K, 4, 0, whole=True)
    ad, a, b, sc = H.adapters(rng, n, Rk, N, K, dtype, whole=True)
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, whole=4)
    y, _ = _call(moe.LinearConfig(N, K), codes, scales, ad, ids, x, dtype=dtype)
    rows = np.sort(rng.permutation(T)[:400])
    want = x64[rows] @ R.weights(q, s).T + R.low_rank(x64[rows], a, b, sc, R.chosen(i, n, T)[rows], False)[0]
    assert torch.equal(y.cpu()[rows], torch.from_numpy(want.astype(np.float32)).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("T,N,K,bits,group,Rk,n,how", [(1, 256, 544, 4, 0, 16, 4, "mix"), (5, 64, 256, 4, 32, 8, 2, "mix"),
                                                       (31, 192, 96, 8, 0, 24, 3, "runs"), (140, 4096, 320, 4, 64, 48, 5, "mix"),
                                                       (333, 2112, 160, 8, 0, 16, 3, "runs"), (200, 4096, 96, 4, 0, 128, 6, "one")])
def test_against_64_bits(T, N, K, bits, group, Rk, n, how, act, dtype):
    rng = np.random.default_rng(T + N + Rk)
    q, s, codes, scales = H.weights(rng, N, K, bits, group)
    ad, a, b, sc = H.adapters(rng, n, Rk, N, K, dtype)
    ids, i = H.ids_of(rng, T, n, how)
    x, x64 = H.matrix(rng, T, K, dtype, pad=5, shift=1)
    bias = rng.normal(0, 0.5, N).astype(np.float32)
    res, res64 = H.matrix(rng, T, N // 2 if act == "swiglu" else N, dtype, pad=1)
    y, z = _call(moe.LinearConfig(N, K, bits, group, ACT[act]), codes, scales, ad, ids, x, torch.from_numpy(bias).to(DEV), res,
                 True, dtype)
    rows = np.sort(rng.permutation(T)[:64])
    at = R.chosen(i, n, T)[rows]
    wy, ey, wz, ez = R.adapted(q, s, x64[rows], a, b, sc, at, dtype, act, bias.astype(np.float64), res64[rows])
    assert np.all(R.within(y.double().cpu().numpy()[rows], wy, ey, dtype))
    assert np.all(R.within(z.double().cpu().numpy()[rows], wz, ez, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K", [(1, 192, 96), (7, 320, 64), (33, 12352, 64), (300, 1088, 96)])
def test_without_adapters_it_is_the_product(T, N, K, dtype):
    """No adapters, and adapters that no token has: the bits of moe_linear."""
    rng = np.random.default_rng(T + N)
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    x, _ = H.matrix(rng, T, K, dtype)
    cfg = moe.LinearConfig(N, K, act=ACT["gelu"])
    y = torch.empty((T, N), dtype=DT[dtype], device=DEV)
    moe.moe_linear(cfg, codes, scales, x, y, H.space(moe.moe_linear_workspace_bytes(cfg, T)))
    ad = H.adapters(rng, 2, 8, N, K, dtype)[0]
    ids, _ = H.ids_of(rng, T, 2, "none")
    for a, i in ((None, None), (ad, ids)):
        assert torch.equal(_call(cfg, codes, scales, a, i, x, dtype=dtype)[0], y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K,how", [(3, 128, 64, "mix"), (32, 128, 64, "mix"), (300, 2048, 64, "mix"), (300, 2048, 64, "runs")])
def test_what_an_adapter_holds_stays_with_its_tokens(T, N, K, how, dtype):
    """One adapter of NaN and infinity, one token of NaN: the others' bits are those without them."""
    rng = np.random.default_rng(T)
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, 4, 16, N, K, dtype)
    ids, i = H.ids_of(rng, T, 4, how)
    i[T // 2] = 1
    ids.copy_(torch.from_numpy(i))
    x, _ = H.matrix(rng, T, K, dtype)
    cfg = moe.LinearConfig(N, K)
    clean, _ = _call(cfg, codes, scales, ad, ids, x, dtype=dtype)
    a, b, _ = ad._keep
    a[2, 3, 5] = float("inf")
    b[2, ::2] = float("nan")
    x[T // 2, 7] = float("nan")
    y, _ = _call(cfg, codes, scales, ad, ids, x, dtype=dtype)
    bad = (i == 2) | (np.arange(T) == T // 2)
    assert torch.equal(y[torch.from_numpy(~bad)], clean[torch.from_numpy(~bad)])
    assert bool((~torch.isfinite(y[torch.from_numpy(bad)])).all())


def test_a_residual_may_be_the_result():
    rng = np.random.default_rng(3)
    for T, N in ((4, 128), (200, 4096)):
        _, _, codes, scales = H.weights(rng, N, 64, 4, 0)
        ad, *_ = H.adapters(rng, 3, 8, N, 64, "bf16")
        ids, _ = H.ids_of(rng, T, 3, "mix")
        x, _ = H.matrix(rng, T, 64, "bf16")
        res, _ = H.matrix(rng, T, N, "bf16")
        cfg = moe.LinearConfig(N, 64)
        y, _ = _call(cfg, codes, scales, ad, ids, x, res=res, dtype="bf16")
        ws = H.space(moe.moe_linear_adapted_workspace_bytes(cfg, ad, T))
        moe.moe_linear_adapted(cfg, codes, scales, ad, ids, x, res, ws, residual=res)
        assert torch.equal(res, y)


@pytest.mark.parametrize("T,N", [(1, 192), (24, 192), (200, 4096)])
def test_captured_and_replayed_on_changing_inputs(T, N):
    """A captured call follows its inputs, ids included; several replays with eager work between them."""
    rng = np.random.default_rng(T)
    _, _, codes, scales = H.weights(rng, N, 96, 4, 0)
    ad, *_ = H.adapters(rng, 6, 16, N, 96, "bf16")
    cfg = moe.LinearConfig(N, 96, act=ACT["silu"])
    x, _ = H.matrix(rng, T, 96, "bf16")
    ids, _ = H.ids_of(rng, T, 6, "mix")
    y = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    ws = H.space(moe.moe_linear_adapted_workspace_bytes(cfg, ad, T))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        moe.moe_linear_adapted(cfg, codes, scales, ad, ids, x, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_linear_adapted(cfg, codes, scales, ad, ids, x, y, ws)
    for k in range(4):
        x.copy_(H.matrix(rng, T, 96, "bf16")[0])
        ids.copy_(H.ids_of(rng, T, 6, "mix" if k % 2 else "runs")[0])
        graph.replay()
        got = y.clone()
        want, _ = _call(cfg, codes, scales, ad, ids, x, dtype="bf16")
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [3, 70])
def test_rows_far_apart(T):
    """Rows whose offsets pass 2^31 elements, of the activations, the residual, the result and the values kept."""
    rng = np.random.default_rng(T)
    N, K = 8192, 64
    far = (1 << 31) // (T - 1) // 8 * 8 + 64
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, 2, 8, N, K, "bf16")
    ids, _ = H.ids_of(rng, T, 2, "mix")
    cfg = moe.LinearConfig(N, K, act=ACT["silu"])
    x, _ = H.matrix(rng, T, K, "bf16")
    res, _ = H.matrix(rng, T, N, "bf16")
    y, z = _call(cfg, codes, scales, ad, ids, x, res=res, keep=True, dtype="bf16")
    spread = [torch.empty((T - 1) * far + N, dtype=torch.bfloat16, device=DEV).as_strided((T, c), (far, 1)) for c in (K, N, N, N)]
    spread[0].copy_(x)
    spread[1].copy_(res)
    ws = H.space(moe.moe_linear_adapted_workspace_bytes(cfg, ad, T))
    moe.moe_linear_adapted(cfg, codes, scales, ad, ids, spread[0], spread[2], ws, residual=spread[1], pre=spread[3])
    assert torch.equal(spread[2], y) and torch.equal(spread[3], z)


def test_two_streams_with_a_workspace_each():
    rng = np.random.default_rng(5)
    T, N, K = 300, 4096, 128
    _, _, codes, scales = H.weights(rng, N, K, 4, 0)
    ad, *_ = H.adapters(rng, 5, 16, N, K, "bf16")
    cfg = moe.LinearConfig(N, K)
    xs = [H.matrix(rng, T, K, "bf16")[0] for _ in range(2)]
    ids = [H.ids_of(rng, T, 5, "mix")[0] for _ in range(2)]
    want = [_call(cfg, codes, scales, ad, ids[k], xs[k], dtype="bf16")[0] for k in range(2)]
    ys = [torch.empty((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ws = [H.space(moe.moe_linear_adapted_workspace_bytes(cfg, ad, T)) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k in range(2):
            moe.moe_linear_adapted(cfg, codes, scales, ad, ids[k], xs[k], ys[k], ws[k], stream=streams[k])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])


def test_binding_refuses_what_does_not_fit():
    rng = np.random.default_rng(0)
    _, _, codes, scales = H.weights(rng, 128, 64, 4, 0)
    cfg = moe.LinearConfig(128, 64)
    ad, *_ = H.adapters(rng, 2, 8, 128, 64, "bf16")
    x, y = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    ids, ws = torch.zeros(4, dtype=torch.int32, device=DEV), H.space(moe.moe_linear_adapted_workspace_bytes(cfg, ad, 4))
    moe.moe_linear_adapted(cfg, codes, scales, ad, ids, x, y, ws)
    for kw in (dict(ids=ids[:3]), dict(ids=ids.long()), dict(x=x.float(), y=y.float()), dict(y=y[:3]), dict(y=None),
               dict(pre=y.float()), dict(pre=y[:, :100]), dict(residual=y[:2]), dict(cfg=moe.LinearConfig(192, 64)),
               dict(codes=codes[:-1]), dict(scales=scales[:-1]), dict(bias=scales[:100])):
        args = dict(cfg=cfg, codes=codes, scales=scales, adapters=ad, ids=ids, x=x, y=y, ws=ws) | kw
        with pytest.raises(moe.ArgError):
            moe.moe_linear_adapted(**args)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_adapted(cfg, codes, scales, ad, ids, x, y, ws[:-1])
    a, b, s = ad._keep
    for bad in ((a, b[:1], s), (a, b.float(), s), (a, b, s[:1]), (a[0], b, s), (a.transpose(1, 2), b, s), (a, b, s.double())):
        with pytest.raises(moe.ArgError):
            moe.Adapters(*bad)


@pytest.mark.parametrize("T,n", [(4000, 2), (20000, 7), (20000, 64), (33000, 1024)])
def test_order_of_many_steps_that_share_adapters(T, n):
    """Every 64 tokens have adapters that the 64 before them had, found by other lanes: each count and position that a step
    leaves in shared memory is the next one's. Whole numbers, so every token's result says whether its position was right."""
    rng = np.random.default_rng(T + n)
    N, K, Rk = 64, 32, 8
    q, s, codes, scales = H.weights(rng, N, K, 4, 0, whole=True)
    ad, a, b, sc = H.adapters(rng, n, Rk, N, K, "bf16", whole=True)
    i = ((np.arange(T) * 5 + np.arange(T) // 64 * 3) % (n + 1)).astype(np.int32)  # n: no adapter
    x, x64 = H.matrix(rng, T, K, "bf16", whole=4)
    y, _ = _call(moe.LinearConfig(N, K), codes, scales, ad, torch.from_numpy(i).to(DEV), x, dtype="bf16")
    want = x64 @ R.weights(q, s).T + R.low_rank(x64, a, b, sc, i, False)[0]
    assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K,Rk,how", [(64, 64, 96, 128, "mix"), (300, 2048, 160, 16, "mix"), (700, 1088, 96, 40, "runs"),
                                          (1100, 4096, 64, 8, "mix"), (520, 128, 96, 8, "none")])
def test_one_adapter_that_some_tokens_have(T, N, K, Rk, how, dtype):
    """One adapter and ids with others beside it, which take no order: whole numbers, bit for bit; then an adapter of NaN and
    infinity, which the tokens without it do not see."""
    rng = np.random.default_rng(T + N)
    q, s, codes, scales = H.weights(rng, N, K, 4, 0, whole=True)
    ad, a, b, sc = H.adapters(rng, 1, Rk, N, K, dtype, whole=True)
    i = rng.choice([0, -1, 1, 2 ** 31 - 1], T) if how == "mix" else H.ids_of(rng, T, 1, how)[1]
    i = i.astype(np.int32)
    ids = torch.from_numpy(i).to(DEV)
    x, x64 = H.matrix(rng, T, K, dtype, whole=4)
    cfg = moe.LinearConfig(N, K)
    y, z = _call(cfg, codes, scales, ad, ids, x, keep=True, dtype=dtype)
    want = x64 @ R.weights(q, s).T + R.low_rank(x64, a, b, sc, i, False)[0]
    want = torch.from_numpy(want.astype(np.float32)).to(DT[dtype])
    assert torch.equal(y.cpu(), want) and torch.equal(z.cpu(), want)
    ta, tb, _ = ad._keep
    ta[0, 1, 3], tb[0, ::2] = float("inf"), float("nan")
    y, _ = _call(cfg, codes, scales, ad, ids, x, dtype=dtype)
    own = torch.from_numpy(i == 0)
    assert torch.equal(y.cpu()[~own], want[~own])
    assert bool((~torch.isfinite(y.cpu()[own])).all())
