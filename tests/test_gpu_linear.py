"""moe_linear on the GPU against a plain 64-bit implementation (tests/ops_reference.py, which derives the bound), and
bit for bit where every sum is a whole number that fp32 holds."""
import numpy as np
import pytest

from tests import ops_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import int4_quantized_expert_amd as moe  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACT = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
       "gelu_tanh": moe.MOE_ACT_GELU_TANH, "swiglu": moe.MOE_ACT_SWIGLU}


def _weights(rng, N, K, bits, group, whole=False):
    """Codes over their whole range, scales, and both on the device in the tiled layouts."""
    lim = 8 if bits == 4 else 128
    q = rng.integers(-lim, lim, (N, K)).astype(np.int8)
    G = group or K
    s = rng.choice([0.5, 1.0, 2.0], (N, K // G)) if whole else rng.uniform(0.2, 1.0, (N, K // G)) / (lim * np.sqrt(K))
    s = s.astype(np.float32)
    if bits == 4:
        u = (q & 15).astype(np.uint8)
        row = torch.from_numpy(u[:, 0::2] | (u[:, 1::2] << 4)).to(DEV)
    else:
        row = torch.from_numpy(q).to(DEV)
    codes = torch.empty(row.numel(), dtype=torch.uint8, device=DEV)
    (moe.moe_tile_int4 if bits == 4 else moe.moe_tile_int8)(row, codes)
    sc = torch.from_numpy(s).to(DEV)
    scales = sc.view(-1)
    if group:
        scales = torch.empty_like(scales)
        moe.moe_tile_group_scales(sc, scales)
    return q.astype(np.float64), s.astype(np.float64), codes, scales


def _call(cfg, codes, scales, x, out, bias=None, res=None, y=None):
    T = x.shape[0]
    y = torch.full((T + 1, out + 3), 9.0, dtype=x.dtype, device=DEV) if y is None else y
    ws = torch.full((moe.moe_linear_workspace_bytes(cfg, T),), 0xFF, dtype=torch.uint8, device=DEV)
    moe.moe_linear(cfg, codes, scales, x, y[:T, :out], ws, bias=bias, residual=res)
    torch.cuda.synchronize()
    assert bool((y[T] == 9).all()) and bool((y[:, out:] == 9).all())  # nothing behind rows and columns
    return y[:T, :out]


def _x(rng, T, K, dtype, pad=0, shift=0, whole=False):
    v = rng.integers(-8, 9, (T, K)).astype(np.float32) if whole else rng.normal(0, 1, (T, K)).astype(np.float32)
    if not whole:
        v[:, ::37] *= 50.0
    t = torch.from_numpy(v).to(DT[dtype])
    buf = torch.full((T * (K + pad) + shift,), float("nan"), dtype=DT[dtype], device=DEV)
    d = buf[shift:].as_strided((T, K), (K + pad, 1))
    d.copy_(t)
    return d, t.double().numpy()


SHAPES = [(1, 64, 32), (1, 192, 96), (2, 128, 2080), (3, 320, 64), (16, 64, 160), (17, 448, 224), (31, 128, 1024),
          (33, 192, 512), (64, 576, 96), (65, 64, 320), (129, 320, 160), (200, 1088, 64), (300, 128, 544)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_whole_numbers_are_exact(T, N, K, bits, group, dtype):
    """Small whole activations and scales of 1/2, 1 and 2: every partial sum is a multiple of 1/2 below 2^23, so any
    order of additions gives the same fp32 value, rounded once to the type."""
    K = (K + group - 1) // group * group if group else K
    rng = np.random.default_rng(T * 1000 + N + K)
    q, s, codes, scales = _weights(rng, N, K, bits, group, whole=True)
    x, x64 = _x(rng, T, K, dtype, whole=True)
    y = _call(moe.LinearConfig(N, K, bits, group), codes, scales, x, N)
    want = x64 @ (q * np.repeat(s, K // s.shape[1], axis=1)).T
    assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)).to(DT[dtype]))


# Enough tiles for each way in which larger batches are laid out over the card: whole turns of 512 tiles of 128 x 256, up
# to 256 with wavefronts that share the columns, halves and quarters; with 64-token tiles (fp32, group scales) the same.
BATCHES = [(1024, 16384, 64), (600, 8128, 96), (300, 8192, 160), (191, 6080, 352), (70, 6144, 1056), (520, 16320, 32),
           (1700, 11072, 128), (193, 4160, 96), (33, 12352, 544)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group,act", [(4, 0, "none"), (8, 0, "none"), (4, 32, "none"), (4, 128, "none"), (4, 0, "relu")])
@pytest.mark.parametrize("T,N,K", BATCHES)
def test_whole_numbers_are_exact_in_large_batches(T, N, K, bits, group, act, dtype):
    K = (K + group - 1) // group * group if group else K
    rng = np.random.default_rng(T + N + K)
    q, s, codes, scales = _weights(rng, N, K, bits, group, whole=True)
    x, x64 = _x(rng, T, K, dtype, whole=True)
    y = _call(moe.LinearConfig(N, K, bits, group, ACT[act]), codes, scales, x, N)
    wt = torch.from_numpy(q * np.repeat(s, K // s.shape[1], axis=1)).to(DEV)
    want = torch.mm(torch.from_numpy(x64).to(DEV), wt.t().contiguous())
    want = want.clamp(min=0) if act == "relu" else want
    assert torch.equal(y, want.float().to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group,act", [(4, 0, "none"), (8, 0, "relu"), (4, 32, "none"), (4, 64, "none"), (4, 128, "none")])
@pytest.mark.parametrize("T,N,K", [(1, 16448, 256), (3, 33024, 384), (4, 24640, 1152), (1, 8256, 2176)])
def test_heads_are_exact(T, N, K, bits, group, act, dtype):
    """Few tokens and many rows, whole numbers: a workgroup's rows in several turns, the last of them not full."""
    rng = np.random.default_rng(T + N + K)
    q, s, codes, scales = _weights(rng, N, K, bits, group, whole=True)
    x, x64 = _x(rng, T, K, dtype, whole=True)
    b = rng.integers(-64, 65, N).astype(np.float32)
    y = _call(moe.LinearConfig(N, K, bits, group, ACT[act]), codes, scales, x, N, torch.from_numpy(b).to(DEV))
    want = torch.mm(torch.from_numpy(x64).to(DEV), torch.from_numpy(q * np.repeat(s, K // s.shape[1], axis=1)).to(DEV).t().contiguous())
    want = want + torch.from_numpy(b).to(DEV).double()
    want = want.clamp(min=0) if act == "relu" else want
    assert torch.equal(y, want.float().to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K,bits,group", [(1024, 16384, 64, 4, 0), (600, 8064, 96, 8, 0), (300, 8192, 160, 4, 0),
                                              (191, 6080, 352, 4, 0), (520, 16320, 128, 4, 128), (33, 12352, 544, 4, 32)])
def test_swiglu_in_large_batches(T, N, K, bits, group, dtype):
    rng = np.random.default_rng(T + N + K)
    q, s, codes, scales = _weights(rng, N, K, bits, group)
    x, x64 = _x(rng, T, K, dtype)
    b = rng.normal(0, 0.5, N).astype(np.float32)
    res = torch.from_numpy(rng.normal(0, 1, (T, N // 2)).astype(np.float32)).to(DT[dtype])
    y = _call(moe.LinearConfig(N, K, bits, group, ACT["swiglu"]), codes, scales, x, N // 2, torch.from_numpy(b).to(DEV),
              res.to(DEV))
    rows = rng.permutation(T)[:24]
    ref, err = R.linear(q, s, x64[rows], "swiglu", b.astype(np.float64), res.double().numpy()[rows])
    got = y.double().cpu().numpy()[rows]
    assert np.all(np.abs(got - ref) <= err + R.HALF_STEP[dtype] * (np.abs(ref) + err) + 1e-37)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("T,N,K,bits,group", [(1, 256, 544, 4, 0), (5, 64, 256, 4, 32), (16, 192, 96, 8, 0),
                                              (30, 448, 256, 4, 64), (40, 128, 1024, 8, 0), (131, 320, 384, 4, 128),
                                              (257, 576, 160, 4, 0)])
def test_epilogues(T, N, K, bits, group, act, dtype):
    rng = np.random.default_rng(N + K + T)
    q, s, codes, scales = _weights(rng, N, K, bits, group)
    x, x64 = _x(rng, T, K, dtype)
    out = N // 2 if act == "swiglu" else N
    cfg = moe.LinearConfig(N, K, bits, group, ACT[act])
    b = rng.normal(0, 0.5, N).astype(np.float32)
    r = torch.from_numpy(rng.normal(0, 1, (T, out)).astype(np.float32)).to(DT[dtype])
    for bias, res in ((None, None), (b, None), (None, r), (b, r)):
        y = _call(cfg, codes, scales, x, out, None if bias is None else torch.from_numpy(bias).to(DEV),
                  None if res is None else res.to(DEV))
        ref, err = R.linear(q, s, x64, act, None if bias is None else bias.astype(np.float64),
                            None if res is None else res.double().numpy())
        tiny = 2.0 ** -25 if dtype == "f16" else 1e-37
        tol = err + R.HALF_STEP[dtype] * (np.abs(ref) + err) + tiny
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("dtype,pad,shift", [("bf16", 8, 0), ("bf16", 3, 1), ("f32", 1, 3), ("f16", 0, 1), ("f16", 24, 8)])
@pytest.mark.parametrize("T", [1, 6, 45])
def test_strides(T, dtype, pad, shift):
    rng = np.random.default_rng(pad + T)
    N, K = 192, 352
    q, s, codes, scales = _weights(rng, N, K, 4, 0, whole=True)
    x, x64 = _x(rng, T, K, dtype, pad, shift, whole=True)
    want = x64 @ (q * s).T
    y = _call(moe.LinearConfig(N, K), codes, scales, x, N)
    assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)).to(DT[dtype]))
    # residual with its own stride, and the output over the residual itself
    buf = torch.full((T + 1, N + 3), 9.0, dtype=DT[dtype], device=DEV)
    res = torch.from_numpy(rng.integers(-4, 5, (T, N)).astype(np.float32)).to(DT[dtype])
    buf[:T, :N] = res.to(DEV)
    wide = torch.zeros((T, N + 7), dtype=DT[dtype], device=DEV)
    wide[:, :N] = res.to(DEV)
    want = torch.from_numpy((want + res.double().numpy()).astype(np.float32)).to(DT[dtype])
    assert torch.equal(_call(moe.LinearConfig(N, K), codes, scales, x, N, res=wide[:, :N]).cpu(), want)
    assert torch.equal(_call(moe.LinearConfig(N, K), codes, scales, x, N, res=buf[:T, :N], y=buf).cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N", [(1, 128), (9, 128), (70, 128), (70, 6144)])
def test_extreme_activations(T, N, dtype):
    """Zero tokens, tiny and huge ones next to each other, and a token with an infinity or NaN, which leaves the other
    tokens as they are."""
    rng = np.random.default_rng(T)
    K = 256
    q, s, codes, scales = _weights(rng, N, K, 4, 64)
    cfg = moe.LinearConfig(N, K, 4, 64)
    big, small = {"f32": (1e30, 1e-30), "bf16": (1e30, 1e-30), "f16": (2000.0, 1e-3)}[dtype]
    v = rng.normal(0, 1, (T, K)).astype(np.float32)
    v[0] *= small
    if T > 4:
        v[1] = 0
        v[2] *= big
        v[3, ::2] *= small
        v[4, 5] *= big
    t = torch.from_numpy(v).to(DT[dtype])
    y = _call(cfg, codes, scales, t.to(DEV), N).clone()
    ref, err = R.linear(q, s, t.double().numpy())
    # below the normal range of the output type a rounding is off by half of its smallest step
    tiny = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}[dtype]
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= err + R.HALF_STEP[dtype] * (np.abs(ref) + err) + tiny)
    if T > 4:
        assert bool((y[1] == 0).all())
        for bad in (float("inf"), float("-inf"), float("nan")):
            t2 = t.clone()
            t2[5, 17] = bad
            y2 = _call(cfg, codes, scales, t2.to(DEV), N)
            assert not bool(torch.isfinite(y2[5]).any())
            keep = [i for i in range(T) if i != 5]
            assert torch.equal(y2[keep], y[keep])


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("T,N", [(2, 128), (20, 128), (70, 6144)])
def test_nan_stays_behind_every_activation(T, N, act):
    rng = np.random.default_rng(N)
    K = 64
    _, _, codes, scales = _weights(rng, N, K, 4, 0)
    x, _ = _x(rng, T, K, "f32")
    x[1, 7] = float("nan")
    y = _call(moe.LinearConfig(N, K, 4, 0, ACT[act]), codes, scales, x, N // 2 if act == "swiglu" else N)
    assert bool(y[1].isnan().all()) and bool(y[0].isfinite().all()) and bool(y[2:].isfinite().all())


@pytest.mark.parametrize("dtype,pad,shift", [("f32", 0, 0), ("f32", 1, 3), ("bf16", 8, 0), ("bf16", 3, 1), ("f16", 24, 8),
                                             ("f16", 0, 1)])
@pytest.mark.parametrize("T,N,K", [(100, 4160, 8352), (130, 4096, 16448)])
def test_long_rows_in_batches(T, N, K, dtype, pad, shift):
    """Rows longer than the lanes that convert them hold at once, aligned and not; the residual in place in a buffer
    whose rows are four apart, and one whose rows are not."""
    rng = np.random.default_rng(K + pad)
    q, s, codes, scales = _weights(rng, N, K, 4, 0, whole=True)
    x, x64 = _x(rng, T, K, dtype, pad, shift, whole=True)
    res = torch.from_numpy(rng.integers(-64, 65, (T, N)).astype(np.float32)).to(DT[dtype]).to(DEV)
    want = torch.mm(torch.from_numpy(x64).to(DEV), torch.from_numpy(q * s).to(DEV).t().contiguous())
    want = (want + res.double()).float().to(DT[dtype])
    for extra in (4, 3):
        y = torch.full((T + 1, N + extra), 9.0, dtype=DT[dtype], device=DEV)
        y[:T, :N] = res
        assert torch.equal(_call(moe.LinearConfig(N, K), codes, scales, x, N, res=y[:T, :N], y=y), want)


def test_calls_at_once():
    """Calls on two streams that run at the same time, each with its own workspace."""
    rng = np.random.default_rng(5)
    N, K = 6144, 1024
    _, _, codes, scales = _weights(rng, N, K, 4, 64)
    cfg = moe.LinearConfig(N, K, 4, 64)
    xs = [_x(rng, T, K, "bf16")[0] for T in (2, 40, 300, 700)]
    want = [_call(cfg, codes, scales, x, N).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = [torch.empty((x.shape[0], N), dtype=torch.bfloat16, device=DEV) for x in xs]
    ws = [torch.empty(moe.moe_linear_workspace_bytes(cfg, x.shape[0]), dtype=torch.uint8, device=DEV) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, y, w, st in zip(xs, got, ws, streams):
            moe.moe_linear(cfg, codes, scales, x, y, w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_codes_beyond_2_to_the_31_elements():
    """Rows beyond 2^31 code elements apart (a head of 131,072 rows over 16,416 columns)."""
    N, K, T = 131072, 16416, 2
    codes = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device=DEV)
    scales = torch.ones(N, device=DEV)
    x = torch.zeros((T, K), dtype=torch.float32, device=DEV)
    x[0, K - 1] = 1.0
    x[1, 0] = 2.0
    cfg = moe.LinearConfig(N, K)
    y = torch.empty((T, N), device=DEV)
    ws = torch.empty(moe.moe_linear_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV)
    moe.moe_linear(cfg, codes, scales, x, y, ws)
    tiles = codes.view(N // 64, K // 32, 64, 16)
    last = (tiles[:, -1, :, 15] >> 4).to(torch.int16).reshape(-1)
    first = (tiles[:, 0, :, 0] & 15).to(torch.int16).reshape(-1)
    assert torch.equal(y[0], torch.where(last > 7, last - 16, last).float())
    assert torch.equal(y[1], 2 * torch.where(first > 7, first - 16, first).float())


@pytest.mark.parametrize("T", [1, 20, 70])
def test_dense_feed_forward(T):
    """The two products of a dense layer as they are used: gate and up with SwiGLU, then down into the residual
    stream, in place."""
    rng = np.random.default_rng(T)
    H, I = 256, 320
    q1, s1, c1, d1 = _weights(rng, 2 * I, H, 4, 32)
    q2, s2, c2, d2 = _weights(rng, H, I, 8, 0)
    h, h64 = _x(rng, T, H, "f32")
    up = moe.LinearConfig(2 * I, H, 4, 32, moe.MOE_ACT_SWIGLU)
    down = moe.LinearConfig(H, I, 8)
    a = torch.empty((T, I), device=DEV)
    ws = torch.empty(max(moe.moe_linear_workspace_bytes(c, T) for c in (up, down)), dtype=torch.uint8, device=DEV)
    moe.moe_linear(up, c1, d1, h, a, ws)
    moe.moe_linear(down, c2, d2, a, h, ws, residual=h)
    r1, e1 = R.linear(q1, s1, h64, "swiglu")
    r2, e2 = R.linear(q2, s2, r1, res=h64)
    e2 = e2 + e1 @ np.abs(q2 * s2).T * (1 + 1e-3)
    assert np.all(np.abs(h.double().cpu().numpy() - r2) <= e2 + 2.0 ** -24 * np.abs(r2))


@pytest.mark.parametrize("T,N,K", [(2, 256, 512), (40, 256, 2048), (150, 192, 96)])
def test_streams_and_graph_replays(T, N, K):
    """On a side stream, and captured: every replay equals the eager call, with eager work and synchronizations
    between the replays; equal calls give equal bits."""
    rng = np.random.default_rng(T)
    _, _, codes, scales = _weights(rng, N, K, 4, 32)
    cfg = moe.LinearConfig(N, K, 4, 32, moe.MOE_ACT_SILU)
    x, _ = _x(rng, T, K, "bf16")
    inputs = [_x(rng, T, K, "bf16")[0] for _ in range(4)]
    ya, yb = (torch.empty((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    wa, wb = (torch.empty(moe.moe_linear_workspace_bytes(cfg, T), dtype=torch.uint8, device=DEV) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(cfg, codes, scales, x, ya, wa, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    moe.moe_linear(cfg, codes, scales, x, yb, wb)
    torch.cuda.synchronize()
    assert torch.equal(ya, yb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear(cfg, codes, scales, x, ya, wa)
    for xx in inputs:
        x.copy_(xx)
        moe.moe_linear(cfg, codes, scales, xx, yb, wb)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, yb)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 64)])
@pytest.mark.parametrize("T,N", [(1, 128), (2, 128), (4, 128), (5, 128), (20, 128), (70, 128), (70, 6144), (1, 24704),
                                 (3, 24704)])
@pytest.mark.parametrize("size,scale", [(3e37, 1.0), (1e-39, 1e24)])
def test_sums_beyond_fp32_before_their_scales(T, N, bits, group, dtype, size, scale):
    """Activations near fp32's largest, whose sums with the codes (about 70 or 1,200 times as large) leave its range
    until the scales bring them back, and activations below its normal range under large scales. Both results lie far
    inside the range (about 1e37 and 3e-16), so the bound has no term for overflow or underflow."""
    rng = np.random.default_rng(T + N + bits)
    K = 256
    q, s, codes, scales = _weights(rng, N, K, bits, group)
    s, scales = s * scale, scales * scale
    s = np.float64(np.float32(s / scale) * np.float32(scale))  # as the device multiplies
    x = torch.from_numpy((rng.normal(0, 1, (T, K)) * size).astype(np.float32)).to(DT[dtype])
    y = _call(moe.LinearConfig(N, K, bits, group), codes, scales, x.to(DEV), N)
    ref, err = R.linear(q, s, x.double().numpy())
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= err + R.HALF_STEP[dtype] * (np.abs(ref) + err))


def _device_weights(seed, N, K, bits, group):
    """_weights(whole=True) made on the device, for large matrices: codes, scales and W in 64 bits."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lim = 8 if bits == 4 else 128
    q = torch.randint(-lim, lim, (N, K), generator=g, device=DEV, dtype=torch.int8)
    G = group or K
    s = torch.exp2(torch.randint(-1, 2, (N, K // G), generator=g, device=DEV).float())
    if bits == 4:
        u = (q & 15).view(torch.uint8)
        row = (u[:, 0::2] | (u[:, 1::2] << 4)).contiguous()
    else:
        row = q
    codes = torch.empty(row.numel(), dtype=torch.uint8, device=DEV)
    (moe.moe_tile_int4 if bits == 4 else moe.moe_tile_int8)(row, codes)
    scales = s.view(-1)
    if group:
        scales = torch.empty_like(scales)
        moe.moe_tile_group_scales(s, scales)
    return codes, scales, (q.double().view(N, K // G, G) * s.double()[:, :, None]).view(N, K)


# For 1 to 4 tokens: 6 to 32 blocks of four a wavefront, in whole and in ragged numbers, heads in turns among them; for
# 5 to 32: 7 to 16 a workgroup, with a short last part, 128 KB of fp32 activations (6,656 rows x 8,320), and 65 and more
# parts to add (64 rows). Columns that are no multiple of a group are rounded up to one.
FEW_LONG = [(1, 192, 6144), (1, 64, 8320), (1, 64, 16384), (1, 24640, 4704), (3, 128, 6144), (4, 64, 8160), (2, 24704, 5216),
            (5, 4096, 6144), (8, 6656, 8320), (16, 6144, 6240), (17, 4096, 6144), (24, 6656, 8320), (32, 6144, 6144),
            (32, 64, 8320), (9, 64, 6176), (64, 6144, 2080)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("T,N,K", FEW_LONG)
def test_few_tokens_over_long_rows_are_exact(T, N, K, bits, group, dtype):
    """Whole numbers again, over rows so long that every code in flight is replaced by later ones, and every round in
    which activations are converted is used. A row's sums are multiples of its smallest scale, and the sum of their
    absolute products stays below 2^24 of those, so every partial sum is exact in any order."""
    K = (K + group - 1) // group * group if group else K
    codes, scales, wt = _device_weights(T + N + K, N, K, bits, group)
    x, x64 = _x(np.random.default_rng(K), T, K, dtype, whole=True)
    xd = torch.from_numpy(x64).to(DEV)
    least = scales.view(N // 64, -1, 64).amin(1).view(N) if group else scales
    assert bool((torch.mm(xd.abs(), wt.abs().t().contiguous()) < 2 ** 24 * least.double()).all())
    b = torch.arange(N, device=DEV).float() % 129 - 64
    res = torch.arange(T * N, device=DEV).view(T, N).remainder(17).to(DT[dtype])
    y = _call(moe.LinearConfig(N, K, bits, group), codes, scales, x, N, b, res)
    want = torch.mm(xd, wt.t().contiguous()) + b.double() + res.double()
    assert torch.equal(y, want.float().to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("T,N,K", [(1, 512, 6144), (3, 256, 8192), (1, 49280, 2208), (7, 4096, 6144), (30, 8192, 6240)])
def test_swiglu_of_few_tokens_over_long_rows(T, N, K, bits, group, dtype):
    """The same with SwiGLU, whole numbers times 2^-14: the sums are exact multiples of 2^-15, so only the epilogue
    rounds. Its error relative to the value, counted in 2^-24: the exponential 3 and its argument's part beyond fp32 1,
    1 + e 1, the reciprocal 2, three products 3, the residual's addition 1 of the larger of the two. fp16 below its
    normal range: half of its smallest step, 2^-25."""
    K = (K + group - 1) // group * group if group else K
    codes, scales, wt = _device_weights(T + N + K, N, K, bits, group)
    scales *= 2.0 ** -14
    x, x64 = _x(np.random.default_rng(K), T, K, dtype, whole=True)
    v = torch.mm(torch.from_numpy(x64).to(DEV), wt.t().contiguous()) * 2.0 ** -14
    res = torch.arange(T * (N // 2), device=DEV).view(T, N // 2).remainder(17).to(DT[dtype])
    y = _call(moe.LinearConfig(N, K, bits, group, ACT["swiglu"]), codes, scales, x, N // 2, None, res)
    gate, up = v[:, :N // 2], v[:, N // 2:]
    a = gate / (1 + torch.exp(-gate)) * up
    want = a + res.double()
    err = 2.0 ** -24 * (10 * a.abs() + torch.maximum(want.abs(), a.abs())) + (2.0 ** -25 if dtype == "f16" else 0.0)
    assert bool(((y.double() - want).abs() <= err + R.HALF_STEP[dtype] * (want.abs() + err)).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K,act", [(1 << 20, 64, 32, "none"), (6100, 64, 160, "none"), (1, 1 << 20, 32, "none"),
                                       (20, 1 << 20, 32, "none"), (40, 1 << 20, 64, "relu"), (1, 64, 65536, "none"),
                                       (4, 64, 65536, "none"), (24, 128, 65536, "none"), (70, 64, 65536, "none"),
                                       (70, 6144, 65536, "relu")])
def test_largest_sizes_are_exact(T, N, K, act, dtype):
    """The most tokens, rows and columns that the operator takes, whole numbers; the sums as in the test of long rows."""
    codes, scales, wt = _device_weights(T + N + K, N, K, 4, 0)
    x = torch.randint(-2, 3, (T, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).to(DT[dtype])
    assert 2 * 8 * K < 2 ** 24
    y = _call(moe.LinearConfig(N, K, 4, 0, ACT[act]), codes, scales, x, N)
    for t0 in range(0, T, 1 << 16):
        want = torch.mm(x[t0:t0 + (1 << 16)].double(), wt.t().contiguous())
        want = want.clamp(min=0) if act == "relu" else want
        assert torch.equal(y[t0:t0 + (1 << 16)], want.float().to(DT[dtype]))


@pytest.mark.parametrize("bits,group", [(4, 0), (8, 0), (4, 32)])
@pytest.mark.parametrize("T,N", [(1, 128), (4, 128), (20, 128), (70, 128), (300, 8192)])
def test_activations_below_the_normal_range_of_fp16(T, N, bits, group):
    """fp16 activations that are all whole multiples of its smallest step 2^-24, up to 2^-18: none is lost. The sums are
    exact (whole numbers times 2^-25), and scales of 2^12 to 2^14 bring the results back into fp16's range."""
    rng = np.random.default_rng(T + N)
    K = 256
    q, s, codes, scales = _weights(rng, N, K, bits, group, whole=True)
    v = torch.from_numpy(rng.integers(-64, 65, (T, K)) * 2.0 ** -24).to(torch.float16)
    y = _call(moe.LinearConfig(N, K, bits, group), codes, scales * 2.0 ** 13, v.to(DEV), N)
    want = v.double().numpy() @ (q * np.repeat(s, K // s.shape[1], axis=1)).T * 2.0 ** 13
    assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)).to(torch.float16))
