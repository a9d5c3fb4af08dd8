"""moe_grad_clip on the GPU against the definition in 64 bits."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import int4_quantized_expert_amd as moe  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _tensors(rng, sizes, types, scale=1.0):
    """Gradients at odd addresses: each a part of a larger array of 9."""
    full, grads = [], []
    for n, t in zip(sizes, types):
        lead = int(rng.integers(0, 9))
        f = torch.full((n + lead + 5,), 9.0, dtype=DT[t], device=DEV)
        f[lead:lead + n] = torch.from_numpy((scale * rng.normal(0, 1, n)).astype(np.float32)).to(DT[t]).to(DEV)
        full.append((f, lead, n))
        grads.append(f[lead:lead + n])
    return full, grads


def _clean(full):
    return all(bool((f[:lead] == 9).all()) and bool((f[lead + n:] == 9).all()) for f, lead, n in full)


def _norm(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def _check(before, after, norm, limit):
    """factor and product in fp32 (2^-23 together), one rounding to the type; fp16 below its normal range 2^-25."""
    c = min(1.0, limit / norm)
    for g, o in zip(before, after):
        want = g.double() * c
        err = (2.0 ** -23 + EPS[g.dtype]) * want.abs() + (2.0 ** -25 if g.dtype == torch.float16 else 0.0)
        assert bool(((o.double() - want).abs() <= err).all())


SIZES = [[1], [7, 1, 3], [8192, 8191, 8193, 1, 0, 5], [100003, 64, 0, 17, 20000], [33] * 150, [0, 0]]


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]])
@pytest.mark.parametrize("share", [0.1, 0.999, 1.5, math.inf])
@pytest.mark.parametrize("sizes", SIZES)
def test_against_64_bits(sizes, share, types, inplace):
    rng = np.random.default_rng(sum(sizes) + len(types))
    types = [types[i % len(types)] for i in range(len(sizes))]
    full, grads = _tensors(rng, sizes, types)
    out_full, out = (full, grads) if inplace else _tensors(rng, sizes, types)
    before = [g.clone() for g in grads]
    want = _norm(before)
    limit = share * want if want > 0 else 1.0
    norm = torch.full((1,), -1.0, device=DEV)
    moe.moe_grad_clip(moe.GradTable(grads, None if inplace else out), limit, norm)
    got = float(norm)
    assert abs(got - want) <= 2.0 ** -23 * want
    assert _clean(full) and _clean(out_full)
    if not inplace:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    if share > 1.0:
        assert all(torch.equal(a, b) for a, b in zip(out, before))
    elif want > 0:
        _check(before, out, want, limit)


def test_many_runs_of_chunks():
    """More chunks than workgroups, twice over, from more tensors than one launch of the table takes."""
    rng = np.random.default_rng(1)
    sizes = [int(v) for v in rng.integers(1, 400000, 200)]
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    flat = torch.randn(sum(sizes), generator=g, device=DEV)
    grads = list(torch.split(flat, sizes))
    want = _norm([flat])
    norm, out = torch.zeros(1, device=DEV), torch.empty_like(flat)
    table = moe.GradTable(grads, list(torch.split(out, sizes)))
    moe.moe_grad_clip(table, 1.0, norm)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    _check([flat], [out], want, 1.0)
    first = out.clone()
    for _ in range(3):  # a fixed order of sums: equal bits
        out.zero_()
        moe.moe_grad_clip(table, 1.0, norm)
        assert torch.equal(out, first)


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-42])
def test_squares_beyond_32_bits(value):
    g = torch.full((5000,), value, device=DEV)
    keep = g.clone()
    norm = torch.zeros(1, device=DEV)
    moe.moe_grad_clip(moe.GradTable([g]), 1.0, norm)
    want = float(keep[0].double()) * math.sqrt(5000)
    if want >= 3.4028236e38:  # the norm itself is beyond fp32: the gradients stay
        assert math.isinf(float(norm)) and torch.equal(g, keep)
    else:
        assert abs(float(norm) - want) <= 2.0 ** -23 * want + 1e-45
        _check([keep], [g], want, 1.0)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("inplace", [True, False])
def test_a_norm_that_is_no_number_changes_nothing(bad, inplace):
    rng = np.random.default_rng(2)
    _, grads = _tensors(rng, [1000, 20000], ["f32", "bf16"])
    grads[1][777] = bad
    before = [g.clone() for g in grads]
    out = grads if inplace else [torch.zeros_like(g) for g in grads]
    norm = torch.zeros(1, device=DEV)
    moe.moe_grad_clip(moe.GradTable(grads, out), 0.5, norm)
    assert math.isnan(float(norm)) if math.isnan(bad) else math.isinf(float(norm))
    for a, b in zip(out, before):
        assert torch.equal(torch.nan_to_num(a, nan=123.0), torch.nan_to_num(b, nan=123.0))


def test_captured_and_replayed():
    rng = np.random.default_rng(4)
    _, grads = _tensors(rng, [30000, 5, 9000], ["f32", "bf16", "f16"])
    table, norm = moe.GradTable(grads), torch.zeros(1, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_grad_clip(table, 2.0, norm)
    for k in range(4):
        for g in grads:
            g.copy_(torch.randn(g.shape, device=DEV) * (k + 0.01))
        before = [g.clone() for g in grads]
        graph.replay()
        torch.cuda.synchronize()
        want = _norm(before)
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        _check(before, grads, want, 2.0)


def test_binding_refuses_what_does_not_fit():
    g = torch.zeros(100, device=DEV)
    for bad in ([g.view(10, 10).t()], [g.double()], [g, g.cpu()]):
        with pytest.raises(moe.ArgError):
            moe.GradTable(bad)
    for out in ([g[:50]], [g.bfloat16()], [g, g]):
        with pytest.raises(moe.ArgError):
            moe.GradTable([g], out)
    for grads, out in (([g, g], None), ([g[:60], g[40:]], None), ([g[:50]], [g[10:60]])):
        with pytest.raises(moe.MoeError):
            moe.GradTable(grads, out)
    table = moe.GradTable([g])
    for norm in (torch.zeros(1, device=DEV, dtype=torch.float64), torch.zeros(0, device=DEV), torch.zeros(1)):
        with pytest.raises(moe.ArgError):
            moe.moe_grad_clip(table, 1.0, norm)
    with pytest.raises(moe.MoeError):
        moe.moe_grad_clip(table, 0.0, torch.zeros(1, device=DEV))


@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f32", "bf16"]])
@pytest.mark.parametrize("size,limit", [(1e30, 1e-6), (1e30, 1e-9), (1e30, 1e-14), (3e34, 1e-20)])
@pytest.mark.parametrize("inplace", [True, False])
def test_a_limit_far_below_the_norm(size, limit, types, inplace):
    """The factor is below fp32's normal range, or below all of it; the clipped gradients are not."""
    rng = np.random.default_rng(5)
    sizes = [5000, 37, 9000]
    _, grads = _tensors(rng, sizes, [types[i % len(types)] for i in range(3)], size)
    out = grads if inplace else [torch.zeros_like(g) for g in grads]
    before = [g.clone() for g in grads]
    want = _norm(before)
    norm = torch.zeros(1, device=DEV)
    moe.moe_grad_clip(moe.GradTable(grads, out), limit, norm)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    _check(before, out, want, limit)


@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f16"]])
def test_a_copy_keeps_the_smallest_numbers(types):
    """Within the limit, to other arrays: every bit of values down to the types' smallest subnormals."""
    rng = np.random.default_rng(6)
    _, grads = _tensors(rng, [8000, 33], types * 2, {"f32": 1e-42, "bf16": 1e-39, "f16": 1e-7}[types[0]])
    out = [torch.full_like(g, 9.0) for g in grads]
    norm = torch.zeros(1, device=DEV)
    moe.moe_grad_clip(moe.GradTable(grads, out), 1.0, norm)
    assert all(torch.equal(a, b) for a, b in zip(out, grads)) and all(bool((g != 0).any()) for g in grads)
