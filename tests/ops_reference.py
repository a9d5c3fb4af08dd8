"""Plain 64-bit implementations of the routing and linear operators for the tests, one token at a time."""
from __future__ import annotations

import math

import numpy as np

LOWEST = {"f32": float(np.finfo(np.float32).min), "f16": -65504.0, "bf16": -3.3895313892515355e38}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # of a rounding, relative to the value
FLT_MAX = float(np.finfo(np.float32).max)


def _sig(z):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


def live_of(z, dtype, valid):
    """z [T][E] float64 holding the logits' exact values -> (values with +inf clamped, mask of live experts)."""
    with np.errstate(invalid="ignore"):
        live = z > LOWEST[dtype]
    if valid is not None:
        live = live & (np.asarray(valid) != 0)[:, None]
    return np.where(live, np.minimum(z, FLT_MAX), -np.inf), live


def scores(z, live, softmax):
    if not softmax:
        return np.where(live, _sig(np.where(live, z, 0.0)), 0.0)
    if not live.any():
        return np.zeros_like(z)
    e = np.where(live, np.exp(np.where(live, z, 0.0) - z[live].max()), 0.0)
    return e / e.sum()


def shares(z, on, softmax):
    """s / sum of s over the entries that are on, in the log domain."""
    r = np.zeros(z.shape)
    if not on.any():
        return r
    zz = z[on]
    ls = zz if softmax else np.where(zz >= 0, -np.log1p(np.exp(-np.abs(zz))), zz - np.log1p(np.exp(-np.abs(zz))))
    e = np.exp(ls - ls.max())
    r[on] = e / e.sum()
    return r


def route(z, dtype, K, G=1, KG=1, softmax=False, group_max=False, renorm=True, scale=1.0, bias=None, valid=None):
    z, live = live_of(z, dtype, valid)
    T, E = z.shape
    ids = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    load = np.zeros(E, np.int64)
    imp = np.zeros(E)
    n = E // G
    for t in range(T):
        s = scores(z[t], live[t], softmax)
        s32 = s.astype(np.float32)
        with np.errstate(over="ignore", invalid="ignore"):
            c = s32 + np.asarray(bias, np.float32) if bias is not None else z[t]
            c = np.where(live[t] & (c > -np.inf), c, -np.inf)
        if G > 1:
            by = c if bias is not None or group_max else np.where(live[t], s32, np.float32(-np.inf))
            gs = []
            for g in range(G):
                v = np.sort(by[g * n:(g + 1) * n])[::-1]
                with np.errstate(over="ignore"):
                    two = not group_max and n > 1 and v[1] > -np.inf
                    gs.append(float(np.float32(v[0]) + np.float32(v[1])) if two else float(v[0]))
            best = sorted(range(G), key=lambda g: (-gs[g], g))[:KG]
            for g in range(G):
                if g not in best:
                    c[g * n:(g + 1) * n] = -np.inf
        chosen = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:K]
        on = np.zeros(E, bool)
        on[chosen] = True
        r = shares(z[t], on, softmax) if renorm else s
        for k, e in enumerate(chosen):
            ids[t, k] = e
            w[t, k] = r[e] * scale
            load[e] += 1
        imp += shares(z[t], live[t], softmax)
    return ids, w, load, imp


def route_value(z, dtype, ids, dw, dimp, softmax, renorm, scale, valid=None):
    """sum of dw * w + sum of dimp * importance, the choice held fixed: the function whose gradient is tested."""
    z, live = live_of(z, dtype, valid)
    total = 0.0
    for t in range(z.shape[0]):
        s = scores(z[t], live[t], softmax)
        sel = [(k, e) for k, e in enumerate(ids[t]) if 0 <= e < z.shape[1] and live[t, e]]
        on = np.zeros(z.shape[1], bool)
        on[[e for _, e in sel]] = True
        r = shares(z[t], on, softmax) if renorm else s
        if dw is not None:
            total += sum(dw[t, k] * scale * r[e] for k, e in sel)
        if dimp is not None:
            total += float(shares(z[t], live[t], softmax) @ dimp)
    return total


def route_grad(z, dtype, ids, dw, dimp, softmax, renorm, scale, valid=None):
    """(gradient, size of the terms that cancel in it) by the formulas."""
    z, live = live_of(z, dtype, valid)
    T, E = z.shape
    dz, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if not live[t].any():
            continue
        s = scores(z[t], live[t], softmax)
        miss = np.where(live[t], _sig(np.where(live[t], -z[t], 0.0)), 0.0)
        u, on = np.zeros(E), np.zeros(E, bool)
        for k, e in enumerate(ids[t]):
            if dw is not None and 0 <= e < E and live[t, e]:
                u[e] += dw[t, k] * scale
                on[e] = True
        r = shares(z[t], on, softmax) if renorm else s
        if dw is not None and (renorm or softmax):
            f = 1.0 if softmax else miss
            dz[t] += r * (u - r @ u) * f
            size[t] += r * (np.abs(u) + r @ np.abs(u)) * f
        elif dw is not None:
            dz[t] += u * s * miss
            size[t] += np.abs(u) * s * miss
        if dimp is not None:
            q = shares(z[t], live[t], softmax)
            f = 1.0 if softmax else miss
            dz[t] += q * (dimp - q @ dimp) * f
            size[t] += q * (np.abs(dimp) + q @ np.abs(dimp)) * f
    return dz, size


def activation(v, act):
    """(value, bound on the slope) of a pointwise activation."""
    if act == "relu":
        return np.maximum(v, 0.0), 1.0
    if act == "silu":
        return v * _sig(v), 1.1
    if act == "gelu":
        return np.array([0.5 * a * math.erfc(-a / math.sqrt(2.0)) for a in v.ravel()]).reshape(v.shape), 1.13
    if act == "gelu_tanh":
        return v * _sig(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)), 1.13
    return v, 1.0


def linear(q, s, x, act="none", bias=None, res=None):
    """q [N][K] codes, s [N][groups], x [T][K], all float64 -> (y, bound: error of y for fp32 sums).

    A sum of K products with one rounding of 2^-24 at each addition is off by at most K 2^-24 of the sum of the
    absolute products; scale, bias and the epilogue add a few more, and the activations' conversion 2^-23 of each
    product and 2^-38 of the token's largest activation (K + 24 covers the former)."""
    N, K = q.shape
    wt = q * np.repeat(s, K // s.shape[1], axis=1)
    v = x @ wt.T
    unit = 2.0 ** -24
    err = unit * (K + 24) * (np.abs(x) @ np.abs(wt).T)
    err += 2.0 ** -38 * np.abs(x).max(axis=1, keepdims=True) * np.abs(wt).sum(axis=1)[None, :]
    if bias is not None:
        v = v + bias[None, :]
        err = err + unit * np.abs(v)
    if act == "swiglu":
        g, u = v[:, :N // 2], v[:, N // 2:]
        eg, eu = err[:, :N // 2], err[:, N // 2:]
        a = g * _sig(g)
        y = a * u
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 8 * unit * np.abs(y)
    else:
        y, slope = activation(v, act)
        err = slope * err + (0.0 if act in ("none", "relu") else 24 * unit * np.maximum(np.abs(y), np.abs(v) * 2.0 ** -20))
    if res is not None:
        y = y + res
        err = err + 2 * unit * np.abs(y)
    return y, err
