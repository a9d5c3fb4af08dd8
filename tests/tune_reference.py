"""Plain 64-bit implementations of the adapted linear product, of its gradients and of gradient clipping for the tests,
with the bounds on what the kernels' roundings can do to them."""
from __future__ import annotations

import math

import numpy as np

from tests.ops_reference import HALF_STEP, _sig, activation

UNIT = 2.0 ** -24


def weights(q, s):
    return q * np.repeat(s, q.shape[1] // s.shape[1], axis=1)


def chosen(ids, n, T):
    """Adapter of each token, -1 for none."""
    ids = np.zeros(T, np.int64) if ids is None else np.asarray(ids, np.int64)
    return np.where((ids >= 0) & (ids < n), ids, -1)


def low_rank(x, a, b, sc, ids, split):
    """(scale B (A x), bound on its error) by token. Sums of fp32 products: (terms + 4) 2^-24 of the absolute products; split:
    scale (A x) keeps 16 bits between the two products (2^-16 of it), and an fp16 b may lose the product of the two
    low parts (2^-16 of theirs)."""
    T, N = x.shape[0], b.shape[1]
    v, err = np.zeros((T, N)), np.zeros((T, N))
    at = chosen(ids, a.shape[0], T)
    for e in np.unique(at[at >= 0]):
        t = np.nonzero(at == e)[0]
        h = x[t] @ a[e].T * sc[e]
        eh = (x.shape[1] + 6) * UNIT * (np.abs(x[t]) @ np.abs(a[e]).T) * abs(sc[e])
        v[t] = h @ b[e].T
        err[t] = (eh + ((2.0 ** -15 if split else 0.0) + (a.shape[1] + 6) * UNIT) * np.abs(h)) @ np.abs(b[e]).T
    return v, err


def finish(v, err, act, res):
    """act(v) + res and the bound that `err` of v gives (as ops_reference.linear's)."""
    if act == "swiglu":
        half = v.shape[1] // 2
        g, u, eg, eu = v[:, :half], v[:, half:], err[:, :half], err[:, half:]
        s = g * _sig(g)
        y = s * u
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 8 * UNIT * np.abs(y)
    else:
        y, slope = activation(v, act)
        err = slope * err
        if act not in ("none", "relu"):
            err = err + 24 * UNIT * np.maximum(np.abs(y), np.abs(v) * 2.0 ** -20)
    if res is not None:
        y = y + res
        err = err + 2 * UNIT * np.abs(y)
    return y, err


def adapted(q, s, x, a, b, sc, ids, dtype, act="none", bias=None, res=None):
    """(y, its bound, z, its bound) before the rounding to the type; a None: no adapters."""
    w = weights(q, s)
    z = x @ w.T
    K = x.shape[1]
    err = UNIT * (K + 24) * (np.abs(x) @ np.abs(w).T)
    err = err + 2.0 ** -38 * np.abs(x).max(axis=1, keepdims=True) * np.abs(w).sum(axis=1)[None, :]
    if a is not None:
        v, ev = low_rank(x, a, b, sc, ids, dtype != "f32")
        z, err = z + v, err + ev + UNIT * np.abs(z + v)
    if bias is not None:
        z = z + bias[None, :]
        err = err + UNIT * np.abs(z)
    y, ey = finish(z, err, act, res)
    return y, ey, z, err


def slope(z, act):
    """Derivative of the activation at z."""
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        s = _sig(z)
        return s + z * s * _sig(-z)
    if act == "gelu":
        cdf = np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in z.ravel()]).reshape(z.shape)
        return cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = _sig(2 * c * (z + 0.044715 * z ** 3))
    return s + z * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * z * z)


def grad_in(dy, z, act):
    """(dz, size of the terms in it)."""
    if act == "swiglu":
        half = z.shape[1] // 2
        g, u = z[:, :half], z[:, half:]
        dg, du = dy * u * slope(g, "silu"), dy * g * _sig(g)
        return np.concatenate([dg, du], axis=1), np.concatenate([np.abs(dy * u) * 1.1, np.abs(dy * g)], axis=1)
    d = slope(z, act) if act != "none" else 1.0
    return dy * d, np.abs(dy) * (1.13 if act not in ("none", "relu") else 1.0)


def backward(q, s, x, a, b, sc, ids, dy, z, dtype, act="none", res=None):
    """Gradients dx, d_a, d_b, each with its bound before the rounding to the type. dz is off by `ez`: a few fp32
    roundings of the derivative, and for the adapters' sums its rounding to the type."""
    w = weights(q, s)
    dz, size = grad_in(dy, z, act)
    T, N = dz.shape
    ez = (0.0 if act in ("none", "relu") else 32 * UNIT) * size
    # one rounding of dz times the row's scale (fp32: 2^-22), with group scales one or two of the weight, fp32 sums
    step = 2.0 ** -22 if dtype == "f32" else 2.0 ** -11
    if s.shape[1] > 1:
        step += 2.0 ** -18 if dtype == "f32" else 2.0 ** -10
    dx = dz @ w
    top = np.abs(dz) * np.abs(s).max(axis=1)[None, :]  # what the token's power of two is made for
    ex = (ez + (step + (N + 24) * UNIT) * np.abs(dz)) @ np.abs(w)
    ex = ex + 2.0 ** -38 * top.max(axis=1, keepdims=True) * np.abs(q).sum(axis=0)[None, :]
    # group scales far below their row's largest: half a step of fp16's smallest, 2^-25, over the power of two that puts the
    # largest in [2^11, 2^12)
    if s.shape[1] > 1:
        ex = ex + 2.0 ** -36 * (top @ np.abs(q))
    da = db = ea = eb = None
    if a is not None:
        n, R, K = a.shape
        da, db, ea, eb = np.zeros(a.shape), np.zeros(b.shape), np.zeros(a.shape), np.zeros(b.shape)
        at = chosen(ids, n, T)
        half = HALF_STEP[dtype] if act != "none" else 0.0
        part = 0.0 if dtype == "f32" else 2.0 ** -15
        for e in np.unique(at[at >= 0]):
            t = np.nonzero(at == e)[0]
            d, ed = dz[t], ez[t] + half * (np.abs(dz[t]) + ez[t])
            u = d @ b[e] * sc[e]
            eu = (ed + (N + 6) * UNIT * np.abs(d)) @ np.abs(b[e]) * abs(sc[e])
            h = x[t] @ a[e].T * sc[e]
            eh = (K + 6) * UNIT * (np.abs(x[t]) @ np.abs(a[e]).T) * abs(sc[e])
            sums = part + (len(t) + 24) * UNIT
            da[e] = u.T @ x[t]
            ea[e] = (eu + sums * np.abs(u)).T @ np.abs(x[t])
            db[e] = d.T @ h
            eb[e] = (ed + sums * np.abs(d)).T @ (np.abs(h) + eh) + np.abs(d).T @ eh
            dx[t] += u @ a[e]
            ex[t] += (eu + (part + (R + 6) * UNIT) * np.abs(u)) @ np.abs(a[e])
    if res is not None:
        dx = dx + res
    ex = ex + 3 * UNIT * np.abs(dx)
    return (dx, ex), (da, ea), (db, eb)


def value(q, s, x, a, b, sc, ids, dy, act):
    """<dy, act(z)>, the function whose gradients are tested by differences."""
    z = x @ weights(q, s).T + low_rank(x, a, b, sc, ids, False)[0]
    return float((dy * finish(z, np.zeros_like(z), act, None)[0]).sum())


def within(got, want, err, dtype, tiny=1e-37):
    """Whether one more rounding to the type leaves got inside the bound. fp16's smallest step is 2^-24, and by its rounding
    rule 65520 (half a step above its largest, 65504) and all beyond is infinity: there, and only where the bound reaches
    that far, infinity of the same sign is right."""
    low = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}[dtype]
    ok = np.abs(got - want) <= err + HALF_STEP[dtype] * (np.abs(want) + err) + low + tiny
    if dtype == "f16":
        ok |= np.isinf(got) & (np.sign(got) * want + err >= 65520.0)
    return ok
