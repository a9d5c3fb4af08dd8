"""Inputs on the GPU for the tests of adapted products and their gradients, with the same values in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import int4_quantized_expert_amd as moe

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACT = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
       "gelu_tanh": moe.MOE_ACT_GELU_TANH, "swiglu": moe.MOE_ACT_SWIGLU}


def weights(rng, N, K, bits, group, whole=False):
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


def matrix(rng, T, C, dtype, pad=0, shift=0, whole=0, spread=True):
    """[T][C] on the device, rows C + pad apart and `shift` elements behind an aligned address, and its values."""
    v = rng.integers(-whole, whole + 1, (T, C)).astype(np.float32) if whole else rng.normal(0, 1, (T, C)).astype(np.float32)
    if not whole and spread:
        v[:, ::37] *= 50.0
    t = torch.from_numpy(v).to(DT[dtype])
    buf = torch.full((T * (C + pad) + shift,), float("nan"), dtype=DT[dtype], device=DEV)
    d = buf[shift:].as_strided((T, C), (C + pad, 1))
    d.copy_(t)
    return d, t.double().numpy()


def adapters(rng, n, R, N, K, dtype, whole=False):
    if whole:
        a, b = rng.integers(-1, 2, (n, R, K)), rng.integers(-2, 3, (n, N, R))
        s = rng.choice([0.5, 1.0, 2.0], n)
    else:
        a, b, s = rng.normal(0, 1 / np.sqrt(K), (n, R, K)), rng.normal(0, 0.1, (n, N, R)), rng.uniform(0.5, 2.0, n)
    a, b = (torch.from_numpy(v.astype(np.float32)).to(DT[dtype]) for v in (a, b))
    s = torch.from_numpy(s.astype(np.float32))
    return moe.Adapters(a.to(DEV), b.to(DEV), s.to(DEV)), a.double().numpy(), b.double().numpy(), s.double().numpy()


def ids_of(rng, T, n, how):
    """Adapter of each token: any mix, runs, one for all, none."""
    if how == "mix":
        v = rng.integers(-1, n + 1, T)  # -1 and n: no adapter
    elif how == "runs":
        v = np.repeat(rng.integers(-1, n, T), rng.integers(1, 40, T))[:T]
    elif how == "one":
        v = np.full(T, n - 1)
    elif how == "none":
        v = np.full(T, -1)
    else:
        return None, None
    v = v.astype(np.int32)
    return torch.from_numpy(v).to(DEV), v


def guarded(T, C, dtype, pad=3):
    """A [T][C] part of a larger matrix filled with 9, and that matrix."""
    full = torch.full((T + 1, C + pad), 9.0, dtype=DT[dtype], device=DEV)
    return full[:T, :C], full


def untouched(full, T, C):
    return bool((full[T] == 9).all()) and bool((full[:, C:] == 9).all())


def space(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
