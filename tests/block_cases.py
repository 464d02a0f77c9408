"""Inputs and error bounds shared by the GPU tests of the operators around the retention.

Bounds.  u = 2^-24 is half a step of fp32 relative to a value, half(t) that of the output's
type (torch.finfo(t).eps / 2).  A result that is computed in fp32 with terms of magnitude
`mag` (the sum of the terms' absolute values) and rounded once is off by at most
half(t) |ref| + k u mag, k counting the roundings on the way; each test says how it counts.
"""
import numpy as np
import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def half(t):
    return torch.finfo(t).eps / 2


def draw(seed, shape, dtype="f32", scale=1.0):
    """(CUDA tensor, its exact values in fp64)."""
    v = torch.tensor(np.random.default_rng(seed).standard_normal(shape) * scale).to(TYPES[dtype])
    return v.cuda(), v.double().numpy()


def check(got, ref, mag, k, what=""):
    g = got.detach().double().cpu().numpy()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    h = half(got.dtype)
    room = h * np.abs(ref) + (1 + h) * k * U * mag + 1e-37
    over = np.abs(g - ref) / room
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[i] <= 1, f"{what} at {i}: {g[i]} for {ref[i]}, {over[i]:.2f} of the bound"
