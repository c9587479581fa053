"""The activation, its 8-bit copy and its gradient in plain 64-bit arithmetic,
with the errors that the kernels' float32 steps may leave."""

from __future__ import annotations

import math

import torch

from sort_reference import F64, HALF, TINY, U32

GROUP = 128
# relative error of a float32 sigmoid: an exponential that is off by |z| log2(e) 2^-24 in its exponent (|z| <= 88) and
# a reciprocal of one step for the 16-bit types; a few steps of accurate functions for float32
SIG = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -16, torch.float32: 8 * U32}
SMALL = 2.0 ** -120          # where float32's own range ends


def clamp_of(c):
    return math.inf if c is None else c


def forward(h, c=None):
    """a and its error bound."""
    I, lim, dt = h.shape[1] // 2, clamp_of(c), h.dtype
    g, u = h[:, :I].to(F64).clamp(-lim, lim), h[:, I:].to(F64).clamp(-lim, lim)
    a = g * torch.sigmoid(g) * u
    return a, a.abs() * (SIG[dt] + 4 * U32 + HALF[dt]) * 1.01 + TINY[dt] + SMALL * (1 + u.abs())


def codes(v):
    """int8 codes and float32 scales along the last dimension: quotients of float32 numbers, in 64 bits and rounded to
    32, are the IEEE ones."""
    v = v.to(F64)
    s = (v.abs().amax(-1) / 127).float().clamp_min(1e-8)
    q = (v / s.to(F64)[..., None]).float().to(F64).round().clamp(-127, 127)
    return q.to(torch.int8), s


def keep(h):
    M, I = h.shape[0], h.shape[1] // 2
    n = -(-I // GROUP)
    q, s = torch.empty(h.shape, dtype=torch.int8), torch.empty(M, 2 * n)
    for half in range(2):
        for k in range(n):
            lo, hi = half * I + k * GROUP, half * I + min(I, (k + 1) * GROUP)
            q[:, lo:hi], s[:, half * n + k] = codes(h[:, lo:hi])
    return q, s


def kept(q, s):
    """float32 values of a copy."""
    I = q.shape[1] // 2
    wide = s.view(s.shape[0], 2, -1).repeat_interleave(GROUP, 2)[:, :, :I].reshape(q.shape)
    return q.float() * wide


def backward(da, q, s, c=None):
    """dh in 64 bits at the kept values, and its error bound."""
    I, lim, dt = da.shape[1], clamp_of(c), da.dtype
    v = kept(q, s).to(F64)
    g0, u0, d = v[:, :I], v[:, I:], da.to(F64)
    g, u = g0.clamp(-lim, lim), u0.clamp(-lim, lim)
    sig = torch.sigmoid(g)
    f = 1 + g * (1 - sig)
    dg, du = d * u * sig * f, d * g * sig
    # f: 1 - sig is off by sig's error and half a step, its product with g and the sum by half a step each
    df = g.abs() * (sig * SIG[dt] + 2 * U32) + 2 * U32 * (1 + g.abs() * (1 - sig))
    eg = (d * u).abs() * sig * (f.abs() * SIG[dt] + df) + 4 * U32 * dg.abs()
    eu = du.abs() * (SIG[dt] + 4 * U32)
    val = torch.cat([dg * (g0.abs() <= lim), du * (u0.abs() <= lim)], 1)
    err = torch.cat([eg, eu], 1) * 1.01
    return val, err + (val.abs() + err) * HALF[dt] + TINY[dt] + SMALL * (1 + d.abs() * (1 + u.abs())).repeat(1, 2)
