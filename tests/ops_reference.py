"""Plain 64-bit implementations of the router, the few-token layer and the
block-scaled product, with the error that float32 arithmetic may leave in
each output (first-order bounds, from the operands' magnitudes).

Unit steps: U32 = 2^-24 is half a step of float32 relative to the value, and
a sum of n terms in any order is off by at most n * 2 * U32 * sum|terms|
(every addition rounded, truncation allowed).  Half a step of bf16 is 2^-8.
"""

from __future__ import annotations

import torch

U32 = 2.0 ** -24
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
F64 = torch.float64


def gamma(n: int) -> float:
    return n * 2 * U32


# ------------------------------------------------------------------ router

def route(x, w, bias, K, scoring, renormalize=True, scale=1.0, active=None):
    """ids [T,K] (list of lists), weights [T,K], bound on the weights' error."""
    x, w = x.to(F64), w.to(F64)
    z = x @ w.t()
    # every step of the sum rounds a partial sum of at most |x| |w|; independent roundings, as the kernel's rule states
    dz = (x.norm(dim=1)[:, None] * w.norm(dim=1)[None, :]) * 2 * U32 * (x.shape[1] / 32 + 16) ** 0.5
    if scoring == "softmax":
        z = z if bias is None else z + bias.to(F64)
        score, rank = torch.softmax(z, 1), z
    else:
        score = 1 / (1 + torch.exp(-z))
        rank = z if bias is None else score + bias.to(F64)
    T, E = z.shape
    ids, wts, err = [], torch.zeros(T, K, dtype=F64), torch.zeros(T, K, dtype=F64)
    for t in range(T):
        row = rank[t].tolist()
        # NaN below every number, -inf never
        order = sorted((e for e in range(E) if row[e] != float("-inf")),
                       key=lambda e: (1, 0.0, e) if row[e] != row[e] else (0, -row[e], e))[:K]
        if active is not None and active[t] == 0:
            order = []
        n = len(order)
        ids.append(order + [-1] * (K - n))
        s = score[t, order]
        # relative error: the score's own (d log score / dz <= 1, the softmax sum another max dz), twice with the
        # normalisation, and a dozen float32 roundings
        rel = 4 * dz[t].max() + 16 * U32
        if renormalize and n:
            s = s / (s.sum() + 1e-20)
        wts[t, :n] = s * scale
        err[t, :n] = wts[t, :n].abs() * rel
    return torch.tensor(ids, dtype=torch.int32).view(T, K), wts, err


# ----------------------------------------------------------- block scaling

def quantize(x):
    """Codes (as float8) and scales, decided in IEEE float32 on the CPU."""
    v = x.float().view(x.shape[0], -1, 128)
    amax = v.abs().amax(2)
    s = amax / torch.full_like(amax, 448.0)
    s = torch.where(s < 1e-8, torch.full_like(s, 1e-8), s)
    return (v / s[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(x.shape), s


def quantize_blocks(w):
    """[N][K] float weights to e4m3 codes and scales per 128 x 128 block."""
    N, K = w.shape
    nb = -(-N // 128)
    pad = torch.zeros(nb * 128, K)
    pad[:N] = w.float()
    b = pad.view(nb, 128, K // 128, 128)
    s = (b.abs().amax((1, 3)) / 448.0).clamp_min(1e-8)
    q = (b / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(nb * 128, K)[:N].contiguous(), s


def expand_blocks(w, s):
    """Values of block-scaled weights [N][K] in 64 bits."""
    N, K = w.shape
    return w.to(torch.float32).to(F64) * s.to(F64).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)


def block_matmul(q, s, w, ws):
    """y [M][N] in 64 bits and the bound of the bf16 kernel's error."""
    a = q.to(torch.float32).to(F64) * s.to(F64).repeat_interleave(128, 1)
    b = expand_blocks(w, ws)
    y, mag = a @ b.t(), a.abs() @ b.abs().t()
    # the e4m3 MFMA drops what lies 2^-14 below the largest product of its 128; then K/128 scaled float32 additions
    return y, mag * (2.0 ** -14 + gamma(q.shape[1] // 128 + 2)) + y.abs() * HALF_BF16


# ---------------------------------------------------------- few-token layer

def interleave(w, I):
    """Formula-order rows [2I][...] (gate, up) to the prepared order (groups of 32)."""
    return w.view(2, I // 32, 32, *w.shape[1:]).transpose(0, 1).reshape(w.shape).contiguous()


def moe(x, w1, w2, ids, wts, shared=False, clamp=None, active=None, y_bf16=True):
    """w1: list of formula-order [2I][H] values, w2: list of [H][I] (64-bit).  Returns y and its error bound."""
    T, H = x.shape
    I = w1[0].shape[0] // 2
    x = x.to(F64)
    y, err = torch.zeros(T, H, dtype=F64), torch.zeros(T, H, dtype=F64)
    E = len(w1) - (1 if shared else 0)
    for t in range(T):
        if active is not None and active[t] == 0:
            continue
        routes = [(int(e), float(g)) for e, g in zip(ids[t], wts[t]) if 0 <= int(e) < E]
        if shared:
            routes.append((E, 1.0))
        for e, gate in routes:
            h, mag = w1[e] @ x[t], w1[e].abs() @ x[t].abs()
            dh = mag * gamma(H + 4)
            g, u = h[:I], h[I:]
            dg, du = dh[:I], dh[I:]
            if clamp is not None:
                g, u = g.clamp(-clamp, clamp), u.clamp(-clamp, clamp)
            silu = g / (1 + torch.exp(-g))
            a = silu * u
            # |silu'| <= 1.1; the float32 exponential, quotient and product
            da = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 16 * U32 * a.abs()
            da = da + a.abs() * (HALF_BF16 if y_bf16 else 4 * U32)
            y[t] += gate * (w2[e] @ a)
            err[t] += abs(gate) * (w2[e].abs() @ (da + (a.abs() + da) * gamma(I * 3 + 40)))
    return y, err + (y.abs() + err) * HALF_BF16 if y_bf16 else err
