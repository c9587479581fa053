"""Plain 64-bit implementations of the token sort and of the way back, on the
host, with the error that float32 sums and one rounding may leave.

Half a step: U32 = 2^-24 of float32, HALF[t] of the output's type, each relative
to the value; a subnormal float16 result is off by up to 2^-25.
"""

from __future__ import annotations

import torch

F64 = torch.float64
U32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def order(ids, E, active=None):
    """(counts, offsets, row_of_route, route_of_row) as int32 tensors, by plain Python."""
    T, K = ids.shape
    flat = ids.reshape(-1).tolist()
    of = [[] for _ in range(E)]
    for r, e in enumerate(flat):
        if 0 <= e < E and (active is None or int(active[r // K]) != 0):
            of[e].append(r)
    counts = [len(v) for v in of]
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    route = [r for v in of for r in v]
    row = [-1] * (T * K)
    for p, r in enumerate(route):
        row[r] = p
    route += [-1] * (T * K - len(route))
    i32 = torch.int32
    return (torch.tensor(counts, dtype=i32), torch.tensor(offsets, dtype=i32),
            torch.tensor(row, dtype=i32).view(T, K), torch.tensor(route, dtype=i32))


def rows_of(x, route, K):
    """Rows of x in an order, zeros where no route is; bytes are moved, not computed."""
    out = torch.zeros((route.numel(), x.shape[1]), dtype=x.dtype)
    live = route >= 0
    out[live] = x[route[live].long() // K]
    return out


def combine(rows, row, weights=None, dtype=None):
    """y in 64 bits and the bound on its error: a float32 sum of K terms, one rounding of the result."""
    dtype = rows.dtype if dtype is None else dtype
    T, K = row.shape
    y = torch.zeros((T, rows.shape[1]), dtype=F64)
    mag = torch.zeros_like(y)
    for k in range(K):
        live = row[:, k] >= 0
        v = rows[row[live, k].long()].to(F64)
        if weights is not None:
            v = v * weights[live, k].to(F64)[:, None]
        y[live] += v
        mag[live] += v.abs()
    # K fused additions, each within half a step of a partial sum, which is at most mag
    return y, K * U32 * mag * 1.01 + (y.abs() + K * U32 * mag) * HALF[dtype] + TINY[dtype]


def combine_backward(dy, rows, row, weights):
    """drows, dweights in 64 bits, and the bounds on their errors."""
    T, K = row.shape
    H = rows.shape[1]
    drows = torch.zeros(rows.shape, dtype=F64)
    dw = torch.zeros((T, K), dtype=F64)
    mag = torch.zeros((T, K), dtype=F64)
    for k in range(K):
        live = row[:, k] >= 0
        p, d = row[live, k].long(), dy[live].to(F64)
        drows[p] = d * weights[live, k].to(F64)[:, None]
        dw[live, k] = (d * rows[p].to(F64)).sum(1)
        mag[live, k] = (d * rows[p].to(F64)).abs().sum(1)
    half = HALF[rows.dtype]
    # one float32 product, one rounding to the type; a float32 sum of H products in some order: every product and
    # every addition within half a step of at most mag
    return drows, drows.abs() * (U32 + half) * 1.01 + TINY[rows.dtype], dw, 2 * H * U32 * mag * 1.01
