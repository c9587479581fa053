"""Cases and plain forms of the operators of an expert layer that is put
together from parts, for serving and for training:

* ``sort``: token rows to rows sorted by expert, and their gradient;
* ``combine``: those rows back to tokens, weighted, and the gradients of the
  rows and of the weights;
* ``int8``: products of 8-bit integers with a scale per token and per channel,
  dense or over groups of rows (experts), from codes or from floating rows;
* ``swiglu``: the activation between the two products, with its input kept in
  8 bits for the backward pass.

``own`` False computes each from elementary torch operations in float32 (order
and codes are decided as the operators define them); ``own`` True calls the
library.
"""

from __future__ import annotations

import math

import torch

own = False

GROUP = 128          # values per scale of an activation kept in 8 bits
FLOOR = 1e-8         # smallest quantisation scale
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def _sort(name, T, H, E, K, dtype, grad=False, inactive=0.0):
    return {"name": name, "op": "sort", "T": T, "H": H, "E": E, "K": K, "dtype": dtype, "grad": grad,
            "inactive": inactive}


def _combine(name, T, H, E, K, dtype, grad=False, weighted=True, inactive=0.0):
    return {"name": name, "op": "combine", "T": T, "H": H, "E": E, "K": K, "dtype": dtype, "grad": grad,
            "weighted": weighted, "inactive": inactive}


def _int8(name, M, N, K, G, x, y="bf16"):
    return {"name": name, "op": "int8", "M": M, "N": N, "K": K, "G": G, "x": x, "y": y}


def _swiglu(name, M, I, dtype, form, clamp=0.0):
    """form: "serve" (the activation alone), "keep" (and the 8-bit copy), "train" (forward and backward)."""
    return {"name": name, "op": "swiglu", "M": M, "I": I, "dtype": dtype, "form": form, "clamp": clamp}


def listed():
    return [
        # one decoded token to its 8 experts: latency
        _sort("sort_t1", 1, 7168, 32, 8, "bf16"),
        # a ragged float32 training batch of a mid-size layer, some tokens inactive, both directions
        _sort("sort_t333_grad", 333, 4096, 16, 4, "f32", True, 0.1),
        # a training step's 16K tokens over the 256 experts of a whole layer
        _sort("sort_t16384_grad", 16384, 7168, 256, 8, "bf16", True),
        # a decode batch back to its tokens
        _combine("combine_t64", 64, 7168, 32, 8, "bf16"),
        # a mid-size layer's training batch in float32, some tokens inactive
        _combine("combine_t2048_grad", 2048, 4096, 16, 4, "f32", True, True, 0.1),
        # the 16K tokens of a training step, back and their gradients
        _combine("combine_t16384_grad", 16384, 7168, 256, 8, "bf16", True),
        # a decoded token through one projection, from bf16
        _int8("int8_m1", 1, 7168, 2048, 1, "bf16"),
        # a ragged prefill through one projection, from bf16
        _int8("int8_m4097", 4097, 4096, 7168, 1, "bf16"),
        # the first expert product of an 8K-token prefill, 8 of 32 experts a token: ragged groups, from codes
        _int8("int8_grouped_65536", 65536, 4096, 7168, 32, "codes"),
        # the 8 routes of one decoded token, nothing kept
        _swiglu("swiglu_m8", 8, 2048, "bf16", "serve"),
        # a ragged batch in half precision, clamped, and what it keeps
        _swiglu("swiglu_m1333_keep", 1333, 1408, "f16", "keep", 2.5),
        # the 64K routes of an 8K-token training step
        _swiglu("swiglu_m65536_train", 65536, 2048, "bf16", "train"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, most):
    """Half of the widths whole vectors, the others anything."""
    return 8 * rng.randint(1, most // 8) if rng.random() < 0.5 else _log(rng, 1, most)


def draw(rng):
    op = rng.choice(["sort", "combine", "int8", "int8", "swiglu"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("sort", "combine"):
        E = _log(rng, 2, 256)
        args = ("", _log(rng, 1, 16384), _width(rng, 3584 if dtype == "f32" else 7168), E, rng.randint(1, min(8, E)), dtype,
                rng.random() < 0.5)
        inactive = rng.choice([0.0, 0.1])
        c = _sort(*args, inactive) if op == "sort" else _combine(*args, rng.random() < 0.8, inactive)
    elif op == "int8":
        G = rng.choice([1, 1, rng.randint(2, 32)])
        c = _int8("", _log(rng, 1, 16384), _width(rng, 4096), 16 * rng.randint(1, 448), G, rng.choice([dtype, "codes"]),
                  rng.choice(["bf16", "bf16", "f16", "f32"]))
    else:
        c = _swiglu("", _log(rng, 1, 32768), _width(rng, 2048), dtype, rng.choice(["serve", "keep", "train"]),
                    rng.choice([0.0, 2.5]))
    c.pop("name")
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _routes(g, c):
    """Experts of a skewed router, distinct within a token, some routes masked; and the active tokens."""
    T, E, K = c["T"], c["E"], c["K"]
    z = _randn(g, T, E) + 0.5 * _randn(g, E)
    ids = z.argsort(dim=1, descending=True)[:, :K].to(torch.int32)
    active = None
    if c["inactive"] > 0:
        ids[torch.rand(T, K, generator=g, device=DEV) < 0.05] = -1
        active = (torch.rand(T, generator=g, device=DEV) >= c["inactive"]).to(torch.int8)
    return ids.contiguous(), active


def _order(ids, E, active):
    """counts, offsets, the row of each route and the route of each row: rows by (expert, route), skipped ones last."""
    T, K = ids.shape
    key = torch.where((ids >= 0) & (ids < E), ids, E)
    if active is not None:
        key = torch.where(active[:, None] != 0, key, E)
    key, route = key.reshape(-1).long().sort(stable=True)
    row = torch.empty_like(route)
    row[route] = torch.arange(T * K, device=DEV)
    bounds = torch.searchsorted(key, torch.arange(E + 1, device=DEV))
    kept = torch.arange(T * K, device=DEV) < bounds[E]
    i32 = torch.int32
    return ((bounds[1:] - bounds[:-1]).to(i32), bounds.to(i32), torch.where(row < bounds[E], row, -1).to(i32).view(T, K),
            torch.where(kept, route, -1).to(i32))


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] in ("sort", "combine"):
        T, H, E, K, dt = c["T"], c["H"], c["E"], c["K"], TYPES[c["dtype"]]
        s["ids"], s["active"] = _routes(g, c)
        if c["op"] == "sort":
            s["x"] = _randn(g, T, H, dtype=dt)
            if c["grad"]:
                s["x"].requires_grad_()
                s["drows"] = _randn(g, T * K, H, dtype=dt)
        else:
            s["order"] = _order(s["ids"], E, s["active"])
            s["rows"] = _randn(g, T * K, H, dtype=dt)
            s["w"] = torch.softmax(_randn(g, T, K), 1) if c["weighted"] else None
            if c["grad"]:
                s["rows"].requires_grad_()
                if c["weighted"]:
                    s["w"].requires_grad_()
                s["dy"] = _randn(g, T, H, dtype=dt)
    elif c["op"] == "int8":
        M, N, K, G = c["M"], c["N"], c["K"], c["G"]
        x = (_randn(g, M, K) * torch.exp(0.5 * _randn(g, M, 1))).to(TYPES.get(c["x"], torch.bfloat16))
        if c["x"] == "codes":
            s["q"], s["sx"] = _codes(x)
        else:
            s["x"] = x
        w = torch.empty((G, N, K), dtype=torch.int8, device=DEV)
        ws = torch.empty((G, N), device=DEV)
        for i in range(G):
            w[i], ws[i] = _codes(_randn(g, N, K) * K ** -0.5)
        s["w"], s["ws"] = (w, ws) if G > 1 else (w[0], ws[0])
        s["offsets"] = s["counts"] = None
        if G > 1:                # a skewed split of the rows over the groups; a group may be empty
            share = torch.softmax(0.5 * _randn(g, G), 0).cumsum(0)
            end = (share * M).round().to(torch.int32).clamp_(0, M)
            end[-1] = M
            s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), end]).contiguous()
            s["counts"] = (s["offsets"][1:] - s["offsets"][:-1]).contiguous()
            s["most"] = int(s["counts"].max())
    else:
        M, I, dt = c["M"], c["I"], TYPES[c["dtype"]]
        # rows of different magnitude, as activations have
        s["h"] = (_randn(g, M, 2 * I) * torch.exp(0.5 * _randn(g, M, 1))).to(dt)
        if c["form"] == "train":
            s["h"].requires_grad_()
            s["da"] = _randn(g, M, I, dtype=dt)
    return s


# ------------------------------------------------------------- plain forms

def _codes(v):
    """Codes and scales along the last dimension: s = max(max|v| / 127, 1e-8), q = v / s rounded half to even."""
    v = v.float()
    m = v.abs().amax(-1)
    # by a tensor: torch multiplies by the reciprocal of a number, which rounds differently
    s = (m / torch.full_like(m, 127.0)).clamp_min(FLOOR)
    return (v / s[..., None]).round().clamp(-127.0, 127.0).to(torch.int8), s


def _keep(h, I):
    """The 8-bit copy of h: each half of a row in groups of 128, the last one filled up with zeros."""
    n = -(-I // GROUP)
    v = torch.zeros((h.shape[0], 2, n * GROUP), device=DEV)
    v[:, :, :I] = h.float().view(-1, 2, I)
    q, s = _codes(v.view(-1, 2, n, GROUP))
    return q.view(-1, 2, n * GROUP)[:, :, :I].reshape(h.shape), s.view(-1, 2 * n)


def _kept(q, s, I):
    """The values that the 8-bit copy stands for: gate and up."""
    v = q.float().view(-1, 2, I) * s.view(s.shape[0], 2, -1).repeat_interleave(GROUP, 2)[:, :, :I]
    return v[:, 0], v[:, 1]


def _swiglu_plain(s):
    c, h = s["case"], s["h"]
    I, clamp = c["I"], c["clamp"] if c["clamp"] > 0 else math.inf
    g, u = h[:, :I].float().clamp(-clamp, clamp), h[:, I:].float().clamp(-clamp, clamp)
    a = (g * torch.sigmoid(g) * u).to(h.dtype)
    if c["form"] == "serve":
        return a
    q, sc = _keep(h, I)
    if c["form"] == "keep":
        return a, q.float(), sc
    g0, u0 = _kept(q, sc, I)
    g, u, da = g0.clamp(-clamp, clamp), u0.clamp(-clamp, clamp), s["da"].float()
    sig = torch.sigmoid(g)
    dg = torch.where(g0.abs() <= clamp, da * u * sig * (1 + g * (1 - sig)), 0.0)
    du = torch.where(u0.abs() <= clamp, da * g * sig, 0.0)
    return a, torch.cat([dg, du], 1).to(h.dtype)


def _sort_plain(s):
    c = s["case"]
    counts, offsets, row, route = _order(s["ids"], c["E"], s["active"])
    rows = torch.where(route[:, None] >= 0, s["x"][route.clamp_min(0).long() // c["K"]], 0.0)
    if not c["grad"]:
        return rows, counts, offsets, row, route
    d = s["drows"][row.clamp_min(0).long()].float()
    return rows, counts, offsets, row, route, torch.where(row[:, :, None] >= 0, d, 0.0).sum(1).to(rows.dtype)


def _combine_plain(s):
    c = s["case"]
    _, _, row, route = s["order"]
    taken = row[:, :, None] >= 0
    r = torch.where(taken, s["rows"][row.clamp_min(0).long()].float(), 0.0)
    y = (r * s["w"][:, :, None] if c["weighted"] else r).sum(1).to(s["rows"].dtype)
    if not c["grad"]:
        return y
    at = route.clamp_min(0).long()
    d = s["dy"][at // c["K"]].float()
    if c["weighted"]:
        d = d * s["w"].reshape(-1)[at][:, None]
    drows = torch.where(route[:, None] >= 0, d, 0.0).to(s["rows"].dtype)
    if not c["weighted"]:
        return y, drows
    return y, drows, (r * s["dy"].float()[:, None, :]).sum(2)


def _int8_plain(s):
    c = s["case"]
    q, sx = (s["q"], s["sx"]) if c["x"] == "codes" else _codes(s["x"])
    x, dt = q.float(), TYPES[c["y"]]
    if c["G"] == 1:
        return ((x @ s["w"].float().t()) * s["ws"] * sx[:, None]).to(dt)
    # rows padded to the largest group, one product per group, rows back in place
    at = torch.arange(s["most"], device=DEV)[None, :]
    rows = (s["offsets"][:-1].long()[:, None] + at).clamp_max(c["M"] - 1)
    y = torch.matmul(x[rows], s["w"].float().transpose(1, 2).contiguous()) * s["ws"][:, None, :] * sx[rows][:, :, None]
    return y[at < s["counts"][:, None]].to(dt)


# --------------------------------------------------------------------- run

def run(state):
    c = state["case"]
    if not own:
        with torch.no_grad():
            return {"sort": _sort_plain, "combine": _combine_plain, "int8": _int8_plain, "swiglu": _swiglu_plain}[c["op"]](state)
    from mixture_experts_expert_mm_amd import moe
    if c["op"] == "sort":
        rows, o = moe.sort_tokens(state["x"], state["ids"], c["E"], active=state["active"])
        out = (rows.detach(), o.counts, o.offsets, o.row_of_route, o.route_of_row)
        return out + torch.autograd.grad(rows, state["x"], state["drows"]) if c["grad"] else out
    if c["op"] == "combine":
        y = moe.combine_tokens(state["rows"], moe.TokenOrder(*state["order"]), state["w"])
        if not c["grad"]:
            return y
        of = (state["rows"], state["w"]) if c["weighted"] else (state["rows"],)
        return (y.detach(),) + torch.autograd.grad(y, of, state["dy"])
    if c["op"] == "int8":
        if c["x"] == "codes":
            return moe.int8_matmul(state["q"], state["sx"], state["w"], state["ws"], state["offsets"], state["counts"],
                                   y_dtype=c["y"])
        return moe.int8_linear(state["x"], state["w"], state["ws"], state["offsets"], state["counts"], y_dtype=c["y"])
    clamp = c["clamp"] if c["clamp"] > 0 else None
    if c["form"] == "keep":
        a, q, s = moe.swiglu_forward(state["h"], activation_clamp=clamp)
        return a, q.float(), s       # the values that the codes stand for
    a = moe.swiglu(state["h"], activation_clamp=clamp)
    if c["form"] == "serve":
        return a
    return (a.detach(),) + torch.autograd.grad(a, state["h"], state["da"])


# -------------------------------------------------------------------- work

def work(case):
    c = case
    b = 4 if c.get("dtype") == "f32" else 2
    if c["op"] in ("sort", "combine"):
        T, H, R = c["T"], c["H"], c["T"] * c["K"]
        rows, tokens = R * H * b, T * H * b
        if c["op"] == "sort":
            n = tokens + rows + 12 * R
            return {"bytes": n + (rows + tokens if c["grad"] else 0), "flops": R * H if c["grad"] else R}
        w = 4 * R if c["weighted"] else 0
        n, f = rows + tokens + 4 * R + w, 2 * R * H
        if c["grad"]:
            n, f = n + rows + tokens + w, f + 3 * R * H
        return {"bytes": n, "flops": f}
    if c["op"] == "int8":
        M, N, K, G = c["M"], c["N"], c["K"], c["G"]
        x = M * K + 4 * M if c["x"] == "codes" else M * K * (4 if c["x"] == "f32" else 2)
        return {"bytes": x + min(G, M) * (N * K + 4 * N) + M * N * (4 if c["y"] == "f32" else 2), "flops": 2 * M * N * K}
    n, I = c["M"] * c["I"], c["I"]
    scales = 8 * c["M"] * -(-I // GROUP)
    if c["form"] == "train":         # the 8-bit copy is written and read again
        return {"bytes": n * (3 * b + 2 + 2 + 3 * b) + 2 * scales, "flops": 30 * n}
    return {"bytes": n * 3 * b + (2 * n + scales if c["form"] == "keep" else 0), "flops": 12 * n}


# ------------------------------------------------------------------- exact

def _exact_order(ids, E, active):
    """The rows' order by a stable sort on the host: (counts, offsets, row of route, route of row) in numpy."""
    import numpy as np
    e = ids.cpu().numpy().astype(np.int64)
    if active is not None:
        e[active.cpu().numpy() == 0] = E
    e[(e < 0) | (e > E)] = E
    flat = e.ravel()
    order = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E + 1)[:E]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    n = int(offsets[-1])
    row = np.full(flat.size, -1, np.int64)
    row[order[:n]] = np.arange(n)
    route = np.full(flat.size, -1, np.int64)
    route[:n] = order[:n]
    return counts, offsets, row.reshape(e.shape), route, n


def _exact_codes(v):
    """Codes and scales in 64 bits.  Both are defined by 32-bit divisions: a 64-bit quotient of 32-bit numbers
    rounds to the same 32 bits, so each is divided in 64 and rounded to 32 before it is used."""
    v = v.to(torch.float64)
    scale = (v.abs().max(-1).values / 127).float().double()
    scale = torch.where(scale < FLOOR, torch.tensor(FLOOR, dtype=torch.float32, device=DEV).double(), scale)
    code = torch.round((v / scale.unsqueeze(-1)).float().double())
    return torch.minimum(torch.maximum(code, code.new_tensor(-127.0)), code.new_tensor(127.0)), scale


def _exact_swiglu(s, c):
    I, h = c["I"], s["h"].detach().to(torch.float64)
    lim = c["clamp"] if c["clamp"] > 0 else math.inf
    gate, up = h[:, :I].clamp(-lim, lim), h[:, I:].clamp(-lim, lim)
    a = gate / (1 + torch.exp(-gate)) * up
    if c["form"] == "serve":
        return a
    codes, scales, values = torch.empty_like(h), [], torch.empty_like(h)
    for half in (0, I):
        for at in range(half, half + I, GROUP):
            end = min(at + GROUP, half + I)
            codes[:, at:end], sc = _exact_codes(h[:, at:end])
            values[:, at:end] = (codes[:, at:end] * sc[:, None]).float().double()   # kept values are float32 products
            scales.append(sc)
    if c["form"] == "keep":
        return a, codes, torch.stack(scales, 1)
    g0, u0 = values[:, :I], values[:, I:]
    g, u, da = g0.clamp(-lim, lim), u0.clamp(-lim, lim), s["da"].to(torch.float64)
    e = torch.exp(-g)
    dg = da * u * (1 + e + g * e) / (1 + e) ** 2         # the derivative of g / (1 + e^-g)
    du = da * g / (1 + e)
    return a, torch.cat([dg * (g0.abs() <= lim), du * (u0.abs() <= lim)], 1)


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    f64 = torch.float64
    with torch.no_grad():
        if c["op"] in ("sort", "combine"):
            T, H, K = c["T"], c["H"], c["K"]
            counts, offsets, row, route, n = _exact_order(s["ids"], c["E"], s["active"])
            order = tuple(torch.from_numpy(v).to(torch.int32) for v in (counts, offsets, row, route))
            kept = torch.from_numpy(route[:n]).to(DEV)
            if c["op"] == "sort":
                rows = torch.zeros((T * K, H), dtype=f64, device=DEV)
                rows[:n] = s["x"].to(f64)[kept // K]
                if not c["grad"]:
                    return (rows,) + order
                dx = torch.zeros((T, H), dtype=f64, device=DEV)
                dx.index_add_(0, kept // K, s["drows"][:n].to(f64))
                return (rows,) + order + (dx,)
            w = s["w"].reshape(-1)[kept].to(f64) if c["weighted"] else torch.ones(n, dtype=f64, device=DEV)
            r = s["rows"][:n].to(f64)
            y = torch.zeros((T, H), dtype=f64, device=DEV)
            y.index_add_(0, kept // K, r * w[:, None])
            if not c["grad"]:
                return y
            d = s["dy"].to(f64)[kept // K]
            drows = torch.zeros((T * K, H), dtype=f64, device=DEV)
            drows[:n] = d * w[:, None]
            if not c["weighted"]:
                return y, drows
            dw = torch.zeros(T * K, dtype=f64, device=DEV)
            dw[kept] = (d * r).sum(1)
            return y, drows, dw.view(T, K)
        if c["op"] == "swiglu":
            return _exact_swiglu(s, c)
        M, N, G = c["M"], c["N"], c["G"]
        if c["x"] == "codes":
            q, sx = s["q"].to(f64), s["sx"].to(f64)
        else:
            q, sx = _exact_codes(s["x"])
        y = torch.empty((M, N), dtype=f64, device=DEV)
        ends = [0, M] if G == 1 else s["offsets"].tolist()
        for i in range(G):
            w, ws = (s["w"], s["ws"]) if G == 1 else (s["w"][i], s["ws"][i])
            lo, hi = ends[i], ends[i + 1]
            y[lo:hi] = (q[lo:hi] @ w.to(f64).t()) * (sx[lo:hi, None] * ws.to(f64)[None, :])
        return y
