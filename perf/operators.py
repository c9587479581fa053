"""Cases and plain forms of four operators around the routed-expert path:

* ``router``: a token's experts and their weights from its router scores;
* ``moe_few``: a whole mixture-of-experts layer (router, experts, shared
  expert, combine) for at most 64 tokens, as a decode step runs it;
* ``block_quantize``: bf16 rows to e4m3 codes with one scale per 128 values;
* ``block_matmul``: the product of e4m3 matrices with one scale per 128
  values of an activation row and per 128 x 128 block of a weight, dense or
  over groups of rows (experts), from codes or from bf16 rows.

``own`` False computes each from elementary torch operations in float32 (the
router's scores, whose order decides, in float64); ``own`` True calls the
library.  Weights of an expert layer are in the layout that the expert
kernels read: W1 [E][2I][H] with gate and up rows interleaved in groups of
32, W2 [E][H][I]; scales in formula order (gate rows first).
"""

from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
GROUP = 32           # gate / up interleave of the prepared W1
FLOOR = 1e-8         # smallest quantisation scale
DEV = "cuda"


# ------------------------------------------------------------------- cases

def _router(name, T, H, E, K, scoring, bias, renormalize=True, scale=1.0, off=0, inactive=0.0):
    return {"name": name, "op": "router", "T": T, "H": H, "E": E, "K": K, "scoring": scoring, "bias": bias,
            "renormalize": renormalize, "scale": scale, "off": off, "inactive": inactive}


def _few(name, T, H, I, E, K, weights, y, shared=0, routed=True, scoring="softmax", clamp=0.0, inactive=0.0):
    return {"name": name, "op": "moe_few", "T": T, "H": H, "I": I, "E": E, "K": K, "weights": weights, "y": y,
            "shared": shared, "routed": routed, "scoring": scoring, "clamp": clamp, "inactive": inactive}


def listed():
    return [
        # one decoded token's routes in a 32-expert layer: pure latency
        _router("router_t1", 1, 7168, 32, 8, "softmax", False),
        # a mid-size layer's ragged batch, some tokens inactive, one expert switched off
        _router("router_t333", 333, 4096, 16, 4, "softmax", True, False, 1.0, 1, 0.1),
        # a prefill of 16K tokens over the 256 experts of a whole layer, sigmoid scores with a selection bias
        _router("router_t16384", 16384, 7168, 256, 8, "sigmoid", True, True, 2.5),
        # decode of one sequence, bf16 weights: streams 8 experts
        _few("few_t1_bf16", 1, 7168, 2048, 32, 8, "bf16", "bf16"),
        # the same with block-scaled e4m3 weights and a shared expert
        _few("few_t1_block", 1, 7168, 2048, 32, 8, "block", "bf16", 1, True, "sigmoid"),
        # seven sequences on the mid-size layer, float32 output, clamped activations
        _few("few_t7_mid", 7, 4096, 1408, 16, 4, "bf16", "f32", 0, True, "softmax", 2.5, 0.15),
        # 64 sequences with routes from elsewhere, per-channel e4m3 weights: every expert is read
        _few("few_t64_fp8", 64, 7168, 2048, 32, 8, "fp8", "bf16", 0, False),
        # activations of a decode batch, and of a 16K-token prefill
        {"name": "quantize_64", "op": "block_quantize", "M": 64, "K": 7168},
        {"name": "quantize_16384", "op": "block_quantize", "M": 16384, "K": 7168},
        # a decoded token through one projection, from bf16
        {"name": "linear_m1", "op": "block_matmul", "M": 1, "N": 7168, "K": 2048, "G": 1, "x": "bf16"},
        # a ragged batch through one projection, from bf16
        {"name": "linear_m4097", "op": "block_matmul", "M": 4097, "N": 4096, "K": 7168, "G": 1, "x": "bf16"},
        # the first expert product of a prefill: ragged groups of rows, from codes
        {"name": "grouped_32x512", "op": "block_matmul", "M": 16384, "N": 4096, "K": 7168, "G": 32, "x": "codes"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["router", "moe_few", "moe_few", "block_quantize", "block_matmul", "block_matmul"])
    if op == "router":
        E = _log(rng, 4, 256)
        c = _router("", _log(rng, 1, 16384), 256 * rng.randint(1, 28), E, rng.randint(1, min(8, E - 1)),
                    rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.random() < 0.7,
                    rng.choice([1.0, 2.5]), rng.choice([0, 0, 1]), rng.choice([0.0, 0.1]))
        if not c["bias"]:
            c["off"] = 0
    elif op == "moe_few":
        E = rng.randint(4, 32)
        c = _few("", _log(rng, 1, 64), 256 * rng.randint(1, 28), 128 * rng.randint(1, 16), E, rng.randint(1, min(8, E)),
                 rng.choice(["bf16", "fp8", "block"]), rng.choice(["bf16", "f32"]), rng.choice([0, 1]),
                 rng.random() < 0.7, rng.choice(["softmax", "sigmoid"]), rng.choice([0.0, 2.5]),
                 rng.choice([0.0, 0.15]))
    elif op == "block_quantize":
        c = {"op": op, "M": _log(rng, 1, 16384), "K": 128 * rng.randint(1, 56)}
    else:
        G = rng.choice([1, 1, rng.randint(2, 32)])
        c = {"op": op, "M": _log(rng, 1, 16384), "N": 16 * rng.randint(1, 256), "K": 128 * rng.randint(1, 56), "G": G,
             "x": rng.choice(["bf16", "codes"])}
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _expert_weights(g, fmt, E, N, K):
    """[E][N][K] weights of variance 1/K and their scales (per row, per 128 x 128 block, or none)."""
    w = _randn(g, E, N, K, dtype=torch.bfloat16)
    if fmt == "bf16":
        return w.mul_(K ** -0.5), None
    q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((E, N) if fmt == "fp8" else (E, -(-N // BLOCK), K // BLOCK), device=DEV)
    for e in range(E):
        v = w[e].float() * K ** -0.5
        if fmt == "fp8":
            s[e] = (v.abs().amax(1) / 448.0).clamp_min(FLOOR)
            q[e] = (v / s[e][:, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        else:
            nb = -(-N // BLOCK)
            pad = torch.zeros((nb * BLOCK, K), device=DEV)
            pad[:N] = v
            b = pad.view(nb, BLOCK, K // BLOCK, BLOCK)
            s[e] = (b.abs().amax((1, 3)) / 448.0).clamp_min(FLOOR)
            t = (b / s[e][:, None, :, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
            q[e] = t.view(nb * BLOCK, K)[:N]
    return q, s


def _router_inputs(c, g, H, E):
    w = _randn(g, E, H).mul_(H ** -0.5).to(torch.bfloat16)
    bias = None
    if c.get("bias", False):
        bias = _randn(g, E) * (0.5 if c["scoring"] == "softmax" else 0.1)
        if c["off"]:
            bias[: c["off"]] = -math.inf
    return w, bias


def _active(c, g, T):
    return (torch.rand(T, generator=g, device=DEV) >= c["inactive"]).to(torch.int8) if c["inactive"] > 0 else None


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "router":
        s["x"] = _randn(g, c["T"], c["H"]).to(torch.bfloat16)
        s["wr"], s["bias"] = _router_inputs(c, g, c["H"], c["E"])
        s["active"] = _active(c, g, c["T"])
    elif c["op"] == "moe_few":
        T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
        s["x"] = _randn(g, T, H).to(torch.bfloat16)
        s["active"] = _active(c, g, T)
        s["wr"], s["bias"] = _router_inputs(c, g, H, E)
        s["ids"] = s["wts"] = None
        if not c["routed"]:      # routes of a skewed router, made elsewhere
            z = _randn(g, T, E) + 0.5 * _randn(g, E)
            v, i = z.sort(dim=1, descending=True, stable=True)
            s["ids"], s["wts"] = i[:, :K].to(torch.int32).contiguous(), torch.softmax(v[:, :K], 1).contiguous()
        s["w1"], s["s1"] = _expert_weights(g, c["weights"], E + c["shared"], 2 * I, H)
        s["w2"], s["s2"] = _expert_weights(g, c["weights"], E + c["shared"], H, I)
    elif c["op"] == "block_quantize":
        # rows of different magnitude, as activations have
        s["x"] = (_randn(g, c["M"], c["K"]) * torch.exp(_randn(g, c["M"], 1))).to(torch.bfloat16)
    else:
        M, N, K, G = c["M"], c["N"], c["K"], c["G"]
        x = (_randn(g, M, K) * torch.exp(0.5 * _randn(g, M, 1))).to(torch.bfloat16)
        s["x"] = x
        if c["x"] == "codes":
            s["q"], s["sx"] = _quantize(x)
        w, ws = _expert_weights(g, "block", G, N, K)
        s["w"], s["ws"] = (w, ws) if G > 1 else (w[0], ws[0])
        s["offsets"] = s["counts"] = None
        if G > 1:                # a skewed split of the rows over the groups; a group may be empty
            share = torch.softmax(0.5 * _randn(g, G), 0).cumsum(0)
            end = (share * M).round().to(torch.int32).clamp_(0, M)
            end[-1] = M
            s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), end]).contiguous()
            s["counts"] = (s["offsets"][1:] - s["offsets"][:-1]).contiguous()
            s["most"] = int(s["counts"].max())
    return s


# ------------------------------------------------------------- plain forms

def _quantize(x):
    """e4m3 codes and scales of rows of bf16: s = max(max|group| / 448, 1e-8), q = x / s rounded to nearest even."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    # by a tensor: torch multiplies by the reciprocal of a number, which rounds differently
    s = (v.abs().amax(2) / torch.tensor(448.0, device=DEV).expand(v.shape[:2])).clamp_min(FLOOR)
    return (v / s[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(x.shape), s


def _route(x, wr, bias, K, scoring, renormalize, scale, active):
    z = x.double() @ wr.double().t()
    if scoring == "softmax":
        z = z if bias is None else z + bias.double()
        score, select = torch.softmax(z, 1), z
    else:
        score = torch.sigmoid(z)
        select = z if bias is None else score + bias.double()
    v, ids = select.sort(dim=1, descending=True, stable=True)
    v, ids = v[:, :K], ids[:, :K]
    wts = score.gather(1, ids)
    none = v == -math.inf
    if active is not None:
        none = none | (active == 0)[:, None]
    wts = torch.where(none, 0.0, wts)
    if renormalize:
        wts = wts / (wts.sum(1, keepdim=True) + 1e-20)
    return torch.where(none, -1, ids).to(torch.int32), (wts * scale).float()


def _interleave(s, I):
    """Rows in formula order (I gate rows, I up rows) to the prepared W1's order."""
    return s.view(s.shape[0], 2, I // GROUP, GROUP, *s.shape[2:]).transpose(1, 2).reshape(s.shape)


def _dequantize(w, s, fmt, I=0):
    """float32 weights [E][N][K]; I: W1, whose rows are interleaved and its scales not."""
    w = w.float()
    if fmt == "bf16":
        return w
    if fmt == "fp8":
        return w * (_interleave(s, I) if I else s)[:, :, None]
    s = s.repeat_interleave(BLOCK, 1)[:, : w.shape[1]]
    s = _interleave(s, I) if I else s
    return (w.view(*w.shape[:2], -1, BLOCK) * s[..., None]).view(w.shape)


def _swiglu(h, I, clamp):
    h = h.view(*h.shape[:-1], I // GROUP, 2, GROUP)
    if clamp > 0:
        h = h.clamp(-clamp, clamp)
    g, u = h[..., 0, :], h[..., 1, :]
    return (g * torch.sigmoid(g) * u).reshape(*h.shape[:-3], I)


def _few_plain(s):
    c = s["case"]
    T, I, E, K, S, fmt = c["T"], c["I"], c["E"], c["K"], c["shared"], c["weights"]
    x, ids, wts = s["x"].float(), s["ids"], s["wts"]
    if c["routed"]:
        ids, wts = _route(s["x"], s["wr"], s["bias"], K, c["scoring"], True, 1.0, s["active"])
    on = torch.ones(T, device=DEV) if s["active"] is None else (s["active"] != 0).float()
    e, g = ids.long(), torch.where(ids < 0, 0.0, wts) * on[:, None]
    if S:
        e = torch.cat([e, torch.full((T, 1), E, device=DEV)], 1)
        g = torch.cat([g, on[:, None]], 1)
    e = e.clamp_min(0)
    if e.numel() <= E:           # few routes: only their experts' weights
        j = e.reshape(-1)
        w1 = _dequantize(s["w1"][j], None if fmt == "bf16" else s["s1"][j], fmt, I)
        xr = x.repeat_interleave(e.shape[1], 0)
        a = _swiglu(torch.matmul(w1, xr[:, :, None])[..., 0], I, c["clamp"])
        w2 = _dequantize(s["w2"][j], None if fmt == "bf16" else s["s2"][j], fmt)
        y = torch.matmul(w2, a[:, :, None])[..., 0].view(T, e.shape[1], -1)
        y = (y * g[..., None]).sum(1)
    else:                        # every expert on every token, weighted by the gates
        gate = torch.zeros((T, E + S), device=DEV).scatter_add_(1, e, g)
        w1 = _dequantize(s["w1"], s["s1"], fmt, I)
        h = (x @ w1.view(-1, x.shape[1]).t()).view(T, E + S, 2 * I)
        a = _swiglu(h, I, c["clamp"]).transpose(0, 1).contiguous()
        del w1, h
        w2 = _dequantize(s["w2"], s["s2"], fmt)
        y = (torch.matmul(a, w2.transpose(1, 2).contiguous()) * gate.t()[..., None]).sum(0)
    return (y.to(torch.bfloat16) if c["y"] == "bf16" else y), ids, wts


def _matmul_plain(s):
    c = s["case"]
    q, sx = (s["q"], s["sx"]) if c["x"] == "codes" else _quantize(s["x"])
    x = (q.float().view(c["M"], -1, BLOCK) * sx[:, :, None]).view(c["M"], -1)
    if c["G"] == 1:
        return (x @ _dequantize(s["w"][None], s["ws"][None], "block")[0].t()).to(torch.bfloat16)
    # rows padded to the largest group, one product per group, rows back in place
    at = torch.arange(s["most"], device=DEV)[None, :]
    rows = (s["offsets"][:-1].long()[:, None] + at).clamp_max(c["M"] - 1)
    y = torch.matmul(x[rows], _dequantize(s["w"], s["ws"], "block").transpose(1, 2).contiguous())
    return y[at < s["counts"][:, None]].to(torch.bfloat16)


# --------------------------------------------------------------------- run

def run(state):
    c = state["case"]
    if own:
        from mixture_experts_expert_mm_amd import moe
    if c["op"] == "router":
        if own:
            return moe.route(state["x"], state["wr"], state["bias"], topk=c["K"], scoring=c["scoring"],
                             renormalize=c["renormalize"], scale=c["scale"], active=state["active"])
        return _route(state["x"], state["wr"], state["bias"], c["K"], c["scoring"], c["renormalize"], c["scale"],
                      state["active"])
    if c["op"] == "moe_few":
        if own:
            routes = dict(router_weight=state["wr"], router_bias=state["bias"], topk=c["K"], scoring=c["scoring"]) \
                if c["routed"] else dict(topk_ids=state["ids"], topk_weights=state["wts"])
            return moe.moe_few(state["x"], state["w1"], state["w2"], state["s1"], state["s2"],
                               num_shared_experts=c["shared"], y_dtype=c["y"],
                               activation_clamp=c["clamp"] if c["clamp"] > 0 else None, active=state["active"], **routes)
        return _few_plain(state)
    if c["op"] == "block_quantize":
        q, s = moe.block_quantize(state["x"]) if own else _quantize(state["x"])
        return q.float(), s      # the values that the codes stand for
    if own:
        if c["x"] == "bf16":
            return moe.block_linear(state["x"], state["w"], state["ws"], state["offsets"], state["counts"])
        return moe.block_matmul(state["q"], state["sx"], state["w"], state["ws"], state["offsets"], state["counts"])
    return _matmul_plain(state)


# -------------------------------------------------------------------- work

_WEIGHT = {"bf16": 2.0, "fp8": 1.0, "block": 1.0 + 4.0 / BLOCK ** 2}


def work(case):
    c = case
    if c["op"] == "router":
        T, H, E, K = c["T"], c["H"], c["E"], c["K"]
        return {"bytes": 2 * T * H + 2 * E * H + 8 * T * K, "flops": 2 * T * H * E}
    if c["op"] == "moe_few":
        T, H, I, E, K, S = c["T"], c["H"], c["I"], c["E"], c["K"], c["shared"]
        # experts that T * K evenly spread routes reach
        live = E * (1 - (1 - K / E) ** T) + S
        b = live * 3 * H * I * _WEIGHT[c["weights"]] + 2 * T * H + (2 if c["y"] == "bf16" else 4) * T * H + 8 * T * K
        f = 6 * T * (K + S) * H * I
        if c["routed"]:
            b, f = b + 2 * E * H, f + 2 * T * E * H
        return {"bytes": b, "flops": f}
    M, K = c["M"], c["K"]
    if c["op"] == "block_quantize":
        return {"bytes": M * K * 3 + 4 * M * K // BLOCK, "flops": 3 * M * K}
    N, G = c["N"], c["G"]
    x = 2 * M * K if c["x"] == "bf16" else M * K + 4 * M * K // BLOCK
    return {"bytes": x + min(G, M) * N * K * _WEIGHT["block"] + 2 * M * N, "flops": 2 * M * N * K}


# ------------------------------------------------------------------- exact

def _exact_route(x, wr, bias, K, scoring, renormalize, scale, active):
    """Scores in 64 bits; each token's experts by a sort of (-selection, index) on the host."""
    import numpy as np
    logits = (wr.to(torch.float64) @ x.to(torch.float64).t()).t().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()[None, :]
    if scoring == "softmax":
        sel = logits if b is None else logits + b
        p = np.exp(sel - sel.max(1, keepdims=True))
        score = p / p.sum(1, keepdims=True)
    else:
        score = 1.0 / (1.0 + np.exp(-logits))
        sel = logits if b is None else score + b
    ids = np.argsort(-sel, axis=1, kind="stable")[:, :K]
    w = np.take_along_axis(score, ids, 1)
    gone = np.isneginf(np.take_along_axis(sel, ids, 1))
    if active is not None:
        gone |= (active.cpu().numpy() == 0)[:, None]
    ids, w = np.where(gone, -1, ids), np.where(gone, 0.0, w)
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w * scale)


def _exact_codes(x):
    """Code values and scales in 64 bits.  Both are defined by 32-bit divisions: a 64-bit quotient of 32-bit
    numbers rounds to the same 32 bits, so each is divided in 64 and rounded to 32 before it is used."""
    groups = x.to(torch.float64).reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    scale = (groups.abs().max(2).values / 448).float().double()
    scale = torch.where(scale < FLOOR, torch.tensor(FLOOR, dtype=torch.float32, device=DEV).double(), scale)
    code = (groups / scale.unsqueeze(2)).float()
    code = torch.minimum(torch.maximum(code, code.new_tensor(-448.0)), code.new_tensor(448.0))
    return code.to(torch.float8_e4m3fn).double().reshape(x.shape), scale


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    f64 = torch.float64
    if c["op"] == "router":
        return _exact_route(s["x"], s["wr"], s["bias"], c["K"], c["scoring"], c["renormalize"], c["scale"], s["active"])
    if c["op"] == "block_quantize":
        codes, scale = _exact_codes(s["x"])
        return codes, scale
    if c["op"] == "moe_few":
        T, H, I, E, S = c["T"], c["H"], c["I"], c["E"], c["shared"]
        if c["routed"]:
            ids, wts = _exact_route(s["x"], s["wr"], s["bias"], c["K"], c["scoring"], True, 1.0, s["active"])
        else:
            ids, wts = s["ids"], s["wts"]
        ids, gates = ids.to(DEV), wts.to(DEV, f64)
        x, y = s["x"].to(f64), torch.zeros((T, H), dtype=f64, device=DEV)
        alive = torch.ones(T, dtype=torch.bool, device=DEV) if s["active"] is None else s["active"] != 0
        n = torch.arange(2 * I, device=DEV)
        gate_row = (n // (2 * GROUP)) * GROUP + n % (2 * GROUP)       # formula row of each prepared W1 row
        row = torch.where(n % (2 * GROUP) < GROUP, gate_row, gate_row - GROUP + I)
        for e in range(E + S):
            w = ((ids == e) * gates).sum(1) if e < E else torch.ones(T, dtype=f64, device=DEV)
            w = torch.where(alive, w, 0.0)
            t = ((ids == e).any(1) if e < E else alive).logical_and(alive).nonzero()[:, 0]
            if t.numel() == 0:
                continue
            w1, w2 = s["w1"][e].to(f64), s["w2"][e].to(f64)
            if c["weights"] == "fp8":
                w1, w2 = w1 * s["s1"][e].to(f64)[row, None], w2 * s["s2"][e].to(f64)[:, None]
            elif c["weights"] == "block":
                k1, k2 = torch.arange(H, device=DEV) // BLOCK, torch.arange(I, device=DEV) // BLOCK
                w1 = w1 * s["s1"][e].to(f64)[row // BLOCK][:, k1]
                w2 = w2 * s["s2"][e].to(f64)[torch.arange(H, device=DEV) // BLOCK][:, k2]
            h = torch.empty((t.numel(), 2 * I), dtype=f64, device=DEV)
            h[:, row] = x[t] @ w1.t()
            if c["clamp"] > 0:
                h = h.clamp(-c["clamp"], c["clamp"])
            a = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
            y[t] += w[t, None] * (a @ w2.t())
        return y, ids, wts
    if c["x"] == "codes":
        q, sx = s["q"].to(f64), s["sx"].to(f64)
    else:
        q, sx = _exact_codes(s["x"])
    M, N, K, G = c["M"], c["N"], c["K"], c["G"]
    x = q * sx[:, torch.arange(K, device=DEV) // BLOCK]
    y = torch.empty((M, N), dtype=f64, device=DEV)
    ends = [0, M] if G == 1 else s["offsets"].tolist()
    for i in range(G):
        w, ws = (s["w"], s["ws"]) if G == 1 else (s["w"][i], s["ws"][i])
        wd = w.to(f64) * ws.to(f64)[torch.arange(N, device=DEV) // BLOCK][:, torch.arange(K, device=DEV) // BLOCK]
        y[ends[i]:ends[i + 1]] = x[ends[i]:ends[i + 1]] @ wd.t()
    return y
