"""Device-memory plumbing around the C ABI (torch allocates, the library computes).

``ExpertLayer`` holds one plan, the prepared expert weights and a
workspace, and calls the C-ABI entry points through ``binding``.  The
functions ``route``, ``moe_few``, ``block_quantize``, ``block_matmul`` and
``block_linear`` hold nothing: each checks its tensors, allocates the
outputs and a workspace on the calling stream and makes one call.  So do
``sort_tokens``, ``sort_rows``, ``combine_tokens``, ``combine_backward``,
``swiglu``, ``swiglu_forward``, ``swiglu_backward``, ``int8_quantize``,
``int8_matmul`` and ``int8_linear``; sort_tokens, sort_rows, combine_tokens and
swiglu are differentiable.  Nothing here computes any part of the expert path.
"""

from __future__ import annotations

import contextlib
import dataclasses
import functools
import operator

import torch
import torch.autograd.forward_ad as forward_ad

from . import binding as B

_DT = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8, "mxfp8": torch.uint8,
       "mxfp4": torch.uint8}
MX = ("mxfp8", "mxfp4")


def _y_dtype(plan):
    """The type in which the plan's kernels write y, however the caller spelled it."""
    return torch.float32 if plan.prob.y_dtype == B.MM_OUT_F32 else torch.bfloat16


@dataclasses.dataclass
class Intermediates:
    expert_counts: torch.Tensor
    expert_offsets: torch.Tensor
    pool_src: torch.Tensor
    route_to_pool: torch.Tensor
    x_pool: torch.Tensor
    x_pool_scale: torch.Tensor | None
    a_pool: torch.Tensor
    a_pool_scale: torch.Tensor | None


class ExpertLayer:
    def __init__(self, T, H, I, E, K, usecase="bf16", y_dtype="bf16", device="cuda", activation_clamp=None,
                 num_shared_experts=0):
        self.T, self.H, self.I, self.E, self.K = T, H, I, E, K
        self.S = int(num_shared_experts)
        self.Et, self.Ks = E + self.S, K + self.S      # experts with weights; slots per token
        self.usecase = usecase
        self.y_dtype = y_dtype
        self.device = torch.device(device)
        self.plan = B.mm_plan_create(T, H, I, E, K, usecase, y_dtype, activation_clamp, self.S)
        self.w1 = self.w2 = self.s1 = self.s2 = None
        self._ws = None
        self._fused_ws = None

    # ---------------------------------------------------------------- weights
    def load_weights(self, w1, w2, s1=None, s2=None, stream=None):
        """Upload formula-layout weights ([E+S,H,2I], [E+S,I,H]; a shared expert last; e2m1 packed two per
        byte along the last dimension) and relayout them once.  Scales: float32 per output channel (A8W8)
        or E8M0 bytes [E+S][N][K_in/32] (MX)."""
        dt = _DT[self.usecase]
        w1d = w1.to(self.device).contiguous()
        w2d = w2.to(self.device).contiguous()
        assert w1d.dtype == dt and w2d.dtype == dt
        Et = self.Et
        half = 2 if self.usecase == "mxfp4" else 1
        assert tuple(w1d.shape) == (Et, self.H, 2 * self.I // half) and tuple(w2d.shape) == (Et, self.I, self.H // half)
        self.w1 = torch.empty((Et, 2 * self.I, self.H // half), dtype=dt, device=self.device)
        self.w2 = torch.empty((Et, self.H, self.I // half), dtype=dt, device=self.device)
        B.mm_prepare_weights(self.plan, w1d, w2d, self.w1, self.w2, stream)
        if self.usecase in MX:
            assert tuple(s1.shape) == (Et, 2 * self.I, self.H // 32) and tuple(s2.shape) == (Et, self.H, self.I // 32)
            self.s1 = s1.to(self.device, torch.uint8).contiguous()
            self.s2 = s2.to(self.device, torch.uint8).contiguous()
        elif self.usecase != "bf16":
            self.s1 = s1.to(self.device, torch.float32).contiguous()
            self.s2 = s2.to(self.device, torch.float32).contiguous()
        torch.cuda.current_stream(self.device).synchronize() if stream is None else None
        del w1d, w2d

    # -------------------------------------------------------------- buffers
    def workspace(self, fused: bool) -> torch.Tensor:
        n = self.plan.fused_workspace_bytes if fused else self.plan.workspace_bytes
        attr = "_fused_ws" if fused else "_ws"
        ws = getattr(self, attr)
        if ws is None or ws.numel() < n:
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
            setattr(self, attr, ws)
        return ws

    def new_intermediates(self) -> Intermediates:
        P, dev = self.plan.pool_rows, self.device
        q = self.usecase != "bf16"
        es = 2 if self.usecase == "bf16" else 1
        i32 = dict(dtype=torch.int32, device=dev)
        return Intermediates(
            expert_counts=torch.empty(self.Et, **i32),
            expert_offsets=torch.empty(self.Et + 1, **i32),
            pool_src=torch.empty(P, **i32),
            route_to_pool=torch.empty(self.T * self.Ks, **i32),
            x_pool=torch.empty(P * self.H * es, dtype=torch.uint8, device=dev),
            x_pool_scale=self._scale_buf(self.plan.x_pool_scale_bytes) if q else None,
            a_pool=torch.empty(P * self.I * es, dtype=torch.uint8, device=dev),
            a_pool_scale=self._scale_buf(self.plan.a_pool_scale_bytes) if q else None,
        )

    def _scale_buf(self, nbytes):
        """float32 [P] (A8W8) or E8M0 bytes [P][K_in/32] (MX) of a pool."""
        if self.usecase in MX:
            return torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return torch.empty(nbytes // 4, dtype=torch.float32, device=self.device)

    def new_y(self):
        return torch.empty((self.T, self.H), dtype=_y_dtype(self.plan), device=self.device)

    # -------------------------------------------------------------- entries
    def forward(self, x, topk_ids, topk_weights, y=None, counts=None, stream=None, active=None):
        """mega_moe: returns (y, expert_token_nums).  active: int8 [T] x_active_mask or None."""
        y = self.new_y() if y is None else y
        counts = torch.empty(self.E, dtype=torch.int32, device=self.device) if counts is None else counts
        B.mega_moe(self.plan, x, topk_ids, topk_weights, active, self.w1, self.s1, self.w2, self.s2, y, counts,
                   self.workspace(True), stream)
        return y, counts

    def fused_layout(self):
        """Dispatch metadata the last forward() built in its workspace: (offsets, pool_src, route_to_pool)."""
        i32 = dict(dtype=torch.int32, device=self.device)
        off = torch.empty(self.Et + 1, **i32)
        psrc = torch.empty(self.plan.pool_rows, **i32)
        r2p = torch.empty(self.T * self.Ks, **i32)
        B.mm_debug_fused_layout(self.plan, self.workspace(True), off, psrc, r2p)
        return off, psrc, r2p

    def device_error(self, fused: bool = True) -> int:
        """The device error word of the last call on this layer's workspace
        (mm_device_error bits; waits for the device)."""
        return B.mm_read_device_error(self.plan, self.workspace(fused))

    def dispatch(self, x, topk_ids, im: Intermediates, stream=None, active=None):
        B.mm_dispatch_layout(self.plan, topk_ids, active, x, im.expert_counts, im.expert_offsets, im.pool_src,
                             im.route_to_pool, im.x_pool, im.x_pool_scale, self.workspace(False), stream)

    def linear1(self, im: Intermediates, stream=None):
        B.mm_grouped_l1_swiglu(self.plan, im.expert_offsets, im.expert_counts, im.x_pool, im.x_pool_scale,
                               self.w1, self.s1, im.a_pool, im.a_pool_scale, self.workspace(False), stream)

    def linear2_combine(self, im: Intermediates, topk_weights, y, stream=None):
        B.mm_grouped_l2_combine(self.plan, im.expert_offsets, im.expert_counts, im.pool_src, im.route_to_pool,
                                im.a_pool, im.a_pool_scale, self.w2, self.s2, topk_weights, y,
                                self.workspace(False), stream)

    def forward_3call(self, x, topk_ids, topk_weights, stream=None, active=None):
        im = self.new_intermediates()
        y = self.new_y()
        self.dispatch(x, topk_ids, im, stream, active)
        self.linear1(im, stream)
        self.linear2_combine(im, topk_weights, y, stream)
        return y, im

    def forward_few(self, x, topk_ids, topk_weights, y=None, stream=None, active=None):
        """mm_moe_few on this layer's weights (bf16 or fp8): y [T,H] of at most 64 tokens, however many the
        layer's plan was made for.  Activations are not quantised."""
        if self.usecase not in ("bf16", "fp8"):
            raise ValueError(f"forward_few takes bf16 or fp8 weights, not {self.usecase}")
        clamp = self.plan.prob.activation_clamp if self.plan.prob.clamp_activation else None
        return moe_few(x, self.w1, self.w2, self.s1, self.s2, topk_ids=topk_ids, topk_weights=topk_weights,
                       num_shared_experts=self.S, activation_clamp=clamp, y_dtype=self.plan.prob.y_dtype,
                       active=active, y=y, stream=stream)[0]


# ------------------------------------------------- operators without a layer

_router_plan = functools.lru_cache(maxsize=256)(B.mm_router_plan_create)
_few_plan = functools.lru_cache(maxsize=256)(B.mm_few_plan_create)
_block_plan = functools.lru_cache(maxsize=256)(B.mm_block_plan_create)

FEW_MAX_TOKENS = 64


_VEC = 16


def _need(name, t, dtype, shape, device, grad=False, at=1):
    """The one check of a tensor argument: a message that says what it has to be.  grad: the operator has a gradient
    with respect to it.  at: the number of bytes of which its address is a multiple (_VEC where it is read or written in
    whole vectors)."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()
            and (at == 1 or t.data_ptr() % at == 0) and forward_ad._current_level < 0 and (grad or not t.requires_grad)):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor {list(shape)} on {device} is needed, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))
    if t.data_ptr() % at:
        raise ValueError(f"{name}: its address has to be a multiple of {at} bytes, which a part of another tensor may not "
                         f"begin at (clone it)")
    if t.requires_grad and not grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, which this operator does not compute (call it under no_grad)")
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name}: carries a tangent, which this operator does not compute")


def _apart(y, *inputs):
    """y shares no byte with the inputs, which workgroups read while others write y."""
    lo = y.data_ptr()
    hi = lo + y.nbytes
    for t in inputs:
        if t is not None and t.data_ptr() < hi and lo < t.data_ptr() + t.nbytes:
            raise ValueError("y: overlaps an input that is read while y is written")


def _whole(name, n):
    try:
        return operator.index(int(n) if isinstance(n, float) and n.is_integer() else n)
    except TypeError:
        raise ValueError(f"{name}: a whole number is needed, got {n!r}") from None


def _rows(name, x):
    """(rows, columns, device) of a bf16 or e4m3 matrix on a GPU."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name}: a matrix is needed")
    if not x.is_cuda:
        raise ValueError(f"{name}: a tensor on a GPU is needed, got one on {x.device}")
    rows, columns = x.shape
    return rows, columns, x.device


def _stream_of(device, stream):
    """Context in which outputs are allocated and kernels launched: the device of the inputs and, if one is given,
    the stream, so that the allocator knows who uses the buffers."""
    if stream is not None:
        if getattr(stream, "device", device) != device:
            raise ValueError(f"stream: one of {device} is needed, got one of {stream.device}")
        if isinstance(stream, int):        # a raw handle; ExternalStream takes 0 for none given
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        return torch.cuda.stream(stream)
    if device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return _HERE


_HERE = contextlib.nullcontext()


def _raw_stream(device):
    """The device's current stream as the C ABI takes it (a Stream object costs more than the launches)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(n, device):
    # a fresh buffer for every call: two streams, or two captured graphs, never share one
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


def route(x, weight, bias=None, *, topk, scoring="softmax", renormalize=True, scale=1.0, active=None, stream=None):
    """mm_router: (topk_ids int32 [T,K], topk_weights float32 [T,K]) of the tokens x (bf16 [T,H]).

    weight: bf16 [E,H]; bias: float32 [E] or None (softmax: added to the scores; sigmoid: to their ranking);
    active: int8 [T] or None.  Ids are in descending rank, -1 where no expert is left or the token is inactive."""
    T, H, dev = _rows("x", x)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight: a matrix [experts, hidden] is needed")
    E = weight.shape[0]
    _need("x", x, torch.bfloat16, (T, H), dev, at=_VEC)
    _need("weight", weight, torch.bfloat16, (E, H), dev, at=_VEC)
    if bias is not None:
        _need("bias", bias, torch.float32, (E,), dev)
    if active is not None:
        _need("active", active, torch.int8, (T,), dev)
    if scoring not in B.SCORING:
        raise ValueError(f"scoring: one of {sorted(B.SCORING)}, got {scoring!r}")
    K = _whole("topk", topk)
    plan = _router_plan(max(T, 1), H, E, K, scoring, bool(renormalize), float(scale))
    with _stream_of(dev, stream):
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
        wts = torch.empty((T, K), dtype=torch.float32, device=dev)
        if T:
            B.mm_router(plan, x, weight, bias, active, ids, wts, _workspace(plan.workspace_bytes, dev), _raw_stream(dev))
    return ids, wts


def moe_few(x, w1, w2, s1=None, s2=None, *, topk_ids=None, topk_weights=None, router_weight=None, router_bias=None,
            topk=None, scoring="softmax", renormalize=True, route_scale=1.0, num_shared_experts=0,
            activation_clamp=None, y_dtype="bf16", active=None, y=None, stream=None):
    """The whole layer for at most 64 tokens: (y, topk_ids, topk_weights).

    x: bf16 [T,H].  w1 [E+S,2I,H] and w2 [E+S,H,I] are prepared weights (``ExpertLayer.w1``, ``.w2``), bf16, or
    e4m3 with float32 scales in formula order: per output channel (s1 [E+S,2I], s2 [E+S,H]) or per block of 128 x 128
    (s1 [E+S,2I/128,H/128], s2 [E+S,H/128,I/128]).  y_dtype: "bf16" or "f32".  Routes: topk_ids and topk_weights, or router_weight (with
    router_bias, topk, scoring, renormalize and route_scale as in ``route``).  A shared expert is the last of w1, w2.  y
    may be x, but must not overlap another input."""
    T, H, dev = _rows("x", x)
    if T > FEW_MAX_TOKENS:
        raise ValueError(f"x: at most {FEW_MAX_TOKENS} tokens, got {T} (ExpertLayer.forward takes more)")
    S = _whole("num_shared_experts", num_shared_experts)
    if not isinstance(w1, torch.Tensor) or w1.dim() != 3 or w1.shape[1] % 2:
        raise ValueError("w1: prepared weights [experts, 2 * intermediate, hidden] are needed")
    Et, I = w1.shape[0], w1.shape[1] // 2
    E = Et - S
    if w1.dtype == torch.bfloat16:
        fmt = "bf16"
    elif w1.dtype == torch.float8_e4m3fn:
        fmt = "fp8_block" if isinstance(s1, torch.Tensor) and s1.dim() == 3 else "fp8"
    else:
        raise ValueError(f"w1: bf16 or float8_e4m3fn weights are needed, got {w1.dtype}")
    _need("x", x, torch.bfloat16, (T, H), dev, at=_VEC)
    _need("w1", w1, w1.dtype, (Et, 2 * I, H), dev, at=_VEC)
    _need("w2", w2, w1.dtype, (Et, H, I), dev, at=_VEC)
    if fmt == "bf16":
        if s1 is not None or s2 is not None:
            raise ValueError("s1, s2: bf16 weights have no scales")
    else:
        _need("s1", s1, torch.float32, (Et, 2 * I) if fmt == "fp8" else (Et, 2 * I // 128, H // 128), dev, at=_VEC)
        _need("s2", s2, torch.float32, (Et, H) if fmt == "fp8" else (Et, H // 128, I // 128), dev, at=_VEC)
    if active is not None:
        _need("active", active, torch.int8, (T,), dev)
    routed = router_weight is not None
    if routed == (topk_ids is not None) or (topk_ids is None) != (topk_weights is None):
        raise ValueError("routes: either topk_ids and topk_weights, or router_weight")
    if routed:
        if topk is None:
            raise ValueError("topk: needed with router_weight")
        if not isinstance(router_weight, torch.Tensor) or tuple(router_weight.shape) != (E, H):
            raise ValueError(f"router_weight: [{E}, {H}] is needed")
        K = _whole("topk", topk)
    else:
        K = int(topk_ids.shape[1]) if isinstance(topk_ids, torch.Tensor) and topk_ids.dim() == 2 else 0
        _need("topk_ids", topk_ids, torch.int32, (T, K), dev)
        _need("topk_weights", topk_weights, torch.float32, (T, K), dev)
    plan = _few_plan(max(T, 1), H, I, E, K, fmt, y_dtype, activation_clamp, S)
    ydt = _y_dtype(plan)
    if y is not None:
        _need("y", y, ydt, (T, H), dev, at=_VEC)
        _apart(y, w1, w2, s1, s2, topk_ids, topk_weights, active)      # (x has been read by then)
    with _stream_of(dev, stream):
        if y is None:
            y = torch.empty((T, H), dtype=ydt, device=dev)
        if routed:
            topk_ids, topk_weights = route(x, router_weight, router_bias, topk=K, scoring=scoring,
                                           renormalize=renormalize, scale=route_scale, active=active)
        if T:
            B.mm_moe_few(plan, x, topk_ids, topk_weights, active, w1, s1, w2, s2, y,
                         _workspace(plan.workspace_bytes, dev), _raw_stream(dev))
    return y, topk_ids, topk_weights


def block_quantize(x, stream=None):
    """mm_block_quantize: (codes float8_e4m3fn [M,K], scales float32 [M,K/128]) of bf16 rows."""
    M, K, dev = _rows("x", x)
    _need("x", x, torch.bfloat16, (M, K), dev, at=_VEC)
    if K % 128 or K == 0:
        raise ValueError(f"x: the columns have to be a multiple of 128, got {K}")
    with _stream_of(dev, stream):
        q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
        s = torch.empty((M, K // 128), dtype=torch.float32, device=dev)
        if M:
            B.mm_block_quantize(M, K, x, q, s, _raw_stream(dev))
    return q, s


def _group_args(G, offsets, counts, dev):
    if (offsets is None) != (counts is None) or (offsets is None and G > 1):
        raise ValueError("offsets, counts: both are needed, or neither with one matrix")
    if offsets is not None:
        n = offsets.shape[0] if isinstance(offsets, torch.Tensor) and offsets.dim() == 1 else -1
        _need("offsets", offsets, torch.int32, (n if n == G + 1 else G,), dev)
        _need("counts", counts, torch.int32, (G,), dev)


def _block_args(M, K, dev, rows, w, ws, offsets, counts, y):
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w: [out, in] or [groups, out, in] is needed")
    G, N = (1, w.shape[0]) if w.dim() == 2 else (w.shape[0], w.shape[1])
    lead = () if w.dim() == 2 else (G,)
    _need("w", w, torch.float8_e4m3fn, lead + (N, K), dev, at=_VEC)
    _need("ws", ws, torch.float32, lead + (-(-N // 128), K // 128), dev)
    _group_args(G, offsets, counts, dev)
    if y is not None:
        _need("y", y, torch.bfloat16, (M, N), dev, at=_VEC)
        _apart(y, *rows, w, ws, offsets, counts)
    return N, _block_plan(max(M, 1), N, K, G)


def block_matmul(q, s, w, ws, offsets=None, counts=None, y=None, stream=None):
    """mm_block_gemm: y bf16 [M,N] of e4m3 rows (q [M,K], s [M,K/128]) and weights (w [N,K], ws [ceil(N/128),K/128]),
    or, with w [G,N,K] and ws [G,...], of groups of rows: group g covers rows offsets[g] .. offsets[g] + counts[g]
    (int32; offsets may have G + 1 entries).  Rows that no group covers are left as they are (in a new y: unset).  y
    must not overlap an input."""
    M, K, dev = _rows("q", q)
    _need("q", q, torch.float8_e4m3fn, (M, K), dev, at=_VEC)
    _need("s", s, torch.float32, (M, K // 128), dev)
    N, plan = _block_args(M, K, dev, (q, s), w, ws, offsets, counts, y)
    with _stream_of(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if M:
            B.mm_block_gemm(plan, q, s, w, ws, offsets, counts, y, _raw_stream(dev))
    return y


def block_linear(x, w, ws, offsets=None, counts=None, y=None, stream=None):
    """mm_block_linear: block_matmul of x's (bf16 [M,K]) codes and scales, in one call.  y may overlap x."""
    M, K, dev = _rows("x", x)
    _need("x", x, torch.bfloat16, (M, K), dev, at=_VEC)
    N, plan = _block_args(M, K, dev, (), w, ws, offsets, counts, y)
    with _stream_of(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if M:
            B.mm_block_linear(plan, x, w, ws, offsets, counts, y, _workspace(plan.workspace_bytes, dev), _raw_stream(dev))
    return y


# ----------------------------------------------------------- sorted tokens

_sort_plan = functools.lru_cache(maxsize=256)(B.mm_sort_plan_create)


@dataclasses.dataclass
class TokenOrder:
    """Where the routes' rows lie: experts ascending, an expert's rows in the order of their routes t * K + k.

    counts int32 [E]; offsets int32 [E+1], their exclusive prefix (expert e has the rows offsets[e] .. offsets[e + 1]);
    row_of_route int32 [T,K], -1 for a skipped route; route_of_row int32 [T*K], -1 behind the last row."""
    counts: torch.Tensor
    offsets: torch.Tensor
    row_of_route: torch.Tensor
    route_of_row: torch.Tensor


def _element(name, x, summed):
    el = B.ELEMENT.get(x.dtype)
    if el is None or (summed and el == B.MM_ELEMENT_8BIT):
        raise ValueError(f"{name}: bf16, float16 or float32" + ("" if summed else ", or 8-bit codes,") +
                         f" are needed, got {x.dtype}")
    return el


def _order_of(order, device):
    """(T, E, K) of an order, of which what kernels read (offsets, row_of_route) is as it has to be."""
    if not isinstance(order, TokenOrder):
        raise ValueError(f"order: a TokenOrder is needed, got {type(order).__name__}")
    row, offsets = order.row_of_route, order.offsets
    if not isinstance(row, torch.Tensor) or row.dim() != 2:
        raise ValueError("order.row_of_route: a matrix [tokens, topk] is needed")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1:
        raise ValueError("order.offsets: a vector [experts + 1] is needed")
    T, K = row.shape
    E = offsets.shape[0] - 1
    _need("order.offsets", offsets, torch.int32, (E + 1,), device)
    _need("order.row_of_route", row, torch.int32, (T, K), device)
    return T, E, K


def _records(a, b=None):
    """Whether autograd records this call.  Under capture it may not: the engine ends the process where an eager graph
    of the same leaves is alive, which cannot be seen from here."""
    if not (a.requires_grad or (b is not None and b.requires_grad)) or not torch.is_grad_enabled():
        return False
    _not_captured()
    return True


def _not_captured():
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("autograd under stream capture: call the operators under no_grad and their backward "
                           "functions instead")


def _dense(t):
    """A gradient as autograd hands it over (expanded, strided, at any address) in the form that kernels take."""
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() % _VEC else t


def _sort_rows(x, offsets, row_of_route, T, E, K):
    H = x.shape[1]
    rows = torch.empty((T * K, H), dtype=x.dtype, device=x.device)
    if T:
        plan = _sort_plan(T, H, E, K, B.ELEMENT[x.dtype])
        B.mm_sort_rows(plan, x, offsets, row_of_route, rows, _raw_stream(x.device))
    return rows


def _combine(rows, row_of_route, weights, T, E, K):
    H = rows.shape[1]
    y = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
    if T:
        plan = _sort_plan(T, H, E, K, B.ELEMENT[rows.dtype])
        B.mm_combine_tokens(plan, rows, row_of_route, weights, y, _raw_stream(rows.device))
    return y


def _combine_backward(dy, rows, offsets, row_of_route, weights, T, E, K, of_rows, of_weights):
    H, dev = dy.shape[1], dy.device
    drows = torch.empty((T * K, H), dtype=dy.dtype, device=dev) if of_rows else None
    dweights = torch.empty((T, K), dtype=torch.float32, device=dev) if of_weights else None
    if T and (of_rows or of_weights):
        plan = _sort_plan(T, H, E, K, B.ELEMENT[dy.dtype])
        B.mm_combine_backward(plan, dy, rows if of_weights else None, offsets, row_of_route, weights, drows, dweights,
                              _raw_stream(dev))
    return drows, dweights


def _once(backward):
    """once_differentiable, whose wrapping costs more than a launch, where the backward pass is recorded itself."""
    recorded = torch.autograd.function.once_differentiable(backward)
    return lambda ctx, *grads: recorded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)


def _keep(ctx, *tensors):
    """Saves tensors for the backward pass: they themselves, since the caller's TokenOrder may hold others by then."""
    ctx.save_for_backward(*tensors)
    ctx.kept = [(t.dtype, t.nbytes, True, t.get_device()) for t in tensors]


def _kept(ctx, *names):
    """What _keep saved, looked at again: data exchanged under a tensor, or by a hook of saved tensors, is not noticed by
    autograd, and the kernels would read past its end."""
    try:
        tensors = ctx.saved_tensors
    except RuntimeError as e:
        if "inplace operation" not in str(e):
            raise
        raise RuntimeError(f"{', '.join(names)}: one of them was modified in place before the backward pass") from e
    if [(t.dtype, t.nbytes, t.is_contiguous(), t.get_device()) for t in tensors] != ctx.kept:
        what = ", ".join(f"{n} {t.dtype} {list(t.shape)} on {t.device}" for n, t in zip(names, tensors))
        raise RuntimeError(f"{what}: what the forward call was given is needed, but one of them was exchanged")
    return tensors


def _savable(t):
    """t, or a copy of one that was made in inference mode, which autograd does not save."""
    return t.clone() if t.is_inference() else t


class _SortFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, args, made):
        """made: an order to sort by, or nothing yet, which args then make."""
        ctx.dims = args[-3:]
        if made:
            rows = _sort_rows(x, made[0].offsets, made[0].row_of_route, *ctx.dims)
        else:
            rows, order = _sort_tokens(x, *args)
            made.append(order)
        _keep(ctx, _savable(made[0].row_of_route))
        return rows

    @staticmethod
    @_once
    def backward(ctx, drows):
        _not_captured()
        return _combine(_dense(drows), *_kept(ctx, "row_of_route"), None, *ctx.dims), None, None


class _CombineFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, order, dims):
        ctx.dims = dims
        kept = () if weights is None else (weights, rows) if weights.requires_grad else (weights,)
        _keep(ctx, _savable(order.offsets), _savable(order.row_of_route), *kept)
        return _combine(rows, order.row_of_route, weights, *dims)

    @staticmethod
    @_once
    def backward(ctx, dy):
        _not_captured()
        dy = _dense(dy)
        of_rows, of_weights, _, _ = ctx.needs_input_grad
        offsets, row, *saved = _kept(ctx, "offsets", "row_of_route", "weights", "rows")
        if not saved:
            return _sort_rows(dy, offsets, row, *ctx.dims), None, None, None
        weights, rows = saved if of_weights else (saved[0], None)
        return *_combine_backward(dy, rows, offsets, row, weights, *ctx.dims, of_rows, of_weights), None, None


def _sort_tokens(x, topk_ids, active, plan, T, E, K):
    R, dev = T * K, x.device
    rows = torch.empty((R, x.shape[1]), dtype=x.dtype, device=dev)
    # one allocation for the four, each with a version of its own: what a program writes into one (counts of several
    # batches summed up, say) is no change of another, which the backward pass reads
    buffer = (torch.empty if T else torch.zeros)(2 * (E + R) + 1, dtype=torch.int32, device=dev)
    counts, offsets, row, route = torch.unsafe_split_with_sizes(buffer, (E, E + 1, R, R))
    if T:
        ws = _workspace(plan.workspace_bytes, dev) if plan.workspace_bytes else None
        B.mm_sort_tokens(plan, topk_ids, active, x, counts, offsets, row, route, rows, ws, _raw_stream(dev))
    return rows, TokenOrder(counts, offsets, row.view(T, K), route)


def sort_tokens(x, topk_ids, num_experts, *, active=None, stream=None):
    """mm_sort_tokens: (rows [T*K,H], TokenOrder) of the tokens x [T,H] (bf16, float16, float32, or 8-bit codes).

    topk_ids: int32 [T,K]; a route with an id outside [0, num_experts), or of a token whose entry of active (int8 [T])
    is 0, is skipped.  Row p is the token of route ``order.route_of_row[p]``; rows behind the last one are 0.
    Differentiable with respect to x; the gradient is ``combine_tokens(drows, order)``."""
    T, H, dev = _rows("x", x)
    el = _element("x", x, False)
    _need("x", x, x.dtype, (T, H), dev, el != B.MM_ELEMENT_8BIT, _VEC)
    K = topk_ids.shape[1] if isinstance(topk_ids, torch.Tensor) and topk_ids.dim() == 2 else 0
    _need("topk_ids", topk_ids, torch.int32, (T, K), dev)
    if active is not None:
        _need("active", active, torch.int8, (T,), dev)
    E = num_experts if type(num_experts) is int else _whole("num_experts", num_experts)
    plan = _sort_plan(T or 1, H, E, K, el)
    with _stream_of(dev, stream):
        if _records(x):
            made = []
            return _SortFunction.apply(x, (topk_ids, active, plan, T, E, K), made), made[0]
        return _sort_tokens(x, topk_ids, active, plan, T, E, K)


def sort_rows(x, order, *, stream=None):
    """mm_sort_rows: the rows [T*K,H] of another x [T,H] (codes, scales, a gradient) in an order that sort_tokens has
    made.  Differentiable as sort_tokens is."""
    T, H, dev = _rows("x", x)
    el = _element("x", x, False)
    _need("x", x, x.dtype, (T, H), dev, el != B.MM_ELEMENT_8BIT, _VEC)
    dims = _order_of(order, dev)
    if dims[0] != T:
        raise ValueError(f"order: one of {T} tokens is needed, got one of {dims[0]}")
    _sort_plan(max(T, 1), H, dims[1], dims[2], el)
    with _stream_of(dev, stream):
        if _records(x):
            return _SortFunction.apply(x, dims, [order])
        return _sort_rows(x, order.offsets, order.row_of_route, *dims)


def _combine_args(name, rows, order, weights):
    R, H, dev = _rows(name, rows)
    el = _element(name, rows, True)
    dims = T, E, K = _order_of(order, dev)
    _need(name, rows, rows.dtype, (T * K, H), dev, True, _VEC)
    if weights is not None:
        _need("weights", weights, torch.float32, (T, K), dev, grad=True)
    _sort_plan(max(T, 1), H, E, K, el)
    return dims, H, dev


def combine_tokens(rows, order, weights=None, *, stream=None):
    """mm_combine_tokens: y [T,H] = the weighted sum of every token's rows (bf16, float16 or float32 [T*K,H], sorted by
    ``order``; weights float32 [T,K], None: 1), in float32 in the order of k, rounded once.  Differentiable with respect
    to rows and weights; the gradients are ``combine_backward(dy, rows, order, weights)``."""
    dims, _, dev = _combine_args("rows", rows, order, weights)
    with _stream_of(dev, stream):
        if _records(rows, weights):
            return _CombineFunction.apply(rows, weights, order, dims)
        return _combine(rows, order.row_of_route, weights, *dims)


def combine_backward(dy, rows, order, weights, *, stream=None):
    """mm_combine_backward: (drows [T*K,H], dweights float32 [T,K]) of combine_tokens for y's gradient dy [T,H], as its
    autograd computes them; for steps that are captured into a graph."""
    if weights is None:
        raise ValueError("weights: needed (without weights the gradient is sort_rows(dy, order))")
    dims, H, dev = _combine_args("rows", rows, order, weights)
    for name, t in (("rows", rows), ("weights", weights)):
        _need(name, t, t.dtype, t.shape, dev)
    _need("dy", dy, rows.dtype, (dims[0], H), dev, at=_VEC)
    with _stream_of(dev, stream):
        return _combine_backward(dy, rows, order.offsets, order.row_of_route, weights, *dims, True, True)


# ------------------------------------------------- activation, kept in 8 bits

def _swiglu_args(h, activation_clamp, gate_up_group, grad):
    M, N, dev = _rows("h", h)
    el = _element("h", h, True)
    _need("h", h, h.dtype, (M, N), dev, grad, _VEC)
    if N % 2 or N == 0:
        raise ValueError(f"h: [rows, 2 * intermediate] is needed, got {N} columns")
    return M, N // 2, dev, el, _turn_of(gate_up_group, N // 2), _clamp_of(activation_clamp)


def _turn_of(gate_up_group, I):
    g = gate_up_group if type(gate_up_group) is int else _whole("gate_up_group", gate_up_group)
    if g < 0 or (g and (g % 8 or I % g)):
        raise ValueError(f"gate_up_group: 0, or a multiple of 8 that divides {I}, is needed, got {gate_up_group!r}")
    return g


def _clamp_of(activation_clamp):
    if activation_clamp is None:
        return None
    c = float(activation_clamp)
    if not c >= 0.0:
        raise ValueError(f"activation_clamp: None or a number from 0 on is needed, got {activation_clamp!r}")
    return c


def _swiglu(h, M, I, el, turn, clamp, keep):
    dev = h.device
    a = torch.empty((M, I), dtype=h.dtype, device=dev)
    q = torch.empty((M, 2 * I), dtype=torch.int8, device=dev) if keep else None
    s = torch.empty((M, 2 * -(-I // 128)), dtype=torch.float32, device=dev) if keep else None
    if M:
        B.mm_swiglu(M, I, el, turn, h, clamp, a, q, s, _raw_stream(dev))
    return a, q, s


def _swiglu_backward(da, q, s, turn, clamp):
    M, I = da.shape
    dh = torch.empty((M, 2 * I), dtype=da.dtype, device=da.device)
    if M:
        B.mm_swiglu_backward(M, I, B.ELEMENT[da.dtype], turn, da, q, s, clamp, dh, _raw_stream(da.device))
    return dh


class _SwigluFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, M, I, el, turn, clamp):
        a, q, s = _swiglu(h, M, I, el, turn, clamp, True)
        ctx.how = turn, clamp
        _keep(ctx, q, s)
        return a

    @staticmethod
    @_once
    def backward(ctx, da):
        _not_captured()
        return _swiglu_backward(_dense(da), *_kept(ctx, "codes", "scales"), *ctx.how), None, None, None, None, None


def swiglu(h, *, activation_clamp=None, gate_up_group=0, stream=None):
    """mm_swiglu: a [M,I] = SiLU(gate) * up of h [M,2I] (bf16, float16 or float32), gate and up clamped to
    [-activation_clamp, activation_clamp] first unless that is None.  gate_up_group: 0 where h is [gate | up]; behind the
    rows of ``ExpertLayer.w1`` gate and up columns alternate in groups of ``layer.plan.gate_up_group``.  Differentiable:
    what it keeps for the backward pass is h in 8 bits, with a float32 scale per 128 gate or up values, and the gradient
    is that at the kept values."""
    M, I, dev, el, turn, clamp = _swiglu_args(h, activation_clamp, gate_up_group, True)
    with _stream_of(dev, stream):
        if _records(h):
            return _SwigluFunction.apply(h, M, I, el, turn, clamp)
        return _swiglu(h, M, I, el, turn, clamp, False)[0]


def swiglu_forward(h, *, activation_clamp=None, gate_up_group=0, stream=None):
    """(a, codes int8 [M,2I], scales float32 [M,2*ceil(I/128)]): swiglu and the copy of h that swiglu_backward takes
    (codes lie as h does; scales of the gates come first)."""
    M, I, dev, el, turn, clamp = _swiglu_args(h, activation_clamp, gate_up_group, False)
    with _stream_of(dev, stream):
        return _swiglu(h, M, I, el, turn, clamp, True)


def swiglu_backward(da, codes, scales, *, activation_clamp=None, gate_up_group=0, stream=None):
    """mm_swiglu_backward: h's gradient [M,2I] from a's [M,I] and what swiglu_forward kept."""
    M, I, dev = _rows("da", da)
    _element("da", da, True)
    _need("da", da, da.dtype, (M, I), dev, at=_VEC)
    _need("codes", codes, torch.int8, (M, 2 * I), dev, at=_VEC)
    _need("scales", scales, torch.float32, (M, 2 * -(-I // 128)), dev)
    turn, clamp = _turn_of(gate_up_group, I), _clamp_of(activation_clamp)
    with _stream_of(dev, stream):
        return _swiglu_backward(da, codes, scales, turn, clamp)


# ------------------------------------------------- 8-bit integer product

_int8_plan = functools.lru_cache(maxsize=256)(B.mm_int8_plan_create)
_Y_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def int8_quantize(x, stream=None):
    """mm_int8_quantize: (codes int8 [M,K], scales float32 [M]) of rows of x, tokens or a weight's output channels
    (bf16, float16 or float32; K a multiple of 16)."""
    M, K, dev = _rows("x", x)
    el = _element("x", x, True)
    _need("x", x, x.dtype, (M, K), dev, at=_VEC)
    if K % 16 or K == 0:
        raise ValueError(f"x: the columns have to be a multiple of 16, got {K}")
    with _stream_of(dev, stream):
        q = torch.empty((M, K), dtype=torch.int8, device=dev)
        s = torch.empty(M, dtype=torch.float32, device=dev)
        if M:
            B.mm_int8_quantize(M, K, el, x, q, s, _raw_stream(dev))
    return q, s


def _int8_args(M, K, dev, x_element, rows, w, ws, offsets, counts, y_dtype, y):
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w: [out, in] or [groups, out, in] is needed")
    G, N = (1, w.shape[0]) if w.dim() == 2 else (w.shape[0], w.shape[1])
    lead = () if w.dim() == 2 else (G,)
    _need("w", w, torch.int8, lead + (N, K), dev, at=_VEC)
    _need("ws", ws, torch.float32, lead + (N,), dev, at=1 if N % 4 else _VEC)
    _group_args(G, offsets, counts, dev)
    if y_dtype not in _Y_TYPES:
        raise ValueError(f"y_dtype: one of {sorted(_Y_TYPES)} is needed, got {y_dtype!r}")
    dt = _Y_TYPES[y_dtype]
    if y is not None:
        _need("y", y, dt, (M, N), dev, at=_VEC)
        _apart(y, *rows, w, ws, offsets, counts)
    return N, dt, _int8_plan(max(M, 1), N, K, G, x_element, B.ELEMENT[dt])


def int8_matmul(q, s, w, ws, offsets=None, counts=None, *, y_dtype="bf16", y=None, stream=None):
    """mm_int8_gemm: y [M,N] of int8 rows (q [M,K], s float32 [M]) and weights (w int8 [N,K], ws float32 [N]), or, with
    w [G,N,K] and ws [G,N], of groups of rows as in ``block_matmul``; sort_tokens' order has their offsets and counts.
    y_dtype: "bf16", "f16" or "f32".  Sums are exact.  y must not overlap an input."""
    M, K, dev = _rows("q", q)
    _need("q", q, torch.int8, (M, K), dev, at=_VEC)
    _need("s", s, torch.float32, (M,), dev)
    N, dt, plan = _int8_args(M, K, dev, B.MM_ELEMENT_BF16, (q, s), w, ws, offsets, counts, y_dtype, y)
    with _stream_of(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=dt, device=dev)
        if M:
            B.mm_int8_gemm(plan, q, s, w, ws, offsets, counts, y, _raw_stream(dev))
    return y


def int8_linear(x, w, ws, offsets=None, counts=None, *, y_dtype="bf16", y=None, stream=None):
    """mm_int8_linear: int8_matmul of x's (bf16, float16 or float32 [M,K]) codes and scales, in one call."""
    M, K, dev = _rows("x", x)
    el = _element("x", x, True)
    _need("x", x, x.dtype, (M, K), dev, at=_VEC)
    N, dt, plan = _int8_args(M, K, dev, el, (x,), w, ws, offsets, counts, y_dtype, y)
    with _stream_of(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=dt, device=dev)
        if M:
            n = plan.dense_workspace_bytes if offsets is None else plan.workspace_bytes
            B.mm_int8_linear(plan, x, w, ws, offsets, counts, y, _workspace(n, dev) if n else None, _raw_stream(dev))
    return y
