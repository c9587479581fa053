"""Device-memory plumbing around the C ABI (torch allocates, the library computes).

``ExpertLayer`` holds one plan, the prepared expert weights and a
workspace, and calls the C-ABI entry points through ``binding``.  The
functions ``route``, ``moe_few``, ``block_quantize``, ``block_matmul`` and
``block_linear`` hold nothing: each checks its tensors, allocates the
outputs and a workspace on the calling stream and makes one call.  Nothing
here computes any part of the expert path.
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


def _need(name, t, dtype, shape, device):
    """The one check of a tensor argument: a message that says what it has to be."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor {list(shape)} on {device} is needed, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))
    if t.requires_grad and torch.is_grad_enabled():
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
    return *x.shape, x.device


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
    _need("x", x, torch.bfloat16, (T, H), dev)
    _need("weight", weight, torch.bfloat16, (E, H), dev)
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
    _need("x", x, torch.bfloat16, (T, H), dev)
    _need("w1", w1, w1.dtype, (Et, 2 * I, H), dev)
    _need("w2", w2, w1.dtype, (Et, H, I), dev)
    if fmt == "bf16":
        if s1 is not None or s2 is not None:
            raise ValueError("s1, s2: bf16 weights have no scales")
    else:
        _need("s1", s1, torch.float32, (Et, 2 * I) if fmt == "fp8" else (Et, 2 * I // 128, H // 128), dev)
        _need("s2", s2, torch.float32, (Et, H) if fmt == "fp8" else (Et, H // 128, I // 128), dev)
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
        _need("y", y, ydt, (T, H), dev)
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
    _need("x", x, torch.bfloat16, (M, K), dev)
    if K % 128 or K == 0:
        raise ValueError(f"x: the columns have to be a multiple of 128, got {K}")
    with _stream_of(dev, stream):
        q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
        s = torch.empty((M, K // 128), dtype=torch.float32, device=dev)
        if M:
            B.mm_block_quantize(M, K, x, q, s, _raw_stream(dev))
    return q, s


def _block_args(M, K, dev, rows, w, ws, offsets, counts, y):
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w: [out, in] or [groups, out, in] is needed")
    G, N = (1, w.shape[0]) if w.dim() == 2 else (w.shape[0], w.shape[1])
    lead = () if w.dim() == 2 else (G,)
    _need("w", w, torch.float8_e4m3fn, lead + (N, K), dev)
    _need("ws", ws, torch.float32, lead + (-(-N // 128), K // 128), dev)
    if (offsets is None) != (counts is None) or (offsets is None and G > 1):
        raise ValueError("offsets, counts: both are needed, or neither with one matrix")
    if offsets is not None:
        n = offsets.shape[0] if isinstance(offsets, torch.Tensor) and offsets.dim() == 1 else -1
        _need("offsets", offsets, torch.int32, (n if n == G + 1 else G,), dev)
        _need("counts", counts, torch.int32, (G,), dev)
    if y is not None:
        _need("y", y, torch.bfloat16, (M, N), dev)
        _apart(y, *rows, w, ws, offsets, counts)
    return N, _block_plan(max(M, 1), N, K, G)


def block_matmul(q, s, w, ws, offsets=None, counts=None, y=None, stream=None):
    """mm_block_gemm: y bf16 [M,N] of e4m3 rows (q [M,K], s [M,K/128]) and weights (w [N,K], ws [ceil(N/128),K/128]),
    or, with w [G,N,K] and ws [G,...], of groups of rows: group g covers rows offsets[g] .. offsets[g] + counts[g]
    (int32; offsets may have G + 1 entries).  Rows that no group covers are left as they are (in a new y: unset).  y
    must not overlap an input."""
    M, K, dev = _rows("q", q)
    _need("q", q, torch.float8_e4m3fn, (M, K), dev)
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
    _need("x", x, torch.bfloat16, (M, K), dev)
    N, plan = _block_args(M, K, dev, (), w, ws, offsets, counts, y)
    with _stream_of(dev, stream):
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if M:
            B.mm_block_linear(plan, x, w, ws, offsets, counts, y, _workspace(plan.workspace_bytes, dev), _raw_stream(dev))
    return y
