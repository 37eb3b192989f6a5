"""torch.autograd wrappers of dispatch and combine (binding layer only).

Every forward and backward step runs in the library's kernels
(moe_layout + moe_dispatch, moe_combine, moe_combine_backward,
moe_dispatch_backward); these Functions only route tensors. Use one
MoeDispatcher(backward=True) per MoE layer. The small per-call state the
backward needs (row map, true total) is copied at forward time, so a later
forward of the same layer cannot overwrite it.

The dispatched rows are another matter: by default dispatch() returns a view
of the dispatcher's persistent x_e buffer, which the layer's next forward
rewrites. An expert that saves its input for its weight gradient then sees
the newer rows. So each forward records the dispatcher's x_e generation, and
the combine's backward (which runs before the expert's backward) raises if a
later dispatch on the same dispatcher rewrote x_e in between. Schedules with
several forwards in flight per layer (pipelining with micro-batches,
activation recompute) use MoeTokenDispatcher(..., clone_x_e=True): dispatch
then returns a copy of the rows that the layer owns.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd import forward_ad

from . import _lib as L
from .experts import _activation, _offsets, _rows, _weights
from .moe import MoeDispatcher, _call, _stream


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, scores, ids, disp: MoeDispatcher, ntpr: int, clone_x_e: bool):
        lay = disp.layout(ids, ntpr)
        out = disp.dispatch(x, scores.detach(), ids, lay.counts, num_tokens_per_rank=ntpr)
        row_map = lay.row_map.clone()
        total = lay.offsets[-1:].clone()
        ctx.disp, ctx.T, ctx.ntpr, ctx.row_map = disp, x.shape[0], ntpr, row_map
        ctx.mark_non_differentiable(row_map, total)
        # A fresh tensor object per call: autograd attaches this call's node to
        # it, and the binding hands out one shared view per extent.
        x_e = out.x_e.clone() if clone_x_e else out.x_e.view(out.x_e.shape)
        return x_e, row_map, total

    @staticmethod
    def backward(ctx, grad_x_e, _grad_row_map, _grad_total):
        g = grad_x_e.contiguous()
        grad_x = ctx.disp.dispatch_backward(g, ctx.row_map, ctx.T, num_tokens_per_rank=ctx.ntpr)
        return grad_x.clone(), None, None, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y_e, scores, row_map, total, disp: MoeDispatcher, ntpr: int,
                generation: Optional[int]):
        rows = disp.rows_for(ntpr)
        if y_e.shape[0] != rows:
            raise ValueError(f"y_e must have round_up4(num_tokens_per_rank) * topk = {rows} "
                             f"rows (the dispatched rows), got {y_e.shape[0]}")
        y = disp.combine(y_e, row_map, scores, num_tokens_per_rank=ntpr)
        ctx.save_for_backward(y_e, scores, row_map, total)
        ctx.disp, ctx.ntpr, ctx.generation = disp, ntpr, generation
        return y.clone()

    @staticmethod
    def backward(ctx, grad_y):
        if ctx.generation is not None and ctx.disp.x_e_generation != ctx.generation:
            raise RuntimeError(
                "x_e of this MoE layer was rewritten by a later dispatch before this backward "
                "(several forwards in flight on one MoeDispatcher); the expert's saved input "
                "would be the newer rows. Use MoeTokenDispatcher(..., clone_x_e=True).")
        y_e, scores, row_map, total = ctx.saved_tensors
        # The library writes the slots' rows and +0.0 into the rows from the
        # true total on (no slot reaches them), reading the total on the device.
        g_e, g_s = ctx.disp.combine_backward(grad_y.contiguous(), y_e, row_map, scores,
                                             num_tokens_per_rank=ctx.ntpr, total=total)
        return g_e.clone(), g_s.clone(), None, None, None, None, None


class MoeTokenDispatcher:
    """Differentiable dispatch/combine of one MoE layer.

        d = MoeTokenDispatcher(MoeDispatcher(nmax, D, E, K, backward=True))
        x_e = d.dispatch(x, scores, ids)        # [round_up4(ntpr) * K, D]
        y_e = experts(x_e)                      # rows [0, total) are the tokens'
        y = d.combine(y_e, scores)              # [T, D]
        y.backward(...)                         # dL/dx, dL/dscores, dL/dy_e

    clone_x_e=False (default): x_e is a view of the dispatcher's buffer and a
    second forward before the first one's backward is detected and raises.
    clone_x_e=True: x_e is a copy owned by the caller; any number of forwards
    may be in flight.
    """

    def __init__(self, dispatcher: MoeDispatcher, clone_x_e: bool = False):
        if not dispatcher.backward_enabled:
            raise ValueError("the MoeDispatcher needs backward=True")
        self.disp = dispatcher
        self.clone_x_e = bool(clone_x_e)
        self._row_map: Optional[torch.Tensor] = None
        self._total: Optional[torch.Tensor] = None
        self._ntpr: Optional[int] = None
        self._generation: Optional[int] = None

    def dispatch(self, x: torch.Tensor, topk_scores: torch.Tensor, topk_ids: torch.Tensor,
                 num_tokens_per_rank: Optional[int] = None) -> torch.Tensor:
        ntpr = x.shape[0] if num_tokens_per_rank is None else int(num_tokens_per_rank)
        x_e, self._row_map, self._total = _Dispatch.apply(
            x.contiguous(), topk_scores.contiguous(), topk_ids.contiguous(), self.disp, ntpr,
            self.clone_x_e)
        self._ntpr = ntpr
        self._generation = None if self.clone_x_e else self.disp.x_e_generation
        return x_e

    def combine(self, y_e: torch.Tensor, topk_scores: torch.Tensor) -> torch.Tensor:
        if self._row_map is None:
            raise RuntimeError("combine() needs a preceding dispatch() on this layer")
        return _Combine.apply(y_e.contiguous(), topk_scores.contiguous(), self._row_map,
                              self._total, self.disp, self._ntpr, self._generation)


def _ffn_forward(x, w_gate_up, w_down, offsets, act: int, pre: Optional[torch.Tensor]):
    """(h, y) of checked arguments: the calls of gated_grouped_gemm and
    grouped_gemm_forward. h's rows outside the segments stay unwritten, y's are
    zero."""
    dev, off = x.device, offsets.data_ptr()
    R, k_in = x.shape
    E, n_out, hidden = w_down.shape
    h, y = x.new_empty((R, hidden)), x.new_empty((R, n_out))
    _call("moe_gated_grouped_gemm", dev, x.data_ptr(), w_gate_up.data_ptr(), off, E, R, k_in,
          hidden, act, h.data_ptr(), 0 if pre is None else pre.data_ptr(), 0)
    _call("moe_grouped_gemm_forward", dev, h.data_ptr(), w_down.data_ptr(), off, E, R, hidden,
          n_out, y.data_ptr(), L.MOE_GEMM_ZERO_OUTSIDE)
    return h, y


class _ExpertFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate_up, w_down, offsets, act: int):
        # The layout's offsets are a persistent buffer the next layout
        # rewrites: the backward keeps its own copy.
        offsets = offsets.clone()
        pre = torch.empty((x.shape[0], w_gate_up.shape[1]), dtype=torch.float32,
                          device=x.device)
        h, y = _ffn_forward(x, w_gate_up, w_down, offsets, act, pre)
        ctx.save_for_backward(x, w_gate_up, w_down, offsets, pre, h)
        ctx.act = act
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        # The forward has checked every size; these are the calls of
        # grouped_gemm_backward_weight, gated_grouped_gemm_backward and
        # grouped_gemm_backward_input.
        x, w_gate_up, w_down, offsets, pre, h = ctx.saved_tensors
        need_x, need_gate_up, need_down = ctx.needs_input_grad[:3]
        g = grad_y.contiguous()
        if g.data_ptr() % 16 != 0:
            g = g.clone()           # a slice of a larger gradient may begin anywhere
        dev, off = x.device, offsets.data_ptr()
        R, k_in = x.shape
        E, n_out, hidden = w_down.shape
        grad_x = grad_gate_up = grad_down = None
        if need_down:
            grad_down = torch.empty_like(w_down)
            _call("moe_grouped_gemm_backward_weight", dev, g.data_ptr(), h.data_ptr(), off, E, R,
                  hidden, n_out, L.MOE_BF16, grad_down.data_ptr(), 0)
        if need_x or need_gate_up:
            # Rows outside the segments are read by neither product below.
            grad_pre = x.new_empty((R, 2 * hidden))
            _call("moe_gated_grouped_gemm_backward", dev, g.data_ptr(), w_down.data_ptr(),
                  pre.data_ptr(), off, E, R, hidden, n_out, ctx.act, grad_pre.data_ptr(), 0)
            if need_gate_up:
                grad_gate_up = torch.empty_like(w_gate_up)
                _call("moe_grouped_gemm_backward_weight", dev, grad_pre.data_ptr(), x.data_ptr(),
                      off, E, R, k_in, 2 * hidden, L.MOE_BF16, grad_gate_up.data_ptr(), 0)
            if need_x:
                grad_x = torch.empty_like(x)
                _call("moe_grouped_gemm_backward_input", dev, grad_pre.data_ptr(),
                      w_gate_up.data_ptr(), off, E, R, k_in, 2 * hidden, grad_x.data_ptr(),
                      L.MOE_GEMM_ZERO_OUTSIDE)
        return grad_x, grad_gate_up, grad_down, None, None


# Whether a leaf's gradient accumulator was made on the default stream, as far as
# the calls here can tell: noted by the first of them that meets it.
_ON_DEFAULT_STREAM = "combine_moe_layout.default_stream"


def _watch_accumulators(node, stream: int) -> None:
    """Looks at the gradient accumulators of the leaves that a call's node
    leads to. The engine runs an accumulator on the stream it was made on, and
    it lives as long as any graph that reaches it. One made on the default
    stream cannot join a capture: the backward would fail inside the engine and
    end the process, so such a capture is refused here. Calls that only use an
    accumulator do not change where it belongs."""
    leaves = [fn for fn, _ in node.next_functions if hasattr(fn, "variable")]
    capturing = torch.cuda.is_current_stream_capturing()
    for fn in leaves:
        on_default = fn.metadata.setdefault(_ON_DEFAULT_STREAM, stream == 0 and not capturing)
        if capturing and on_default:
            raise RuntimeError(
                "expert_ffn cannot be captured while the output of an earlier call on the default "
                "stream that reaches the same leaf tensors is alive: its gradient accumulators "
                "belong to that stream. Delete that output first, or run the calls before the "
                "capture on a side stream.")


def expert_ffn(x_expert: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
               offsets: torch.Tensor, activation: str = "silu") -> torch.Tensor:
    """Differentiable gated feed-forward block of the experts, between
    dispatch and combine: for the rows r of expert e,
        y[r] = (act(x[r] @ Wg[e].T) * (x[r] @ Wu[e].T)) @ Wd[e].T

    x_expert bf16 [R, k_in]; w_gate_up bf16 [E, 2 n_hidden, k_in] (the gate's
    rows first); w_down bf16 [E, n_out, n_hidden]; offsets int32 [E+1] (e.g.
    Layout.offsets); y bf16 [R, n_out], its rows of no segment (from offsets[E] on
    and before offsets[0]) zero.
    Gradients reach x_expert and both weights (bf16, in one rounding of an fp32
    sum). Between the kernels h = act(g) * u and, in the backward, the gradients
    of g and u are rounded to bf16: they are operands of matrix-core products.
    g and u themselves are kept in fp32. Forward-mode derivatives are refused.
    x_expert is kept for the backward, not copied: rows in a MoeDispatcher's
    buffer must not be dispatched anew before it (MoeTokenDispatcher watches for
    that in combine()'s backward).

    A step can be captured into a graph (forward and backward together) after
    warm-up calls on a side stream. While an output of a call on the default
    stream that takes the same leaf tensors is alive, the capture is refused.
    Two cases only the caller can know of, and has to avoid, since such a
    backward ends the process: a graph of another operation on the same leaves
    (a penalty on a weight, say) that was made on the default stream and is
    alive across the capture, and one of the leaves from which an input was
    computed."""
    dev = x_expert.device
    act = _activation(activation)
    E, n2, k_in = _weights("w_gate_up", w_gate_up, dev)
    E2, _, hidden = _weights("w_down", w_down, dev)
    if E2 != E or 2 * hidden != n2:
        raise ValueError("shapes: w_gate_up [E, 2 n_hidden, k_in], w_down [E, n_out, n_hidden]; "
                         f"got {tuple(w_gate_up.shape)}, {tuple(w_down.shape)}")
    _rows("x_expert", x_expert, k_in, dev)
    _offsets(offsets, E, dev)
    if any(forward_ad.unpack_dual(t).tangent is not None for t in (x_expert, w_gate_up, w_down)):
        raise NotImplementedError("expert_ffn has no forward-mode derivative")
    if torch.is_grad_enabled() and (x_expert.requires_grad or w_gate_up.requires_grad
                                    or w_down.requires_grad):
        if n2 > L.MOE_MAX_GEMM_WIDTH and (x_expert.requires_grad or w_gate_up.requires_grad):
            raise ValueError(f"n_hidden must be at most {L.MOE_MAX_GEMM_WIDTH // 2} for gradients "
                             f"of x_expert and w_gate_up, got {hidden}")
        y = _ExpertFfn.apply(x_expert, w_gate_up, w_down, offsets, act)
        _watch_accumulators(y.grad_fn, _stream(dev))
        return y
    return _ffn_forward(x_expert, w_gate_up, w_down, offsets, act, None)[1]
