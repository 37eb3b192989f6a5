"""Python binding of the router: expert ids and scores from the router's
logits, and the logits' gradient (argument marshalling only; the work is done
by the library's HIP kernels)."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .autograd import _watch_accumulators
from .moe import _DTYPES, _call, _check_rows, _refuse_tangents, _stream

SCORES = {"softmax": L.MOE_SCORE_SOFTMAX, "sigmoid": L.MOE_SCORE_SIGMOID}


class Routing(NamedTuple):
    ids: torch.Tensor        # int32 [T, K], -1 = no expert
    scores: torch.Tensor     # float32 [T, K], 0 where there is none


def _check_logits(logits: torch.Tensor) -> None:
    if logits.dtype not in _DTYPES:
        raise TypeError(f"logits must be one of {list(_DTYPES)}, got {logits.dtype}")
    _check_rows("logits", logits, logits.dtype, 2, logits.device)


def _forward(logits, topk, score, bias, flags, scale, num_groups, topk_groups):
    dev = logits.device
    T, E = logits.shape
    ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    scores = torch.empty((T, topk), dtype=torch.float32, device=dev)
    _call("moe_route_topk", dev, logits.data_ptr(), _DTYPES[logits.dtype],
          0 if bias is None else bias.data_ptr(), T, E, topk, score, flags, scale, num_groups,
          topk_groups, ids.data_ptr(), scores.data_ptr())
    return ids, scores


def _backward(grad_scores, logits, ids, score, flags, scale):
    grad = torch.empty_like(logits)
    T, E = logits.shape
    _call("moe_route_topk_backward", logits.device, logits.data_ptr(), _DTYPES[logits.dtype],
          ids.data_ptr(), grad_scores.data_ptr(), T, E, ids.shape[1], score, flags, scale,
          grad.data_ptr())
    return grad


class _RouteTopk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, score, bias, flags, scale, num_groups, topk_groups):
        ids, scores = _forward(logits, topk, score, bias, flags, scale, num_groups, topk_groups)
        ctx.save_for_backward(logits, ids)
        ctx.args = score, flags, scale
        ctx.mark_non_differentiable(ids)
        # No zeros for the ids' gradient, which is none: that would be a launch.
        ctx.set_materialize_grads(False)
        return ids, scores

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _grad_ids, grad_scores):
        if grad_scores is None:
            return (None,) * 8
        logits, ids = ctx.saved_tensors
        score, flags, scale = ctx.args
        grad = _backward(grad_scores.contiguous(), logits, ids, score, flags, scale)
        return grad, None, None, None, None, None, None, None


def _score(name: str) -> int:
    try:
        return SCORES[name]
    except KeyError:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {name!r}") from None


def route_topk(logits: torch.Tensor, topk: int, *, score: str = "softmax",
               bias: Optional[torch.Tensor] = None, renormalize: bool = True, scale: float = 1.0,
               num_groups: int = 1, topk_groups: int = 1) -> Routing:
    """The topk experts of every token and their scores (moe_route_topk): the
    ids and scores that layout(), dispatch() and combine() take. Differentiable
    in the logits.

    logits fp32 or bf16 [T, E]. With p = softmax(logits) or sigmoid(logits) the
    experts with the largest p + bias are chosen (without a bias those with the
    largest logits), equal ones by ascending index; scores = scale * p, divided by
    the sum of the chosen p if renormalize. bias, fp32 [E], goes with the sigmoid
    only; it decides who is chosen, does not enter the scores and gets no
    gradient. num_groups > 1: only the experts of the topk_groups best of
    num_groups groups of neighbouring experts can be chosen, by the group's
    largest p (softmax) or the sum of its two largest p + bias (sigmoid).

    A logit of NaN or -inf takes its expert out of the token's choice (and out
    of the softmax's sum); a slot for which no expert is left has id -1 and
    score 0, so a row of -inf routes nowhere. Forward-mode derivatives are
    refused; a step can be captured into a graph under expert_ffn's conditions."""
    dev = logits.device
    _check_logits(logits)
    kind = _score(score)
    if bias is not None:
        if kind != L.MOE_SCORE_SIGMOID:
            raise ValueError("bias goes with score='sigmoid'")
        _check_rows("bias", bias, torch.float32, 1, dev)
        if bias.shape[0] != logits.shape[1]:
            raise ValueError(f"bias must have {logits.shape[1]} entries, got {bias.shape[0]}")
    topk = int(topk)
    if not 1 <= topk <= L.MOE_MAX_TOPK:
        raise ValueError(f"topk must be 1 to {L.MOE_MAX_TOPK}, got {topk}")
    args = (topk, kind, bias, L.MOE_ROUTE_RENORMALIZE if renormalize else 0, float(scale),
            int(num_groups), int(topk_groups))
    _refuse_tangents("route_topk", logits)
    if torch.is_grad_enabled() and logits.requires_grad:
        out = Routing(*_RouteTopk.apply(logits, *args))
        _watch_accumulators(out.scores.grad_fn, _stream(dev), "route_topk")
        return out
    return Routing(*_forward(logits, *args))


def route_topk_backward(grad_scores: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *,
                        score: str = "softmax", renormalize: bool = True,
                        scale: float = 1.0) -> torch.Tensor:
    """Gradient of route_topk's scores with respect to the logits
    (moe_route_topk_backward), [T, E] of the logits' type: grad_scores fp32
    [T, K], logits and ids as route_topk took and gave them. The call that
    route_topk's own backward makes. Records no gradient; forward-mode
    derivatives are refused."""
    dev = logits.device
    _check_logits(logits)
    kind = _score(score)
    _check_rows("ids", ids, torch.int32, 2, dev)
    _check_rows("grad_scores", grad_scores, torch.float32, 2, dev)
    if ids.shape[0] != logits.shape[0] or grad_scores.shape != ids.shape:
        raise ValueError("shapes: logits [T, E], ids and grad_scores [T, K]; got "
                         f"{tuple(logits.shape)}, {tuple(ids.shape)}, {tuple(grad_scores.shape)}")
    _refuse_tangents("route_topk_backward", grad_scores, logits)
    return _backward(grad_scores, logits, ids, kind,
                     L.MOE_ROUTE_RENORMALIZE if renormalize else 0, float(scale))
