"""Python binding of the whole expert layer for a few tokens (argument
marshalling only; the work is done by the library's HIP kernels)."""
from __future__ import annotations

from typing import Union

import torch

from . import _lib as L
from .experts import _activation
from .moe import Mxfp4ExpertWeights, _call, _check_rows, _refuse_tangents


def moe_layer(x_TD: torch.Tensor, topk_scores_TK: torch.Tensor, topk_expert_ids_TK: torch.Tensor,
              w_gate_up: Union[torch.Tensor, Mxfp4ExpertWeights],
              w_down: Union[torch.Tensor, Mxfp4ExpertWeights], *,
              activation: str = "silu") -> torch.Tensor:
    """The expert layer of a decoding step in two launches
    (moe_few_tokens_layer), for the sum over a token's slots k
        y[t] = sum of scores[t, k] * (act(x[t] @ Wg[e].T) * (x[t] @ Wu[e].T)) @ Wd[e].T
    with e = ids[t, k]: what layout, dispatch, gated_grouped_gemm,
    grouped_gemm and combine give, with no MoeDispatcher and fewer roundings.

    x bf16 [T, D]; scores fp32 and ids int32 [T, K] (e.g. route_topk's), T * K
    at most 512; a slot whose id is no expert's adds nothing. Weights bf16
    [E, 2 F, D] (gate rows first) and [E, D, F], or both as Mxfp4ExpertWeights.
    Made for the few tokens of a decoding step; the separate calls read an
    expert's weights fewer times where it has several slots. From where they
    are the faster ones depends on the shape: 256 experts of 7168 x 2048 and 8
    slots a token, from about 4 tokens on in bf16 (by 2 to 4 %) and between 32
    and 64 in 4 bits; 8 experts of 4096 x 4096 and 2 slots, between 8 and 64
    tokens (by 39 and 55 % at 64).
    activation "silu" or "gelu" (tanh form). Result bf16 [T, D]. Records no
    gradient: training goes through MoeTokenDispatcher and expert_ffn.
    Forward-mode derivatives are refused."""
    dev = x_TD.device
    act = _activation(activation)
    _check_rows("x_TD", x_TD, torch.bfloat16, 2, dev)
    _check_rows("topk_scores_TK", topk_scores_TK, torch.float32, 2, dev)
    _check_rows("topk_expert_ids_TK", topk_expert_ids_TK, torch.int32, 2, dev)
    T, D = x_TD.shape
    K = topk_scores_TK.shape[1]
    if topk_scores_TK.shape[0] != T or topk_expert_ids_TK.shape != topk_scores_TK.shape:
        raise ValueError("shapes: x_TD [T, D], topk_scores_TK and topk_expert_ids_TK [T, K]; got "
                         f"{tuple(x_TD.shape)}, {tuple(topk_scores_TK.shape)}, "
                         f"{tuple(topk_expert_ids_TK.shape)}")
    if T * K > L.MOE_MAX_LAYER_SLOTS:
        raise ValueError(f"moe_layer takes at most {L.MOE_MAX_LAYER_SLOTS} slots (T * K), got "
                         f"{T * K}; larger batches go through a MoeDispatcher")
    four = isinstance(w_gate_up, Mxfp4ExpertWeights)
    if four != isinstance(w_down, Mxfp4ExpertWeights):
        raise TypeError("w_gate_up and w_down must both be bf16 or both Mxfp4ExpertWeights")
    if four:
        w_gate_up.check(dev)
        w_down.check(dev)
        shapes = ((w_gate_up.num_experts, w_gate_up.n_out, w_gate_up.k_in),
                  (w_down.num_experts, w_down.n_out, w_down.k_in))
        w1, w2 = w_gate_up.data, w_down.data
    else:
        _check_rows("w_gate_up", w_gate_up, torch.bfloat16, 3, dev)
        _check_rows("w_down", w_down, torch.bfloat16, 3, dev)
        shapes = tuple(w_gate_up.shape), tuple(w_down.shape)
        w1, w2 = w_gate_up, w_down
    E, _, F = shapes[1]
    if shapes != ((E, 2 * F, D), (E, D, F)):
        raise ValueError(f"shapes: w_gate_up [E, 2 F, {D}], w_down [E, {D}, F]; got {shapes[0]}, "
                         f"{shapes[1]}")
    _refuse_tangents("moe_layer", x_TD, topk_scores_TK, w1, w2)
    y = torch.empty_like(x_TD)
    # h between the two launches (moe_few_tokens_workspace_bytes).
    nbytes = 4 * T * K * (-(-F // 128) * 128)
    h = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call("moe_few_tokens_layer", dev, x_TD.data_ptr(), topk_scores_TK.data_ptr(),
          topk_expert_ids_TK.data_ptr(), T, K, w1.data_ptr(), w2.data_ptr(),
          L.MOE_WEIGHTS_MXFP4 if four else L.MOE_WEIGHTS_ROW_MAJOR, E, D, F, act, h.data_ptr(),
          nbytes, y.data_ptr())
    return y
