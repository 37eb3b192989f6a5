"""GPU tests of the expert block's corners: segments that begin behind row 0."""
import pytest
import torch

import expert_ref as ref
from combine_moe_layout_05_amd import (
    expert_ffn, gated_grouped_gemm, gated_grouped_gemm_backward, grouped_gemm,
    grouped_gemm_backward_input, grouped_gemm_forward, mxfp4_expert_weights)

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF)


def _spoil(*shape):
    """Leaves NaN in the allocator's next block of this size."""
    t = torch.full(shape, float("nan"), dtype=BF, device=DEV)
    sync_or_fail()
    del t


# Rows before the first segment, in the segments, behind the last one; the
# streamed form of few rows, the tiled forms of many.
@pytest.mark.parametrize("before, counts, behind", [
    (5, (7, 20), 9), (3, (0, 40), 0), (20, (70, 60), 11), (0, (90, 31), 4), (600, (300, 900), 77)])
def test_rows_outside_the_segments_of_a_fresh_output_are_zero(before, counts, behind):
    off = [before + o for o in ref.offsets_of(counts)]
    total, R, D, F, E = off[-1], off[-1] + behind, 96, 2048, 2
    off_d = torch.tensor(off, dtype=torch.int32, device=DEV)
    note(f"segments {off} of {R} rows")
    x, dy = _rand((R, D), 1), _rand((R, D), 2)
    for t in (x, dy):
        t[:before], t[total:] = float("nan"), float("nan")
    x, dy = x.to(DEV), dy.to(DEV)
    w1, w2 = _rand((E, 2 * F, D), 3, D ** -0.5).to(DEV), _rand((E, D, F), 4, F ** -0.5).to(DEV)
    values = torch.randint(0, 256, (E, 2 * F, D // 2), dtype=torch.uint8, device=DEV)
    scales = torch.randint(118, 126, (E, 2 * F, D // 32), dtype=torch.uint8, device=DEV)
    packed = mxfp4_expert_weights(values, scales)
    pre = torch.ones(R, 2 * F, device=DEV)
    calls = {
        "gated": (F, lambda: gated_grouped_gemm(x, w1, off_d)),
        "forward": (2 * F, lambda: grouped_gemm_forward(x, w1, off_d)),
        "backward input": (F, lambda: grouped_gemm_backward_input(dy, w2, off_d)),
        "gated backward": (2 * F, lambda: gated_grouped_gemm_backward(dy, w2, pre, off_d)),
        "4-bit": (2 * F, lambda: grouped_gemm(x, packed, off_d)),
        "4-bit gated": (F, lambda: gated_grouped_gemm(x, packed, off_d)),
    }
    for name, (width, call) in calls.items():
        _spoil(R, width)
        out = call()
        sync_or_fail()
        assert (out[:before].view(torch.int16) == 0).all(), name
        assert (out[total:].view(torch.int16) == 0).all(), name
        assert torch.isfinite(out[before:total]).all(), name
    leaf = x.clone().requires_grad_(True)
    _spoil(R, D)
    y = expert_ffn(leaf, w1, w2, off_d)
    _spoil(R, D)
    grad, = torch.autograd.grad(y, leaf, dy)
    sync_or_fail()
    for t in (y, grad):
        assert (t[:before] == 0).all() and (t[total:] == 0).all()
        assert torch.isfinite(t[before:total]).all()
