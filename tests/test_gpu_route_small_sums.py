"""GPU tests of the renormalized sigmoid router where the chosen sigmoids are
as small as fp32 numbers get, against plain 64-bit forms (layer_ref.py)."""
import math

import pytest
import torch

import layer_ref as ref
from combine_moe_layout_05_amd import route_topk, route_topk_backward

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(chosen, E):
    """Logits [T, E] with the given ones at places of each row's own, all
    others -inf."""
    T, K = chosen.shape
    l = torch.full((T, E), -math.inf)
    for t in range(T):
        l[t, torch.randperm(E, generator=_gen(t))[:K]] = chosen[t]
    return l


def _check_gradient(l, K, grad, scale=1.0):
    ids = ref.select(l, K, "sigmoid")
    want, err = ref.gradient(l, ids, grad, "sigmoid", True, scale)
    leaf = l.to(DEV).requires_grad_(True)
    r = route_topk(leaf, K, score="sigmoid", scale=scale)
    assert torch.equal(r.ids.cpu().long(), ids)
    got, = torch.autograd.grad(r.scores, leaf, grad.to(DEV))
    direct = route_topk_backward(grad.to(DEV), leaf.detach(), r.ids, score="sigmoid", scale=scale)
    sync_or_fail()
    assert torch.isfinite(got).all() and torch.equal(got, direct)
    got = got.double().cpu()
    half = ref.B if l.dtype == BF else ref.U
    # bf16 keeps multiples of 2^-133 below its normal numbers, fp32 of 2^-149.
    assert ((got - want).abs() <= err + half * got.abs() + 2.0 ** -133).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [32, 257])
def test_gradient_of_small_sums(E, bf16):
    """Sums of the chosen sigmoids down to 2^-127, upstream gradients up to
    2^16 as a scaled loss has them, and a sigmoid of 0 beside one that is not:
    no quotient may leave fp32 on the way to a finite gradient."""
    note(f"gradient of small sums E={E} bf16={bf16}")
    chosen = [(-88.0, -88.0), (-88.0, -88.0), (-80.0, -200.0), (-88.0, -200.0), (-76.0, -76.5)]
    grad = [(5.0, -5.0), (65536.0, -65536.0), (65536.0, 0.0), (1.0, -5.0), (65536.0, 1.0)]
    for a in range(24):
        first = -76.0 - 0.5 * a
        for second in (first - 0.5, -88.5, -200.0):
            chosen.append((first, second))
            g = torch.randn(2, generator=_gen(len(chosen))) * 2.0 ** (16 * (a % 2))
            grad.append(tuple(g.tolist()))
    l = _rows(torch.tensor(chosen), E)
    _check_gradient(l.to(BF) if bf16 else l, 2, torch.tensor(grad))


@pytest.mark.parametrize("E", [32, 257])
def test_gradient_of_a_sum_of_zero(E):
    """Scores that are 0 whatever the logits are have a gradient of 0."""
    l = torch.full((3, E), -200.0)
    grad = torch.tensor([[1.0, -2.0, 65536.0]] * 3, device=DEV)
    leaf = l.to(DEV).requires_grad_(True)
    r = route_topk(leaf, 3, score="sigmoid")
    assert (r.scores == 0).all()
    got, = torch.autograd.grad(r.scores, leaf, grad)
    sync_or_fail()
    assert (got == 0).all()
