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


def _check_gradient(l, K, grad, scale=1.0, renormalize=True):
    ids = ref.select(l, K, "sigmoid")
    want, err = ref.gradient(l, ids, grad, "sigmoid", renormalize, scale)
    leaf = l.to(DEV).requires_grad_(True)
    r = route_topk(leaf, K, score="sigmoid", renormalize=renormalize, scale=scale)
    assert torch.equal(r.ids.cpu().long(), ids)
    got, = torch.autograd.grad(r.scores, leaf, grad.to(DEV))
    direct = route_topk_backward(grad.to(DEV), leaf.detach(), r.ids, score="sigmoid",
                                 renormalize=renormalize, scale=scale)
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


def _far(T, K, seed):
    """Rows of chosen logits from -103 to -86: sigmoids that fp32 holds in few
    bits or in none of an exponential's of the other sign; in some rows beside
    ordinary ones and ones that saturate."""
    l = -86.0 - 17.0 * torch.rand(T, K, generator=_gen(seed))
    l[1::4, 0] = 2.0
    l[2::8, -1] = 95.0
    l[3::8] += 20.0
    return l


# E, K: 16 lanes per token, a wavefront per token
FAR = [(32, 3), (200, 8), (64, 12), (300, 2), (257, 16)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E, K", FAR)
def test_scores_of_small_sigmoids(E, K, renormalize):
    """Off by the relative bound of fp32, and by units of its last place where
    there are no more: one of the exponential times the scale, halves of the
    division and of the product, together less than 4."""
    note(f"small sigmoids E={E} K={K} renormalize={renormalize}")
    l = _rows(_far(64, K, E + K), E)
    ids = ref.select(l, K, "sigmoid")
    want, rel = ref.scores(l, ids, "sigmoid", renormalize, 2.5)
    r = route_topk(l.to(DEV), K, score="sigmoid", renormalize=renormalize, scale=2.5)
    sync_or_fail()
    assert torch.equal(r.ids.cpu().long(), ids)
    off = (r.scores.double().cpu() - want).abs()
    assert (off <= rel * want + 4 * 2.0 ** -149).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E, K", FAR)
def test_gradient_of_small_sigmoids(E, K, renormalize, bf16):
    note(f"gradient of small sigmoids E={E} K={K} renormalize={renormalize} bf16={bf16}")
    l = _rows(_far(64, K, 3 * E + K), E)
    grad = torch.randn(64, K, generator=_gen(E)) * 64
    _check_gradient(l.to(BF) if bf16 else l, K, grad, 2.5, renormalize)


def test_below_the_range_of_fp32_all_scores_are_zero():
    """exp(-103.97) is half of the smallest fp32 number: a token without a
    larger chosen sigmoid has scores and a gradient of 0."""
    l = torch.full((2, 40), -300.0)
    l[0, :4] = -104.0
    l[1, :4] = torch.tensor([-104.0, -103.9, -104.0, -104.0])
    leaf = l.to(DEV).requires_grad_(True)
    r = route_topk(leaf, 4, score="sigmoid")
    got, = torch.autograd.grad(r.scores, leaf, torch.randn(2, 4, generator=_gen(1)).to(DEV))
    sync_or_fail()
    assert (r.scores[0] == 0).all() and (got[0] == 0).all()
    assert float((r.scores.detach()[1].sum() - 1).abs()) <= 8 * ref.U
