"""GPU tests of the router and its gradient against plain 64-bit forms
(layer_ref.py holds the formulas and the derivation of the error bounds)."""
import math

import pytest
import torch

import layer_ref as ref
from combine_moe_layout_05_amd import route_topk, route_topk_backward

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# T, E, K, groups, topk_groups
SHAPES = [
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 8, 2, 1, 1), (5, 60, 6, 1, 1), (4, 64, 8, 4, 2),
    (7, 65, 3, 5, 3), (6, 128, 8, 1, 1), (9, 160, 6, 8, 3), (67, 256, 8, 1, 1),
    (70, 256, 8, 8, 4), (13, 257, 16, 1, 1), (5, 512, 7, 16, 2), (4, 1000, 16, 1, 1),
    (3, 1024, 8, 64, 5), (11, 96, 4, 3, 3), (130, 32, 4, 2, 1),
    # 16 lanes per token: all widths, groups of one lane to all of them
    (9, 17, 8, 1, 1), (33, 48, 5, 1, 1), (21, 200, 8, 1, 1), (18, 32, 3, 16, 5), (18, 64, 8, 8, 3),
    (22, 128, 6, 2, 1), (22, 128, 8, 16, 4), (4100, 64, 4, 4, 2), (19, 256, 8, 16, 9),
    (5, 256, 9, 8, 4), (6, 224, 8, 7, 3),
    # lanes that hold fewer experts than they have places for
    (25, 48, 5, 4, 2), (9, 144, 8, 16, 7), (30, 16, 2, 8, 3), (40, 160, 6, 2, 1),
    (12, 240, 8, 4, 2), (17, 80, 3, 16, 3), (16, 96, 8, 2, 2),
]
KINDS = [("softmax", False), ("sigmoid", False), ("sigmoid", True)]


def _logits(T, E, seed, bf16, scale=1.5):
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * scale
    return l.to(BF) if bf16 else l


def _bias(E, seed):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.1


def _check_scores(got, want, rel):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= rel * want.abs())
    assert not bad.any(), float(((got - want).abs() / want.abs().clamp(min=1e-300)).max())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score, biased", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_choice_and_scores(shape, score, biased, bf16):
    T, E, K, G, kept = shape
    note(f"route {shape} {score} bias={biased} bf16={bf16}")
    l = _logits(T, E, T * E, bf16)
    if T > 3:
        l[1, ::2] = -math.inf                   # half of the experts masked
        l[2] = -math.inf                        # a row that is masked whole
        l[3, 1:] = float("nan")                 # one expert left
    bias = _bias(E, E) if biased else None
    want = ref.select(l, K, score, bias, G, kept)
    for renormalize, scale in ((True, 2.5), (False, 1.0)):
        r = route_topk(l.to(DEV), K, score=score, bias=None if bias is None else bias.to(DEV),
                       renormalize=renormalize, scale=scale, num_groups=G, topk_groups=kept)
        sync_or_fail()
        assert r.ids.dtype == torch.int32 and r.scores.dtype == torch.float32
        assert torch.equal(r.ids.cpu().long(), want)
        _check_scores(r.scores, *ref.scores(l, want, score, renormalize, scale))
        assert not r.scores.requires_grad


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, G, kept", [(256, 1, 1), (256, 8, 4), (60, 4, 2), (1024, 1, 1)])
def test_ties_go_to_the_lowest_index(E, G, kept, score):
    """Few distinct values: every choice is between equal ones."""
    l = torch.randint(0, 3, (64, E), generator=torch.Generator().manual_seed(E)).float()
    bias = None if score == "softmax" else torch.zeros(E)
    for x in (l, l.to(BF), torch.zeros(64, E)):
        want = ref.select(x, 8, score, bias, G, kept)
        r = route_topk(x.to(DEV), 8, score=score, bias=None if bias is None else bias.to(DEV),
                       num_groups=G, topk_groups=kept)
        assert torch.equal(r.ids.cpu().long(), want)


@pytest.mark.parametrize("G, kept", [(1, 1), (8, 4), (4, 1)])
def test_near_values_keep_the_order_of_the_formula(G, kept):
    """Selection values a few 1e-9 apart, which fp32 cannot tell apart: the
    bias undoes the sigmoid up to such a rest."""
    gen = torch.Generator().manual_seed(7)
    T, E = 96, 256
    l = torch.randn(T, E, generator=gen) * 1.5
    l[:, ::3] = l[:, :1]
    near = l[:, :1] + torch.arange(E) * 2.0 ** -23
    l[:, 1::3] = near[:, 1::3]
    bias = torch.zeros(E)
    bias[::5] = 2.0 ** -30
    want = ref.select(l, 8, "sigmoid", bias, G, kept)
    r = route_topk(l.to(DEV), 8, score="sigmoid", bias=bias.to(DEV), num_groups=G,
                   topk_groups=kept)
    assert torch.equal(r.ids.cpu().long(), want)


@pytest.mark.parametrize("E", [256, 128, 23])
@pytest.mark.parametrize("K", [1, 5, 8])
def test_one_expert_near_to_the_last(K, E):
    """The K-th and the next expert alone lie nearer than fp32 can tell, the
    lower or the higher index ahead by the bias, or both equal."""
    gen = torch.Generator().manual_seed(E + K)
    T = 60
    l = torch.stack([torch.randperm(E, generator=gen) for _ in range(T)]).float() / E * 3 - 1.5
    bias = torch.zeros(E)
    bias[1::3], bias[2::3] = 2.0 ** -28, 2.0 ** -29
    order = l.argsort(dim=1, descending=True)
    rows = torch.arange(T)
    l[rows, order[:, K]] = l[rows, order[:, K - 1]]
    want = ref.select(l, K, "sigmoid", bias)
    r = route_topk(l.to(DEV), K, score="sigmoid", bias=bias.to(DEV))
    assert torch.equal(r.ids.cpu().long(), want)
    # a second one, and a third
    l[rows, order[:, K + 1]] = l[rows, order[:, K]]
    l[::2][torch.arange(T // 2), order[::2, K + 2]] = l[::2][torch.arange(T // 2), order[::2, K]]
    want = ref.select(l, K, "sigmoid", bias)
    r = route_topk(l.to(DEV), K, score="sigmoid", bias=bias.to(DEV))
    assert torch.equal(r.ids.cpu().long(), want)


@pytest.mark.parametrize("E, G, kept", [(256, 8, 4), (256, 16, 3), (64, 4, 1), (128, 4, 2),
                                        (32, 16, 8), (256, 2, 1), (160, 8, 3), (48, 4, 2),
                                        (96, 3, 1)])
@pytest.mark.parametrize("biased", [True, False])
def test_groups_near_to_the_last_kept(E, G, kept, biased):
    """The groups' two largest are the same numbers in two, three or all
    groups, or apart by a bias of 2^-28; some groups hold three equal ones, or
    one expert alone."""
    gen = torch.Generator().manual_seed(E + G)
    T, size = 64, E // G
    l = torch.randn(T, G, size, generator=gen) - 2.0
    top = torch.rand(T, G, 2, generator=gen) + 1.0
    top[:24, 1] = top[:24, 0]
    if G > 2:
        top[8:24, 2] = top[8:24, 0].flip(-1)
    top[24:40] = top[24:40, :1]
    for t in range(T):
        for g in range(G):
            at = torch.randperm(size, generator=gen)[:3]
            l[t, g, at[:2]] = top[t, g][:len(at[:2])]
            if t % 4 == 3 and size > 2:
                l[t, g, at[2]] = top[t, g].min()
    l[40:44, ::2, 1:] = float("-inf")
    l = l.reshape(T, E)
    bias = None
    if biased:
        bias = torch.zeros(E)
        bias[torch.randint(0, E, (E // 8,), generator=gen)] = 2.0 ** -28
    K = min(6, size * kept)
    for x in (l, l.to(BF)):
        want = ref.select(x, K, "sigmoid", bias, G, kept)
        r = route_topk(x.to(DEV), K, score="sigmoid", num_groups=G, topk_groups=kept,
                       bias=None if bias is None else bias.to(DEV))
        assert torch.equal(r.ids.cpu().long(), want)


@pytest.mark.parametrize("groups", [(1, 1), (8, 4)])
def test_far_biases_and_near_sums(groups):
    """Biases far below zero: a group's second value decides its sum, and the
    sums of groups lie as near as fp32 numbers of their size."""
    gen = torch.Generator().manual_seed(17)
    T, E = 70, 256
    l = torch.randn(T, E, generator=gen)
    bias = torch.full((E,), -1e6) + torch.randint(0, 4, (E,), generator=gen) * 0.0625
    bias[::32] = torch.randn(8, generator=gen)
    for b in (bias, bias * 1e-3, torch.where(bias < -1, bias, bias - 3e4)):
        want = ref.select(l, 8, "sigmoid", b, *groups)
        r = route_topk(l.to(DEV), 8, score="sigmoid", bias=b.to(DEV), num_groups=groups[0],
                       topk_groups=groups[1])
        assert torch.equal(r.ids.cpu().long(), want)


@pytest.mark.parametrize("E, G, kept", [(256, 8, 4), (256, 1, 1), (128, 4, 2), (160, 8, 3)])
def test_saturated_sigmoids(E, G, kept):
    """Sigmoids that are 1 in 64 bits: without a bias the logits decide, with
    one the index does between them."""
    gen = torch.Generator().manual_seed(E)
    l = 60.0 + torch.randn(40, E, generator=gen)
    l[:, ::7] = torch.randn(40, len(range(0, E, 7)), generator=gen)
    for dtype in (torch.float32, BF):
        for bias in (None, torch.zeros(E)):
            x = l.to(dtype)
            want = ref.select(x, 6, "sigmoid", bias, G, kept)
            r = route_topk(x.to(DEV), 6, score="sigmoid", num_groups=G, topk_groups=kept,
                           bias=None if bias is None else bias.to(DEV))
            assert torch.equal(r.ids.cpu().long(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_further_apart_than_a_key_holds(score):
    """Distances above 16 and below 2^-20 between the chosen."""
    gen = torch.Generator().manual_seed(18)
    far = torch.randn(64, 256, generator=gen) * 1000
    near = 3.0 + torch.randint(0, 1 << 14, (64, 256), generator=gen) * 2.0 ** -22
    for l in (far, near, near - 1e5, near * 1e-8):
        want = ref.select(l, 8, score)
        assert torch.equal(route_topk(l.to(DEV), 8, score=score).ids.cpu().long(), want)


@pytest.mark.parametrize("big", [0.0, 100.0, 1e6, -1e6])
def test_far_values(big):
    """Logits and biases far from zero, a bias of infinity either way."""
    l = _logits(40, 256, 5, False, 30.0) + big
    bias = _bias(256, 3) * 1000
    bias[7], bias[9], bias[11] = math.inf, -math.inf, float("nan")
    for score, b in (("softmax", None), ("sigmoid", bias), ("sigmoid", None)):
        for G, kept in ((1, 1), (8, 4)):
            want = ref.select(l, 8, score, b, G, kept)
            r = route_topk(l.to(DEV), 8, score=score, bias=None if b is None else b.to(DEV),
                           num_groups=G, topk_groups=kept, renormalize=score == "softmax")
            assert torch.equal(r.ids.cpu().long(), want), (score, G)
            assert torch.isfinite(r.scores).all()
            if b is not None:
                assert (r.ids != 9).all() and (r.ids != 11).all()


@pytest.mark.parametrize("E", [64, 256])
def test_infinite_logits(E):
    """+inf: the largest of the choice; a softmax over it is NaN, as the
    formula says, a sigmoid 1."""
    l = _logits(4, E, 9, False)
    l[0, 5] = math.inf
    r = route_topk(l.to(DEV), 4, score="softmax", renormalize=False)
    assert int(r.ids[0, 0]) == 5 and bool(torch.isnan(r.scores[0]).all())
    assert torch.isfinite(r.scores[1:]).all()
    r = route_topk(l.to(DEV), 4, score="sigmoid", renormalize=False)
    assert int(r.ids[0, 0]) == 5 and float(r.scores[0, 0]) == 1.0


def test_a_sum_of_zero_gives_zeros():
    """Sigmoids below fp32's range: no quotient of zeros."""
    l = torch.full((3, 32), -200.0)
    l.requires_grad_(True)
    r = route_topk(l.detach().to(DEV).requires_grad_(True), 4, score="sigmoid")
    assert (r.scores == 0).all() and r.ids.tolist() == [[0, 1, 2, 3]] * 3


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score, biased", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient(shape, score, biased, renormalize, bf16):
    T, E, K, G, kept = shape
    note(f"route gradient {shape} {score} bias={biased} renorm={renormalize} bf16={bf16}")
    l = _logits(T, E, 3 * T * E, bf16)
    if T > 3:
        l[1, ::2] = -math.inf
        l[2] = -math.inf
        l[3, 1:] = float("nan")
    bias = _bias(E, E) if biased else None
    ids = ref.select(l, K, score, bias, G, kept)
    grad = torch.randn(T, K, generator=torch.Generator().manual_seed(T + E))
    want, err = ref.gradient(l, ids, grad, score, renormalize, 2.5)
    leaf = l.to(DEV).requires_grad_(True)
    r = route_topk(leaf, K, score=score, bias=None if bias is None else bias.to(DEV),
                   renormalize=renormalize, scale=2.5, num_groups=G, topk_groups=kept)
    assert torch.equal(r.ids.cpu().long(), ids) and not r.ids.requires_grad
    got, = torch.autograd.grad(r.scores, leaf, grad.to(DEV))
    direct = route_topk_backward(grad.to(DEV), leaf.detach(), r.ids, score=score,
                                 renormalize=renormalize, scale=2.5)
    sync_or_fail()
    assert got.dtype == l.dtype and torch.equal(got, direct)
    got = got.double().cpu()
    half = ref.B if bf16 else ref.U
    # bf16 keeps multiples of 2^-133 below its normal numbers, fp32 of 2^-149.
    assert ((got - want).abs() <= err + half * got.abs() + 2.0 ** -133).all()


@pytest.mark.parametrize("score, renormalize", [("softmax", True), ("softmax", False),
                                                ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, renormalize):
    """Central differences of the 64-bit scores: off by h^2 / 6 times a third
    derivative, which is at most 2 p scale for these functions' magnitudes."""
    T, E, K, h = 2, 24, 4, 1e-4
    l = _logits(T, E, 21, False)
    ids = ref.select(l, K, score)
    grad = torch.randn(T, K, generator=torch.Generator().manual_seed(2))
    r = route_topk(l.to(DEV).requires_grad_(True), K, score=score, renormalize=renormalize)
    assert torch.equal(r.ids.cpu().long(), ids)
    got = route_topk_backward(grad.to(DEV), l.to(DEV), r.ids, score=score,
                              renormalize=renormalize).double().cpu()
    f = lambda x: (ref.scores(x, ids, score, renormalize, 1.0)[0] * grad.double()).sum()
    for t in range(T):
        for e in range(E):
            step = torch.zeros(T, E, dtype=torch.float64)
            step[t, e] = h
            d = (f(l.double() + step) - f(l.double() - step)) / (2 * h)
            assert abs(float(got[t, e] - d)) <= 20 * h * h + 1e-6 * float(grad.abs().sum())


def test_an_expert_in_two_slots():
    """ids of the caller's own: the contributions add; ids outside are none."""
    l = _logits(2, 16, 4, False)
    grad = torch.tensor([[1.0, 2.0, 3.0], [1.0, -1.0, 0.5]])
    ids = torch.tensor([[3, 3, 5], [16, 2, -1]], dtype=torch.int32)
    got = route_topk_backward(grad.to(DEV), l.to(DEV), ids.to(DEV), score="sigmoid",
                              renormalize=False).cpu().double()
    s = torch.sigmoid(l.double())
    want = torch.zeros(2, 16, dtype=torch.float64)
    want[0, 3], want[0, 5], want[1, 2] = 3.0, 3.0, -1.0
    assert ((got - want * s * (1 - s)).abs() <= 64 * ref.U).all()


def test_logits_that_begin_anywhere():
    """A slice of a larger tensor: aligned to an element only."""
    for dtype in (torch.float32, BF):
        big = torch.randn(1 + 9 * 256, generator=torch.Generator().manual_seed(6)).to(dtype)
        l = big[1:].view(9, 256)
        want = ref.select(l, 8, "softmax")
        d = big.to(DEV)[1:].view(9, 256)
        assert torch.equal(route_topk(d, 8).ids.cpu().long(), want)
        a = route_topk_backward(torch.ones(9, 8, device=DEV), d, route_topk(d, 8).ids,
                                renormalize=False)
        b = route_topk_backward(torch.ones(9, 8, device=DEV), l.to(DEV), route_topk(d, 8).ids,
                                renormalize=False)
        assert torch.equal(a, b)


def test_no_tokens():
    l = torch.empty(0, 16, device=DEV, requires_grad=True)
    r = route_topk(l, 2)
    assert r.ids.shape == (0, 2) and r.scores.shape == (0, 2)
    g, = torch.autograd.grad(r.scores.sum(), l)
    assert g.shape == (0, 16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_captured_step(score):
    """Forward and backward captured together and replayed with other logits,
    eager work between the replays."""
    T, E, K = 37, 256, 8
    bias = None if score == "softmax" else _bias(E, 1).to(DEV)
    leaf = torch.zeros(T, E, device=DEV, requires_grad=True)
    grad = torch.randn(T, K, generator=torch.Generator().manual_seed(8)).to(DEV)

    def step():
        r = route_topk(leaf, K, score=score, bias=bias, num_groups=8, topk_groups=4)
        return r.ids, r.scores.detach(), torch.autograd.grad(r.scores, leaf, grad)[0]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for seed in range(4):
        with torch.no_grad():
            leaf.copy_(_logits(T, E, seed, False))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        with torch.cuda.stream(side):
            want = step()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), seed


def test_capture_beside_an_eager_graph_is_refused():
    """The leaf's accumulator belongs to the default stream: a captured
    backward on it would end the process."""
    leaf = torch.randn(4, 16, device=DEV, requires_grad=True)
    alive = route_topk(leaf, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="route_topk cannot be captured"):
        with torch.cuda.graph(graph):
            route_topk(leaf, 2)
    torch.cuda.synchronize()
    assert alive.scores.shape == (4, 2)


def test_another_stream():
    l = _logits(300, 256, 12, False).to(DEV)
    want = route_topk(l, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = route_topk(l, 8)
    s.synchronize()
    assert torch.equal(got.ids, want.ids) and torch.equal(got.scores, want.scores)
