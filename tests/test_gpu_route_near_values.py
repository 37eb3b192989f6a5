"""GPU tests of the router's choice between values nearer than fp32 can tell,
in the form that takes a wavefront per token: more than 256 experts, more than 8
of them per token, groups that do not cover whole lanes."""
import math

import pytest
import torch

from combine_moe_layout_05_amd import route_topk

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# E, K, groups, topk_groups
SHAPES = [(257, 8, 1, 1), (384, 8, 8, 4), (512, 10, 16, 5), (1000, 16, 1, 1), (1024, 16, 64, 9),
          (256, 10, 1, 1), (256, 16, 8, 4), (224, 8, 7, 3), (60, 9, 5, 2), (96, 12, 32, 6)]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _select(logits, K, score, bias, G, kept):
    """ids [T, K], one number after the other: equal logits have equal sigmoids
    wherever they stand in a row, which a vectorized exponential and the form of
    it that takes a row's last elements need not give. The logits are finite and
    the kept groups hold K experts."""
    T, E = logits.shape
    size = E // G
    out = torch.empty(T, K, dtype=torch.int64)
    for t, l in enumerate(logits.double().tolist()):
        counts = v = l
        if score == "sigmoid":
            counts = [1.0 / (1.0 + math.exp(-x)) for x in l]
            if bias is not None:
                counts = v = [p + b for p, b in zip(counts, bias.double().tolist())]
        value = []
        for g in range(G):
            mine = sorted(range(g * size, (g + 1) * size), key=lambda e: (-v[e], e))
            value.append(sum(counts[e] for e in mine[:2 if score == "sigmoid" else 1]))
        best = sorted(range(G), key=lambda g: (-value[g], g))[:kept]
        ok = [e for e in range(E) if e // size in best]
        out[t] = torch.tensor(sorted(ok, key=lambda e: (-v[e], e))[:K])
    return out


@pytest.mark.parametrize("E, K, G, kept", SHAPES)
def test_near_values(E, K, G, kept):
    """A third of the experts at one logit and a third at steps of 2^-23 from
    it, biases that part equal ones by 2^-30, and sums of groups as near."""
    note(f"near values E={E} K={K} groups={G}/{kept}")
    gen = _gen(E + K)
    l = torch.randn(48, E, generator=gen) * 1.5
    l[:, ::3] = l[:, :1]
    l[:, 1::3] = (l[:, :1] + torch.arange(E) * 2.0 ** -23)[:, 1::3]
    l[::6] += 2.0
    bias = torch.zeros(E)
    bias[::5] = 2.0 ** -30
    for x in (l, l.to(BF)):
        for b in (bias, None):
            want = _select(x, K, "sigmoid", b, G, kept)
            r = route_topk(x.to(DEV), K, score="sigmoid", num_groups=G, topk_groups=kept,
                           bias=None if b is None else b.to(DEV))
            assert torch.equal(r.ids.cpu().long(), want), (x.dtype, b is None)
        want = _select(x, K, "softmax", None, G, kept)
        r = route_topk(x.to(DEV), K, num_groups=G, topk_groups=kept)
        assert torch.equal(r.ids.cpu().long(), want), x.dtype
