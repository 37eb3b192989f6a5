"""GPU tests of the router's choice between values nearer than fp32 can tell,
in the form that takes a wavefront per token: more than 256 experts, more than 8
of them per token, groups that do not cover whole lanes (layer_ref.py has the
plain form)."""
import pytest
import torch

import layer_ref as ref
from combine_moe_layout_05_amd import route_topk

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# E, K, groups, topk_groups
SHAPES = [(257, 8, 1, 1), (384, 8, 8, 4), (512, 10, 16, 5), (1000, 16, 1, 1), (1024, 16, 64, 9),
          (256, 10, 1, 1), (256, 16, 8, 4), (224, 8, 7, 3), (60, 9, 5, 2), (96, 12, 32, 6)]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


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
            want = ref.select(x, K, "sigmoid", b, G, kept)
            r = route_topk(x.to(DEV), K, score="sigmoid", num_groups=G, topk_groups=kept,
                           bias=None if b is None else b.to(DEV))
            assert torch.equal(r.ids.cpu().long(), want), (x.dtype, b is None)
        want = ref.select(x, K, "softmax", None, G, kept)
        r = route_topk(x.to(DEV), K, num_groups=G, topk_groups=kept)
        assert torch.equal(r.ids.cpu().long(), want), x.dtype
