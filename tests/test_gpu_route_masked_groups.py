"""GPU tests of the grouped sigmoid router where whole groups are masked, by
logits or by the bias: the choice against a plain form (layer_ref.py), and that
such tokens stay in the form made for them."""
import math

import pytest
import torch

import layer_ref as ref
from combine_moe_layout_05_amd import route_topk

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("by", ["logits", "bias", "logits without a bias"])
@pytest.mark.parametrize("E, G, kept", [(256, 8, 4), (64, 4, 2), (160, 8, 3), (256, 16, 5),
                                        (32, 16, 8), (96, 3, 1), (512, 8, 4)])
def test_choice_beside_masked_groups(E, G, kept, by):
    """One group masked, several, all but the kept ones, more than those, and
    all; in other tokens the last kept group and the next lie near each other, or
    a logit or a bias is infinite."""
    note(f"masked groups {E} / {G}, {kept} kept, by {by}")
    T, K = 48, min(6, E // G * kept)
    gone = [0, 1, 2, G - kept, min(G, G - kept + 1), G]
    for i, n in enumerate(gone):
        gen = _gen(E + 10 * i)
        l = torch.randn(T, G, E // G, generator=gen) * 1.5
        bias = None if by == "logits without a bias" else torch.randn(G, E // G, generator=gen) * 0.1
        dead = torch.randperm(G, generator=gen)[:n]
        if by == "bias":
            bias[dead] = -math.inf
        else:
            l[:, dead] = -math.inf
        live = [g for g in range(G) if g not in dead.tolist()]
        if len(live) > 1:
            l[::5, live[0]] = l[::5, live[1]]
            if bias is not None:
                bias[live[0]] = bias[live[1]]
        if live and bias is not None:
            l[7::9, live[-1], 0] = math.inf
            bias[live[-1], -1] = math.inf if i % 2 else 1e5
        l = l.view(T, E)
        b = None if bias is None else bias.view(E)
        for x in (l, l.to(BF)):
            want = ref.select(x, K, "sigmoid", b, G, kept)
            r = route_topk(x.to(DEV), K, score="sigmoid", num_groups=G, topk_groups=kept,
                           bias=None if b is None else b.to(DEV))
            assert torch.equal(r.ids.cpu().long(), want), (n, x.dtype)


def _least_time(f):
    for _ in range(3):
        f()
    times = []
    for _ in range(20):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        times.append((a, b))
    torch.cuda.synchronize()
    return min(a.elapsed_time(b) for a, b in times)


@pytest.mark.parametrize("by", ["logits", "bias"])
def test_a_masked_group_costs_nothing(by):
    """Tokens that are chosen for one after the other by a whole wavefront take
    seven times as long; a masked group sends none there."""
    T, E = 32768, 256
    l = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    bias = torch.randn(E, generator=_gen(2)).to(DEV) * 0.1
    run = lambda x, b: _least_time(lambda: route_topk(x, 8, score="sigmoid", bias=b, num_groups=8,
                                                      topk_groups=4))
    whole = run(l, bias)
    masked, some = l.clone(), bias.clone()
    (masked[:, 64:96] if by == "logits" else some[64:96]).fill_(-math.inf)
    assert run(masked, some) < 3 * whole
