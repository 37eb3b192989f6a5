"""GPU tests of the whole layer for a few tokens against a plain 64-bit form
(layer_ref.py holds the formulas and the derivation of the bounds), and of the
router, the layer, 4-bit rows and the separate calls together."""
import pytest
import torch

import expert_ref
import layer_ref as ref
from combine_moe_layout_05_amd import (
    MoeDispatcher, MoeTokenDispatcher, expert_ffn, gated_grouped_gemm, grouped_gemm,
    grouped_gemm_forward, moe_layer, mxfp4_expert_weights, quantize_mxfp4, route_topk)

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ids(T, E, K, seed, drop=0.0):
    order = torch.rand(T, E, generator=_gen(seed)).argsort(dim=1)[:, :K].int()
    lost = torch.rand(T, K, generator=_gen(seed + 1)) < drop
    return torch.where(lost, torch.full_like(order, -1), order)


def _case(T, E, K, D, F, four, seed, drop=0.0):
    x = torch.randn(T, D, generator=_gen(seed)).to(BF)
    scores = torch.softmax(torch.randn(T, K, generator=_gen(seed + 2)), dim=1)
    ids = _ids(T, E, K, seed + 3, drop)
    if four:
        q = [quantized(E, 2 * F, D, seed + 4), quantized(E, D, F, seed + 5)]
        numbers = [ref.decode(*w) for w in q]
        weights = [mxfp4_expert_weights(*(v.to(DEV) for v in w)) for w in q]
    else:
        numbers = [(torch.randn(E, 2 * F, D, generator=_gen(seed + 4)) * D ** -0.5).to(BF),
                   (torch.randn(E, D, F, generator=_gen(seed + 5)) * F ** -0.5).to(BF)]
        weights = [w.to(DEV) for w in numbers]
    return x, scores, ids, numbers, weights


def quantized(E, n, k, seed):
    return ref.quantize(torch.randn(E, n, k, generator=_gen(seed)) * k ** -0.5)


def _run(x, scores, ids, weights, name="silu"):
    return moe_layer(x.to(DEV), scores.to(DEV), ids.to(DEV), *weights, activation=name)


# T, E, K, D, F, share of slots without an expert
SHAPES = [
    (1, 1, 1, 32, 32, 0.0), (1, 8, 2, 64, 96, 0.0), (1, 256, 8, 256, 64, 0.0),
    (1, 16, 3, 1056, 352, 0.0), (3, 8, 2, 128, 256, 0.3), (5, 40, 6, 736, 224, 0.1),
    (17, 3, 3, 160, 96, 0.0), (33, 4, 2, 96, 544, 0.1), (64, 8, 8, 64, 64, 0.0),
    (37, 64, 4, 288, 160, 0.2), (64, 256, 8, 96, 32, 0.0), (32, 300, 16, 64, 32, 0.1),
    (512, 5, 1, 32, 64, 0.0), (13, 1024, 7, 32, 32, 0.0), (40, 2, 2, 320, 2080, 0.0),
    # wide outputs: 32 columns per workgroup
    (1, 6, 4, 4128, 64, 0.0), (9, 12, 3, 4192, 160, 0.1), (64, 16, 8, 4128, 32, 0.0),
    (30, 4, 2, 5152, 96, 0.0),
]
ODD = [(1, 4, 2, 8, 8, 0.0), (7, 6, 3, 72, 40, 0.1), (20, 3, 2, 200, 136, 0.0),
       (2, 9, 4, 1000, 328, 0.0), (6, 5, 2, 4104, 72, 0.0)]     # multiples of 8 alone: bf16


@pytest.mark.parametrize("four, shape", [(f, s) for f in (False, True) for s in SHAPES]
                         + [(False, s) for s in ODD])
def test_layer(shape, four):
    T, E, K, D, F, drop = shape
    note(f"layer {shape} 4-bit={four}")
    x, scores, ids, numbers, weights = _case(T, E, K, D, F, four, sum(shape[:5]), drop)
    # a slot without an expert: its score is not read
    spoiled = torch.where(ids < 0, torch.full_like(scores, float("nan")), scores)
    for name in ("silu", "gelu"):
        want, err = ref.layer(x, scores, ids, *numbers, name)
        y = _run(x, spoiled, ids, weights, name)
        again = _run(x, spoiled, ids, weights, name)
        sync_or_fail()
        expert_ref.check(y, want, err, ref.B, name)
        assert torch.equal(y, again)
        assert (y[(ids < 0).all(dim=1).to(DEV)] == 0).all()


@pytest.mark.parametrize("four", [False, True])
def test_ids_of_no_expert_and_one_expert_twice(four):
    x, scores, ids, numbers, weights = _case(6, 4, 3, 64, 64, four, 5)
    ids[0] = 2                                  # one expert in every slot
    ids[1] = torch.tensor([4, -1, -7])          # nothing
    ids[2] = torch.tensor([2 ** 31 - 1, 1, 1])
    ids[3] = torch.tensor([-2 ** 31, 0, 3])
    y = _run(x, scores, ids, weights)
    want, err = ref.layer(x, scores, torch.where((ids < 0) | (ids > 3), -1, ids), *numbers, "silu")
    expert_ref.check(y, want, err, ref.B, "y")
    assert (y[1] == 0).all()
    ids[:] = -1
    assert (_run(x, scores, ids, weights) == 0).all()


@pytest.mark.parametrize("four", [False, True])
def test_all_slots_on_one_expert(four):
    """512 slots of one expert: many passes over its weights."""
    x, scores, ids, numbers, weights = _case(64, 8, 8, 96, 64, four, 9)
    ids[:] = 5
    y = _run(x, scores, ids, weights)
    want, err = ref.layer(x, scores, ids, *numbers, "silu")
    expert_ref.check(y, want, err, ref.B, "y")


@pytest.mark.parametrize("four", [False, True])
def test_not_a_number_stays_in_its_token(four):
    x, scores, ids, numbers, weights = _case(9, 5, 2, 160, 96, four, 13)
    clean = _run(x, scores, ids, weights)
    bad = x.clone()
    bad[4, 159] = float("inf")
    bad[7, 0] = float("nan")
    y = _run(bad, scores, ids, weights)
    others = [t for t in range(9) if t not in (4, 7)]
    assert torch.equal(y[others], clean[others])
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[4]).any()


def test_no_tokens():
    _, _, _, _, weights = _case(1, 4, 2, 64, 64, False, 3)
    y = moe_layer(torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, 2, device=DEV),
                  torch.empty(0, 2, dtype=torch.int32, device=DEV), *weights)
    assert y.shape == (0, 64)


@pytest.mark.parametrize("four", [False, True])
def test_two_streams_at_once(four):
    """Calls in flight together have workspaces of their own."""
    cases = [_case(8, 16, 4, 512, 256, four, s) for s in (20, 30)]
    args = [(c[0].to(DEV), c[1].to(DEV), c[2].to(DEV), *c[4]) for c in cases]
    want = [moe_layer(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(10):
        for i, (a, s) in enumerate(zip(args, streams)):
            with torch.cuda.stream(s):
                got[i].append(moe_layer(*a))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in (0, 1) for y in got[i])


@pytest.mark.parametrize("four", [False, True])
def test_captured_decode_step(four):
    """Router and layer in a graph, replayed with other tokens, eager work
    between the replays; a second graph shares nothing with the first."""
    T, E, K, D, F = 5, 32, 4, 256, 128
    x0, _, _, _, weights = _case(T, E, K, D, F, four, 40)
    bias = (torch.randn(E, generator=_gen(1)) * 0.1).to(DEV)
    x, logits = x0.to(DEV), torch.zeros(T, E, device=DEV)

    def step():
        r = route_topk(logits, K, score="sigmoid", bias=bias, num_groups=4, topk_groups=2)
        return r.ids, moe_layer(x, r.scores, r.ids, *weights)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for seed in range(4):
        x.copy_(torch.randn(T, D, generator=_gen(seed)).to(BF))
        logits.copy_(torch.randn(T, E, generator=_gen(seed + 9)))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        kept = [[t.clone() for t in out] for _, out in graphs]
        want = step()
        for out in kept:
            assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


# ---- Together -----------------------------------------------------------------

def _dispatched(T, D, E, K, x, r):
    disp = MoeDispatcher(T, D, E, K, dtype=BF, device=DEV)
    lay = disp.layout(r.ids, T)
    dsp = disp.dispatch(x, r.scores, r.ids, lay.counts, num_tokens_per_rank=T)
    return disp, lay, dsp.x_e


@pytest.mark.parametrize("four", [False, True])
def test_layer_and_the_separate_calls(four):
    """The same tokens through layout, dispatch, the products and combine:
    within the layer's bound and that of h's and the rows' roundings to bf16,
    B |h| through w2 and B |y_e| for each slot."""
    T, E, K, D, F = 11, 16, 4, 192, 128
    x, _, _, numbers, weights = _case(T, E, K, D, F, four, 60)
    logits = torch.randn(T, E, generator=_gen(2))
    r = route_topk(logits.to(DEV), K, renormalize=False)
    ids, scores = r.ids.cpu().long(), r.scores.cpu()
    assert torch.equal(ids, ref.select(logits, K, "softmax"))
    disp, lay, x_e = _dispatched(T, D, E, K, x.to(DEV), r)
    h = gated_grouped_gemm(x_e, weights[0], lay.offsets)
    y_e = (grouped_gemm if four else grouped_gemm_forward)(h, weights[1], lay.offsets)
    separate = disp.combine(y_e, lay.row_map, r.scores, num_tokens_per_rank=T).clone()
    y = moe_layer(x.to(DEV), r.scores, r.ids, *weights)
    sync_or_fail()
    want, err = ref.layer(x, scores, ids, *numbers, "silu")
    expert_ref.check(y, want, err, ref.B, "layer")
    more = torch.zeros_like(want)
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            pre = x[t].double() @ numbers[0][e].double().t()
            hh = expert_ref.act("silu", pre[:F])[0] * pre[F:]
            w = numbers[1][e].double()
            more[t] += float(scores[t, k]) * 1.1 * ref.B * (hh.abs() @ w.abs().t() + (w @ hh).abs())
    expert_ref.check(separate, want, err + more, ref.B, "separate calls")


def test_rows_in_4_bits_through_the_whole_path():
    """Router, layout, dispatch, quantised rows, both products, combine; each
    product against the 64-bit form of what it was given."""
    T, E, K, D, F = 150, 8, 2, 256, 96
    x = torch.randn(T, D, generator=_gen(70)).to(BF)
    r = route_topk(torch.randn(T, E, generator=_gen(71)).to(DEV), K, score="sigmoid")
    disp, lay, x_e = _dispatched(T, D, E, K, x.to(DEV), r)
    off = lay.offsets.cpu().tolist()
    total = off[-1]
    assert total == T * K
    w13, w2 = quantized(E, 2 * F, D, 72), quantized(E, D, F, 73)
    p13, p2 = (mxfp4_expert_weights(*(v.to(DEV) for v in w)) for w in (w13, w2))
    q = quantize_mxfp4(x_e)
    h = gated_grouped_gemm(q, p13, lay.offsets)
    q2 = quantize_mxfp4(h)
    y_e = grouped_gemm(q2, p2, lay.offsets)
    y = disp.combine(y_e, lay.row_map, r.scores, num_tokens_per_rank=T)
    sync_or_fail()
    values, scales = ref.quantize(x_e[:total].cpu())
    assert torch.equal(q.values[:total].cpu(), values)
    assert torch.equal(q.scales[:total].cpu(), scales)
    pre, dpre = ref.product(ref.decode(values, scales), ref.decode(*w13), off)
    expert_ref.check(h[:total], *ref.gate(pre, dpre, "silu"), ref.B, "h")
    values, scales = ref.quantize(h[:total].cpu())
    assert torch.equal(q2.values[:total].cpu(), values)
    expert_ref.check(y_e[:total], *ref.product(ref.decode(values, scales), ref.decode(*w2), off),
                     ref.B, "y_e")
    # combine sums bf16 rows in fp32, in slot order
    row = lay.row_map.cpu().long()[:T]
    parts = y_e.cpu().double()[row] * r.scores.cpu().double()[:, :, None]
    expert_ref.check(y, parts.sum(dim=1), expert_ref.gamma(K + 1) * parts.abs().sum(dim=1), ref.B,
                     "y")


def test_training_step_reaches_the_logits():
    """Router, dispatch, expert_ffn and combine with their backward: the
    scores' gradient is the dot product of the slot's row and the output's
    gradient, the logits' follows from it by the router's formula."""
    T, E, K, D, F = 48, 8, 2, 64, 96
    x = torch.randn(T, D, generator=_gen(80)).to(BF).to(DEV).requires_grad_(True)
    logits = torch.randn(T, E, generator=_gen(81)).to(DEV).requires_grad_(True)
    w13 = (torch.randn(E, 2 * F, D, generator=_gen(82)) * D ** -0.5).to(BF).to(DEV)
    w2 = (torch.randn(E, D, F, generator=_gen(83)) * F ** -0.5).to(BF).to(DEV)
    w13.requires_grad_(True)
    w2.requires_grad_(True)
    layer = MoeTokenDispatcher(MoeDispatcher(T, D, E, K, dtype=BF, device=DEV, backward=True))
    r = route_topk(logits, K, renormalize=True, scale=1.5)
    r.scores.retain_grad()
    y_e = expert_ffn(layer.dispatch(x, r.scores, r.ids), w13, w2, layer.disp.offsets)
    y = layer.combine(y_e, r.scores)
    gy = torch.randn(T, D, generator=_gen(84)).to(BF)
    y.backward(gy.to(DEV))
    sync_or_fail()
    ids = r.ids.cpu().long()
    row = layer.disp.row_map[:T].cpu().long()
    rows = y_e.detach().cpu().double()[row]                         # [T, K, D]
    dots, mag = rows @ gy.double()[:, :, None], rows.abs() @ gy.double().abs()[:, :, None]
    gs = r.scores.grad.cpu()
    assert ((gs.double() - dots[:, :, 0]).abs() <= 2 * expert_ref.gamma(D) * mag[:, :, 0]).all()
    want, err = ref.gradient(logits.detach().cpu(), ids, gs, "softmax", True, 1.5)
    got = logits.grad.cpu().double()
    assert ((got - want).abs() <= err + ref.U * got.abs() + 2.0 ** -133).all()
    assert float(got.abs().max()) > 0
    for leaf in (x, w13, w2):
        assert leaf.grad is not None and torch.isfinite(leaf.grad).all()
