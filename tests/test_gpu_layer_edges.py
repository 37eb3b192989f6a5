"""GPU tests of the router, of 4-bit rows and of the layer for a few tokens
where the calls are legal and rare: buffers past 4 GiB, masks of the type's
lowest value, padded batches, calls on other streams and threads."""
import threading

import pytest
import torch

import expert_ref
import layer_ref as ref
from combine_moe_layout_05_amd import (
    MoeDispatcher, MoeTokenDispatcher, Mxfp4Rows, dequantize_mxfp4, expert_ffn,
    gated_grouped_gemm, grouped_gemm, moe_layer, mxfp4_expert_weights, quantize_mxfp4, route_topk,
    route_topk_backward)

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _gpu_gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_router_past_4_gib(dtype):
    """The last tokens of a batch whose logits take more than 4 GiB, and
    whose gradient does, against a call on them alone."""
    T = (1 << 32) // (256 * torch.finfo(dtype).bits // 8) + 5000
    note(f"router past 4 GiB: T={T} {dtype}")
    l = torch.zeros(T, 256, dtype=dtype, device=DEV)
    l[-4000:] = torch.randn(4000, 256, generator=_gpu_gen(1), device=DEV).to(dtype)
    r = route_topk(l, 8, renormalize=False)
    alone = route_topk(l[-4000:].clone(), 8, renormalize=False)
    assert torch.equal(r.ids[-4000:], alone.ids) and torch.equal(r.scores[-4000:], alone.scores)
    assert (r.ids[:-4000] == torch.arange(8, dtype=torch.int32, device=DEV)).all()
    g = torch.randn(T, 8, generator=_gpu_gen(2), device=DEV)
    d = route_topk_backward(g, l, r.ids, renormalize=False)
    want = route_topk_backward(g[-4000:].clone(), l[-4000:].clone(), alone.ids, renormalize=False)
    sync_or_fail()
    assert torch.equal(d[-4000:], want)


def test_router_of_the_most_tokens():
    """2^26 - 1 tokens, a wavefront each: whole workgroups of four would be a
    launch of 2^32 threads."""
    T, E, last = (1 << 26) - 1, 257, 9
    note(f"router of {T} tokens of {E} experts")
    l = torch.zeros(T, E, dtype=BF, device=DEV)
    l[-last:] = torch.randn(last, E, generator=_gpu_gen(2), device=DEV).to(BF)
    r = route_topk(l, 1, renormalize=False)
    alone = route_topk(l[-last:].clone(), 1, renormalize=False)
    assert torch.equal(r.ids[-last:], alone.ids) and torch.equal(r.scores[-last:], alone.scores)
    assert (r.ids[:-last] == 0).all()
    grad = route_topk_backward(torch.ones_like(r.scores), l, r.ids, renormalize=False)
    want = route_topk_backward(torch.ones_like(alone.scores), l[-last:].clone(), alone.ids,
                               renormalize=False)
    assert torch.equal(grad[-last:], want) and torch.equal(grad[5], grad[0])
    del l, r, grad
    torch.cuda.empty_cache()


def test_quantisation_past_4_gib():
    """2^31 elements and some: bf16 values, fp32 ones past 8 GiB, and back."""
    R, K = (1 << 31) // 7168 + 40, 7168
    note(f"quantise {R} x {K}")
    for dtype in (BF, torch.float32):
        x = torch.zeros(R, K, dtype=dtype, device=DEV)
        x[-64:] = torch.randn(64, K, generator=_gpu_gen(3), device=DEV).to(dtype)
        q = quantize_mxfp4(x)
        want = quantize_mxfp4(x[-64:].clone())
        assert torch.equal(q.values[-64:], want.values)
        assert torch.equal(q.scales[-64:], want.scales)
        assert not q.values[:-64].any() and not q.scales[:-64].any()
        back = dequantize_mxfp4(q, dtype)
        assert torch.equal(back[-64:], dequantize_mxfp4(want, dtype))
        assert not back[:-64].any()
        del x, q, back
    sync_or_fail()


def test_products_past_4_gib():
    """4-bit rows past 4 GiB, in the tiled form, against a call on the last
    ones alone, in the streamed form: one rounding apart at most."""
    R, K, N, last = (1 << 32) // 3584 + 100, 7168, 16, 40
    note(f"4-bit rows {R} x {K}")
    values = torch.zeros(R, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((R, K // 32), 127, dtype=torch.uint8, device=DEV)
    tail = quantize_mxfp4(torch.randn(last, K, generator=_gpu_gen(4), device=DEV))
    values[-last:], scales[-last:] = tail
    w = [torch.randint(0, 256, (2, N, K // 2), generator=_gen(5), dtype=torch.uint8),
         torch.randint(118, 122, (2, N, K // 32), generator=_gen(6), dtype=torch.uint8)]
    packed = mxfp4_expert_weights(*(v.to(DEV) for v in w))
    off = torch.tensor([0, R - last, R], dtype=torch.int32, device=DEV)
    out = grouped_gemm(Mxfp4Rows(values, scales), packed, off)
    assert not out[:-last].any()
    want, err = ref.product(ref.decode(*(v.cpu() for v in tail)), ref.decode(*w), [0, 0, last])
    expert_ref.check(out[-last:], want, err, ref.B, "last rows")
    del out
    h = gated_grouped_gemm(Mxfp4Rows(values, scales), mxfp4_expert_weights(
        *(v.repeat(1, 2, 1).to(DEV) for v in w)), off)
    pre, dpre = ref.product(ref.decode(*(v.cpu() for v in tail)),
                            ref.decode(*(v.repeat(1, 2, 1) for v in w)), [0, 0, last])
    sync_or_fail()
    expert_ref.check(h[-last:], *ref.gate(pre, dpre, "silu"), ref.B, "last rows, gated")


@pytest.mark.parametrize("four", [False, True])
def test_layer_weights_past_4_gib(four):
    """The last of many experts against a call that holds it alone."""
    D, F, T = 7168, 2048, 3
    E = 300 if four else 80
    note(f"layer with {E} experts of {D} x {F}, 4 bits {four}")
    if four:
        def make(n, k):
            v = torch.randint(0, 256, (E, n, k // 2), generator=_gpu_gen(7), device=DEV,
                              dtype=torch.uint8)
            s = torch.randint(117, 121, (E, n, k // 32), generator=_gpu_gen(8), device=DEV,
                              dtype=torch.uint8)
            return (mxfp4_expert_weights(v, s),
                    mxfp4_expert_weights(v[-1:].contiguous(), s[-1:].contiguous()))
        (w1, one1), (w2, one2) = make(2 * F, D), make(D, F)
    else:
        w1 = torch.zeros(E, 2 * F, D, dtype=BF, device=DEV)
        w2 = torch.zeros(E, D, F, dtype=BF, device=DEV)
        w1[-1].normal_(0, D ** -0.5, generator=_gpu_gen(9))
        w2[-1].normal_(0, F ** -0.5, generator=_gpu_gen(10))
        one1, one2 = w1[-1:].clone(), w2[-1:].clone()
    x = torch.randn(T, D, generator=_gpu_gen(11), device=DEV).to(BF)
    s = torch.rand(T, 1, generator=_gpu_gen(12), device=DEV)
    y = moe_layer(x, s, torch.full((T, 1), E - 1, dtype=torch.int32, device=DEV), w1, w2)
    want = moe_layer(x, s, torch.zeros(T, 1, dtype=torch.int32, device=DEV), one1, one2)
    sync_or_fail()
    assert torch.equal(y, want) and bool(y.float().abs().max() > 0)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("E, G, kept", [(256, 1, 1), (256, 8, 4), (160, 8, 3), (24, 1, 1)])
def test_masks_of_the_lowest_value(E, G, kept, dtype):
    """Logits masked with the type's lowest number: they take part, behind all
    others; a row of them is a choice between equal ones."""
    low = torch.finfo(dtype).min
    l = torch.randn(40, E, generator=_gen(E)).to(dtype)
    l[1], l[2, 3:], l[3, ::2], l[4, : E // 2] = low, low, low, low
    for score, bias in (("softmax", None), ("sigmoid", None), ("sigmoid", torch.zeros(E))):
        want = ref.select(l, 6, score, bias, G, kept)
        for renormalize in (False, True):
            r = route_topk(l.to(DEV), 6, score=score, renormalize=renormalize, num_groups=G,
                           topk_groups=kept, bias=None if bias is None else bias.to(DEV))
            assert torch.equal(r.ids.cpu().long(), want)
            assert torch.isfinite(r.scores).all()
            g = route_topk_backward(torch.ones(40, 6, device=DEV), l.to(DEV), r.ids, score=score,
                                    renormalize=renormalize)
            assert torch.isfinite(g).all()
        if score == "softmax":
            sums = r.scores.sum(dim=1).cpu()
            assert ((sums - 1).abs() <= 16 * ref.U).all()


def test_padded_batch_through_the_training_path():
    """Tokens whose logits are all -inf: no expert, a zero row of y, no
    gradient anywhere; the other tokens as without them."""
    T, E, K, D, F, keep = 24, 8, 2, 64, 32, 17
    x = torch.randn(T, D, generator=_gen(1)).to(BF)
    logits = torch.randn(T, E, generator=_gen(2))
    logits[keep:] = float("-inf")
    w13 = (torch.randn(E, 2 * F, D, generator=_gen(3)) * D ** -0.5).to(BF).to(DEV)
    w2 = (torch.randn(E, D, F, generator=_gen(4)) * F ** -0.5).to(BF).to(DEV)
    gy = torch.randn(T, D, generator=_gen(5)).to(BF).to(DEV)

    def run(n):
        xs = x[:n].to(DEV).requires_grad_(True)
        ls = logits[:n].to(DEV).requires_grad_(True)
        layer = MoeTokenDispatcher(MoeDispatcher(T, D, E, K, dtype=BF, device=DEV, backward=True))
        r = route_topk(ls, K, score="sigmoid")
        y = layer.combine(expert_ffn(layer.dispatch(xs, r.scores, r.ids), w13, w2,
                                     layer.disp.offsets), r.scores)
        y.backward(gy[:n])
        sync_or_fail()
        return r, y.detach(), xs.grad, ls.grad

    r, y, gx, gl = run(T)
    assert (r.ids[keep:] == -1).all() and (r.scores[keep:] == 0).all()
    for t in (y, gx, gl):
        assert (t[keep:] == 0).all()
    r0, y0, gx0, gl0 = run(keep)
    assert torch.equal(r.ids[:keep], r0.ids) and torch.equal(y[:keep], y0)
    assert torch.equal(gx[:keep], gx0) and torch.equal(gl[:keep], gl0)


def test_calls_from_two_threads():
    """Each thread with a stream and inputs of its own."""
    E, K, D, F, T = 16, 4, 256, 128, 9
    w1 = (torch.randn(E, 2 * F, D, generator=_gen(1)) * D ** -0.5).to(BF).to(DEV)
    w2 = (torch.randn(E, D, F, generator=_gen(2)) * F ** -0.5).to(BF).to(DEV)
    inputs = [(torch.randn(T, D, generator=_gen(s)).to(BF).to(DEV),
               torch.randn(T, E, generator=_gen(s + 9)).to(DEV)) for s in (3, 4)]

    def once(x, logits):
        r = route_topk(logits, K)
        return moe_layer(x, r.scores, r.ids, w1, w2), quantize_mxfp4(x).values

    want = [once(*i) for i in inputs]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[k].append(once(*inputs[k]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:          # told to the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and all(len(g) == 20 for g in got)
    for k in (0, 1):
        assert all(torch.equal(a, b) for g in got[k] for a, b in zip(g, want[k]))
