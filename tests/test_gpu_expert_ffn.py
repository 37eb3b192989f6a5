"""GPU tests of the gated expert block, its gradients and the products with
4-bit weights against plain 64-bit forms (expert_ref.py holds the formulas and
the derivation of the error bounds)."""
import pytest
import torch

import expert_ref as ref
from combine_moe_layout_05_amd import (
    MoeDispatcher, MoeTokenDispatcher, expert_ffn, gated_grouped_gemm,
    gated_grouped_gemm_backward, grouped_gemm, grouped_gemm_backward_input,
    grouped_gemm_backward_weight, grouped_gemm_forward, mxfp4_expert_weights)

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
POISON = 0x7F7F            # bf16 bits no kernel writes here


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * scale).to(BF)


def _rows(rows, width, total, seed, scale=1.0):
    """Rows behind the last segment hold NaN: they must never be read."""
    t = _rand((rows, width), seed, scale)
    t[total:] = float("nan")
    return t


def _poisoned(*shape):
    return torch.full(shape, POISON, dtype=torch.int16, device=DEV).view(BF)


def _is_poison(t):
    return bool((t.view(torch.int16) == POISON).all())


def _off(counts):
    off = ref.offsets_of(counts)
    return off, torch.tensor(off, dtype=torch.int32, device=DEV)


# counts, rows behind the last segment, k_in, n_hidden (or n_out)
SHAPES = [
    ([1], 0, 8, 8),                              # one row, one chunk
    ([1, 0, 1, 1, 0, 0, 1, 2], 26, 256, 64),     # a few rows on many experts
    ([3, 0, 7, 17, 1], 12, 1992, 1000),          # ragged sums and features
    ([40, 33, 0, 2, 90], 3, 136, 72),            # 64-row tiles
    ([0, 65, 1, 130, 7], 37, 72, 200),
    ([120, 0, 260, 131], 9, 264, 328),           # 128-row tiles
    ([513, 700, 5], 22, 328, 280),               # 256-row tiles
    ([256, 512], 0, 512, 256),                   # whole tiles everywhere
    ([0, 0, 0], 40, 64, 32),                     # no rows at all
    ([int(i % 5 == 0) * (i % 7) for i in range(300)], 5, 64, 40),   # experts > lanes
]
IDS = [f"{i}" for i in range(len(SHAPES))]


def _case(i):
    counts, tail, k, n = SHAPES[i]
    off, off_d = _off(counts)
    return len(counts), off, off_d, off[-1], off[-1] + tail, k, n


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_gated_forward(i, name):
    E, off, off_d, total, R, D, F = _case(i)
    note(f"gated E={E} rows={total}/{R} D={D} F={F} {name}")
    x = _rows(R, D, total, i)
    w = _rand((E, 2 * F, D), 50 + i, 1.5 * D ** -0.5)
    h, err, pre, dpre = ref.gated(x[:total], w, off, name)
    xd, wd = x.to(DEV), w.to(DEV)
    out = _poisoned(R, F)
    pre_d = torch.full((R, 2 * F), 7.0, device=DEV)
    assert gated_grouped_gemm(xd, wd, off_d, out, activation=name, pre=pre_d) is out
    fresh = gated_grouped_gemm(xd, wd, off_d, activation=name)
    sync_or_fail()
    ref.check(out[:total], h, err, ref.B, "h")
    ref.check(pre_d[:total], pre, dpre, 0.0, "pre")
    assert _is_poison(out[total:]) and (pre_d[total:] == 7.0).all()
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_plain_forward(i):
    E, off, off_d, total, R, K, N = _case(i)
    note(f"forward E={E} rows={total}/{R} K={K} N={N}")
    x, w = _rows(R, K, total, i), _rand((E, N, K), 50 + i, K ** -0.5)
    want, mag = ref.linear(x[:total], w, off)
    out = _poisoned(R, N)
    grouped_gemm_forward(x.to(DEV), w.to(DEV), off_d, out)
    fresh = grouped_gemm_forward(x.to(DEV), w.to(DEV), off_d)
    sync_or_fail()
    ref.check(out[:total], want, ref.gamma(K) * mag, ref.B, "out")
    assert _is_poison(out[total:])
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_backward_input(i):
    E, off, off_d, total, R, K, N = _case(i)
    note(f"backward input E={E} rows={total}/{R} K={K} N={N}")
    dy, w = _rows(R, N, total, i), _rand((E, N, K), 50 + i, N ** -0.5)
    want, mag = ref.linear(dy[:total], w.transpose(1, 2).contiguous(), off)
    out = _poisoned(R, K)
    grouped_gemm_backward_input(dy.to(DEV), w.to(DEV), off_d, out)
    fresh = grouped_gemm_backward_input(dy.to(DEV), w.to(DEV), off_d)
    sync_or_fail()
    ref.check(out[:total], want, ref.gamma(N) * mag, ref.B, "grad x")
    assert _is_poison(out[total:])
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_gated_backward(i, name):
    E, off, off_d, total, R, N, F = _case(i)
    note(f"gated backward E={E} rows={total}/{R} N={N} F={F} {name}")
    dy, w = _rows(R, N, total, i), _rand((E, N, F), 50 + i, N ** -0.5)
    pre = torch.randn(R, 2 * F, generator=_gen(90 + i)) * 2.0
    pre[total:] = float("nan")
    want, err = ref.gated_grad(dy[:total], w, pre[:total], off, name)
    out = _poisoned(R, 2 * F)
    args = dy.to(DEV), w.to(DEV), pre.to(DEV), off_d
    gated_grouped_gemm_backward(*args, out, activation=name)
    fresh = gated_grouped_gemm_backward(*args, activation=name)
    sync_or_fail()
    ref.check(out[:total], want, err, ref.B, "grad pre")
    assert _is_poison(out[total:])
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_backward_weight(i, dtype):
    E, off, off_d, total, R, K, N = _case(i)
    note(f"backward weight E={E} rows={total}/{R} K={K} N={N} {dtype}")
    dy, x = _rows(R, N, total, i), _rows(R, K, total, 30 + i)
    want, err = ref.wgrad(dy[:total], x[:total], off)
    half = ref.B if dtype == BF else ref.U
    out = torch.full((E, N, K), float("nan"), dtype=dtype, device=DEV)
    grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d, out)
    start = _rand((E, N, K), 70 + i).to(dtype)
    acc = start.to(DEV)
    grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d, acc, accumulate=True)
    if dtype == BF:
        fresh = grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d)
        assert torch.equal(fresh, out)
    sync_or_fail()
    ref.check(out, want, err, half, "grad w")
    empty = [e for e in range(E) if off[e] == off[e + 1]]
    assert (out[empty] == 0).all()
    total_want = start.double() + want
    ref.check(acc, total_want, err + ref.U * total_want.abs() + ref.U * err, half, "accumulated")
    assert torch.equal(acc[empty].cpu(), start[empty])


MX = [
    ([1], 0, 32, 32),
    ([1, 0, 1, 1, 0, 0, 1, 2], 26, 256, 64),
    ([3, 0, 7, 17, 1], 12, 2048, 208),
    ([40, 33, 0, 2, 90], 3, 160, 48),
    ([120, 0, 260, 131], 9, 288, 336),
    ([300], 4, 640, 64),
    ([0, 0], 8, 64, 32),
    ([int(i % 5 == 0) * (i % 7) for i in range(300)], 5, 64, 48),
    # many rows and features: the tiled form, last tiles of every size
    ([16, 900, 33, 61, 500, 130], 11, 224, 1040),
    ([2500], 4, 160, 784),
]


def _mx(E, N, K, seed):
    g = _gen(seed)
    values = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(118, 130, (E, N, K // 32), generator=g, dtype=torch.uint8)
    return values, scales, mxfp4_expert_weights(values.to(DEV), scales.to(DEV))


@pytest.mark.parametrize("i", range(len(MX)))
def test_mxfp4_forward(i):
    counts, tail, K, N = MX[i]
    off, off_d = _off(counts)
    total, E = off[-1], len(counts)
    R = total + tail
    N += 8                                        # a partial 16-feature block
    note(f"mxfp4 E={E} rows={total}/{R} K={K} N={N}")
    values, scales, packed = _mx(E, N, K, i)
    x = _rows(R, K, total, 20 + i)
    want, mag = ref.linear(x[:total], ref.mxfp4_weights(values, scales), off)
    out = _poisoned(R, N)
    grouped_gemm(x.to(DEV), packed, off_d, out)
    fresh = grouped_gemm(x.to(DEV), packed, off_d)
    sync_or_fail()
    ref.check(out[:total], want, ref.gamma(K) * mag, ref.B, "out")
    assert _is_poison(out[total:])
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(MX)))
def test_mxfp4_gated(i, name):
    counts, tail, K, F = MX[i]
    off, off_d = _off(counts)
    total, E = off[-1], len(counts)
    R = total + tail
    note(f"mxfp4 gated E={E} rows={total}/{R} K={K} F={F} {name}")
    values, scales, packed = _mx(E, 2 * F, K, i)
    x = _rows(R, K, total, 20 + i, 0.2 * K ** -0.5)
    h, err, _, _ = ref.gated(x[:total], ref.mxfp4_weights(values, scales), off, name)
    out = _poisoned(R, F)
    gated_grouped_gemm(x.to(DEV), packed, off_d, out, activation=name)
    fresh = gated_grouped_gemm(x.to(DEV), packed, off_d, activation=name)
    sync_or_fail()
    ref.check(out[:total], h, err, ref.B, "h")
    assert _is_poison(out[total:])
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("rows", [2, 80, 300, 900])
def test_mxfp4_every_value_and_scale(rows):
    """x is a one in one place per row, so each output is one weight: every
    e2m1 value under every scale byte, exactly (bf16 holds them all)."""
    K = 32
    N = 16 * 256
    values = torch.zeros(1, N, K // 2, dtype=torch.uint8)
    values[0, :, 0] = (torch.arange(N) % 16).to(torch.uint8)
    scales = (torch.arange(N) // 16).to(torch.uint8).view(1, N, 1)
    x = torch.zeros(rows, K)
    x[:, 0] = 1.0
    note(f"mxfp4 values and scales rows={rows}")
    off, off_d = _off([rows])
    packed = mxfp4_expert_weights(values.to(DEV), scales.contiguous().to(DEV))
    got = grouped_gemm(x.to(BF).to(DEV), packed, off_d).float().cpu()
    sync_or_fail()
    want = ref.mxfp4_weights(values, scales)[0, :, 0].float()
    nan = scales.view(-1) == 255
    assert torch.isnan(got[:, nan]).all()
    over = want.isinf() & ~nan
    assert torch.equal(got[:, ~nan & ~over], want[~nan & ~over].expand(rows, -1))
    assert got[:, over].isinf().all()


def _ffn_bounds(x, w1, w2, dy, off, name):
    """64-bit results of the whole block and bounds that follow the roundings
    of h and of the gradients of [g | u] to bf16."""
    B, F = ref.B, w2.shape[2]
    K, N = w1.shape[2], w2.shape[1]
    h, eh, pre, epre = ref.gated(x, w1, off, name)
    eh = eh + B * (h.abs() + eh)
    w2a = w2.double().abs()
    y, ymag = ref.linear(h, w2, off)
    ey, _ = ref.linear(eh, w2a, off)
    ey = ey + ref.gamma(F) * (ymag + ey)
    dh, dhmag = ref.linear(dy, w2.transpose(1, 2).contiguous(), off)
    edh = ref.gamma(N) * dhmag
    g, u = pre[:, :F], pre[:, F:]
    eg, eu = epre[:, :F], epre[:, F:]
    a, s, _ = ref.act(name, g)
    ea, es = ref.act_error(name, g)
    ea, es = ea + ref.SLOPE * eg, es + ref.CURVE * eg
    dg, du = dh * u * s, dh * a
    edg = (edh * (u.abs() + eu) * (s.abs() + es) + dh.abs() * (eu * (s.abs() + es) + u.abs() * es))
    edu = edh * (a.abs() + ea) + dh.abs() * ea
    dpre, edpre = torch.cat((dg, du), 1), torch.cat((edg, edu), 1) * (1 + 4 * ref.U)
    edpre = edpre + B * (dpre.abs() + edpre)
    w1t = w1.double().transpose(1, 2).contiguous()
    dx, dxmag = ref.linear(dpre, w1t, off)
    edx, _ = ref.linear(edpre, w1t.abs(), off)
    edx = edx + ref.gamma(2 * F) * (dxmag + edx)
    dw1, e1 = ref.wgrad(dpre, x, off)
    p1, _ = ref.wgrad(edpre, x.double().abs(), off)
    dw2, e2 = ref.wgrad(dy, h, off)
    p2, _ = ref.wgrad(dy.double().abs(), eh, off)
    grow = 1 + ref.gamma(max(1, x.shape[0]))
    return (y, ey), (dx, edx), (dw1, e1 + p1 * grow), (dw2, e2 + p2 * grow)


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("i", [0, 1, 2, 4, 5, 6, 8])
def test_expert_ffn_gradients(i, name):
    E, off, off_d, total, R, D, F = _case(i)
    note(f"expert_ffn E={E} rows={total}/{R} D={D} F={F} {name}")
    x, dy = _rows(R, D, total, i), _rand((R, D), 10 + i)
    w1, w2 = _rand((E, 2 * F, D), 50 + i, D ** -0.5), _rand((E, D, F), 60 + i, F ** -0.5)
    leaves = [t.to(DEV).requires_grad_(True) for t in (x, w1, w2)]
    y = expert_ffn(*leaves, off_d, activation=name)
    y.backward(dy.to(DEV))
    with torch.no_grad():
        plain = expert_ffn(*leaves, off_d, activation=name)
    sync_or_fail()
    assert torch.equal(plain, y)
    got = (y.detach()[:total], leaves[0].grad[:total], leaves[1].grad, leaves[2].grad)
    want = _ffn_bounds(x[:total], w1, w2, dy[:total], off, name)
    for what, t, (v, err) in zip(("y", "dx", "dw1", "dw2"), got, want):
        ref.check(t, v, err, ref.B, what)
    assert (y[total:] == 0).all() and (leaves[0].grad[total:] == 0).all()


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_expert_ffn_gradients_against_differences(name):
    """<gradient, direction> against a central difference of the 64-bit block:
    off by the gradients' own bounds and the difference's h^2 and 1/h terms."""
    counts = [5, 0, 9, 20]
    off, off_d = _off(counts)
    total, E, D, F = off[-1], 4, 48, 40
    x, dy = _rand((total, D), 1), _rand((total, D), 2)
    w1, w2 = _rand((E, 2 * F, D), 3, D ** -0.5), _rand((E, D, F), 4, F ** -0.5)
    note(f"expert_ffn differences {name}")
    leaves = [t.to(DEV).requires_grad_(True) for t in (x, w1, w2)]
    expert_ffn(*leaves, off_d, activation=name).backward(dy.to(DEV))
    sync_or_fail()
    bounds = _ffn_bounds(x, w1, w2, dy, off, name)[1:]

    def loss(a, b, c):
        h, _, _, _ = ref.gated(a, b, off, name)
        return (ref.linear(h, c, off)[0] * dy.double()).sum()

    args = [t.double() for t in (x, w1, w2)]
    step = 1e-4
    for j in range(3):
        v = torch.randn(args[j].shape, generator=_gen(7 + j), dtype=torch.float64)
        hi, lo = list(args), list(args)
        hi[j], lo[j] = args[j] + step * v, args[j] - step * v
        diff = (loss(*hi) - loss(*lo)) / (2 * step)
        grad = leaves[j].grad.double().cpu()
        slack = ((bounds[j][1] + ref.B * grad.abs()) * v.abs()).sum()
        assert abs(float((grad * v).sum() - diff)) <= float(slack) * (1 + 1e-3)


def test_gradients_only_where_wanted():
    off, off_d = _off([4, 3])
    x, w1, w2 = (t.to(DEV) for t in (_rand((7, 32), 1), _rand((2, 32, 32), 2), _rand((2, 24, 16), 3)))
    full = [t.clone().requires_grad_(True) for t in (x, w1, w2)]
    dy = _rand((7, 24), 4).to(DEV)
    expert_ffn(*full, off_d).backward(dy)
    for j in range(3):
        leaves = [t.clone().requires_grad_(k == j) for k, t in enumerate((x, w1, w2))]
        expert_ffn(*leaves, off_d).backward(dy)
        for k in range(3):
            if k == j:
                assert torch.equal(leaves[k].grad, full[k].grad)
            else:
                assert leaves[k].grad is None


def test_broadcast_and_strided_upstream_gradient():
    off, off_d = _off([4, 3])
    x, w1, w2 = (t.to(DEV) for t in (_rand((7, 32), 1), _rand((2, 32, 32), 2), _rand((2, 24, 16), 3)))
    grads = []
    for dense in (True, False):
        a = x.clone().requires_grad_(True)
        y = expert_ffn(a, w1, w2, off_d)
        dy = torch.ones((), dtype=BF, device=DEV).expand(7, 24)
        y.backward(dy.contiguous() if dense else dy)
        grads.append(a.grad)
    assert torch.equal(*grads)


@pytest.mark.parametrize("shift", [0, 1, 8])
def test_upstream_gradient_that_begins_anywhere(shift):
    """The gradient of a concatenation's part is a view into the whole one."""
    off, off_d = _off([4, 3])
    x, w1, w2 = (t.to(DEV) for t in (_rand((7, 32), 1), _rand((2, 32, 32), 2), _rand((2, 24, 16), 3)))
    dy = _rand((7, 24), 4).to(DEV)
    grads = []
    for joined in (True, False):
        leaves = [t.clone().requires_grad_(True) for t in (x, w1, w2)]
        y = expert_ffn(*leaves, off_d)
        if joined:
            head = torch.zeros(shift, dtype=BF, device=DEV, requires_grad=True)
            torch.cat((head, y.flatten())).backward(torch.cat((torch.zeros_like(head), dy.flatten())))
        else:
            y.backward(dy)
        grads.append([t.grad for t in leaves])
    for a, b in zip(*grads):
        assert torch.equal(a, b)


def test_offsets_are_kept_for_the_backward():
    """The caller's offsets (a layout's persistent buffer) may be rewritten
    between forward and backward."""
    off, off_d = _off([4, 3])
    x, w1, w2 = (t.to(DEV) for t in (_rand((7, 32), 1), _rand((2, 32, 32), 2), _rand((2, 24, 16), 3)))
    dy = _rand((7, 24), 4).to(DEV)
    grads = []
    for spoil in (False, True):
        a = x.clone().requires_grad_(True)
        o = off_d.clone()
        y = expert_ffn(a, w1, w2, o)
        if spoil:
            o.zero_()
        y.backward(dy)
        grads.append(a.grad)
    assert torch.equal(*grads)


@pytest.mark.parametrize("rows", [(6, 5), (100, 90), (300, 301)])
def test_a_row_reaches_only_its_own_outputs(rows):
    """Infinities and NaN in one row leave every other row's output, and every
    other expert's weight gradient, as they were."""
    off, off_d = _off(rows)
    total, D, F = off[-1], 136, 72
    x, w = _rand((total, D), 1).to(DEV), _rand((2, 2 * F, D), 2, D ** -0.5).to(DEV)
    dy = _rand((total, F), 3).to(DEV)
    clean = gated_grouped_gemm(x, w, off_d), grouped_gemm_backward_weight(dy, x, off_d)
    spoilt = x.clone()
    spoilt[2] = float("nan")
    spoilt[3, 5] = float("inf")
    note(f"isolation rows={rows}")
    h, gw = gated_grouped_gemm(spoilt, w, off_d), grouped_gemm_backward_weight(dy, spoilt, off_d)
    sync_or_fail()
    keep = [r for r in range(total) if r not in (2, 3)]
    assert torch.equal(h[keep], clean[0][keep])
    assert torch.isnan(h[2]).all()
    assert torch.equal(gw[1], clean[1][1]) and torch.isnan(gw[0]).all()


def test_repeats_and_streams_give_equal_bits():
    off, off_d = _off([70, 0, 130, 9])
    total, D, F = off[-1], 264, 136
    x, w = _rand((total, D), 1).to(DEV), _rand((4, 2 * F, D), 2, D ** -0.5).to(DEV)
    dy = _rand((total, F), 3).to(DEV)
    first = gated_grouped_gemm(x, w, off_d), grouped_gemm_backward_weight(dy, x, off_d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = gated_grouped_gemm(x, w, off_d), grouped_gemm_backward_weight(dy, x, off_d)
    torch.cuda.current_stream().wait_stream(side)
    sync_or_fail()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls share no state: two streams run the whole block side by side."""
    cases = []
    for seed, counts in ((1, [300, 0, 41]), (2, [9, 5, 290])):
        off, off_d = _off(counts)
        ts = [_rand((off[-1], 264), seed), _rand((3, 272, 264), seed + 2, 264 ** -0.5),
              _rand((3, 264, 136), seed + 4, 136 ** -0.5), _rand((off[-1], 264), seed + 6)]
        cases.append((off_d, [t.to(DEV) for t in ts]))

    def step(off_d, ts):
        leaves = [t.clone().requires_grad_(True) for t in ts[:3]]
        y = expert_ffn(*leaves, off_d)
        y.backward(ts[3])
        return [y.detach(), *(t.grad for t in leaves)]

    want = [step(*c) for c in cases]
    sync_or_fail()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for j, c in enumerate(cases):
            with torch.cuda.stream(streams[j]):
                got[j].append(step(*c))
    sync_or_fail()
    for j in range(2):
        for run in got[j]:
            for a, b in zip(run, want[j]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [40, 700, 9000])
def test_as_many_experts_as_there_can_be(rows):
    """1024 experts: a wavefront's lane looks after 16 of them."""
    E, D, F = 1024, 64, 32
    g = _gen(rows)
    counts = torch.bincount(torch.randint(0, E, (rows,), generator=g), minlength=E)
    counts[7] = 0
    off, off_d = _off(counts.tolist())
    total, R = off[-1], off[-1] + 6
    note(f"1024 experts, {total} rows")
    x, w = _rows(R, D, total, 1), _rand((E, 2 * F, D), 2, D ** -0.5)
    h, err, pre, _ = ref.gated(x[:total], w, off, "silu")
    got = gated_grouped_gemm(x.to(DEV), w.to(DEV), off_d)
    sync_or_fail()
    ref.check(got[:total], h, err, ref.B, "h")
    assert (got[total:].view(torch.int16) == 0).all()
    dy = _rows(R, F, total, 3)
    want, err = ref.wgrad(dy, x, off)
    ref.check(grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d), want, err, ref.B, "dw")
    values, scales, packed = _mx(E, 2 * F, D, 4)
    h, err, _, _ = ref.gated(x[:total], ref.mxfp4_weights(values, scales), off, "silu")
    got = gated_grouped_gemm(x.to(DEV), packed, off_d)
    sync_or_fail()
    ref.check(got[:total], h, err, ref.B, "4-bit h")


def test_segments_are_clamped_to_the_rows():
    """Offsets that begin behind row 0, before it or end past the last row."""
    R, D, F = 150, 72, 40
    x, w = _rand((R, D), 1), _rand((2, 2 * F, D), 2, D ** -0.5)
    dy = _rand((R, F), 3)
    for raw in ([20, 90, 150], [-7, 90, 150], [0, 90, 1 << 30], [-(1 << 30), -5, 1 << 30]):
        off = [min(max(o, 0), R) for o in raw]
        off_d = torch.tensor(raw, dtype=torch.int32, device=DEV)
        note(f"offsets {raw}")
        out = _poisoned(R, F)
        gated_grouped_gemm(x.to(DEV), w.to(DEV), off_d, out)
        h, err, _, _ = ref.gated(x, w, off, "silu")
        sync_or_fail()
        assert _is_poison(out[:off[0]])
        ref.check(out[off[0]:], h[off[0]:], err[off[0]:], ref.B, "h")
        want, err = ref.wgrad(dy, x, off)
        ref.check(grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d), want, err, ref.B, "dw")


@pytest.mark.parametrize("counts", [[1300], [600, 0, 1100]])
def test_backward_weight_of_long_segments(counts):
    """Segments too long for their rows to be touched ahead of the tiles."""
    off, off_d = _off(counts)
    total, D, F = off[-1], 264, 136
    x, dy = _rows(total + 2, D, total, 1), _rows(total + 2, F, total, 2)
    want, err = ref.wgrad(dy, x, off)
    got = grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d)
    sync_or_fail()
    ref.check(got, want, err, ref.B, "dw")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("E, rows", [(64, 400), (8, 33)])
def test_backward_weight_with_rows_touched_ahead(E, rows, accumulate):
    """Enough tiles for the rows to be touched ahead of them: 210 MB of rows a
    few experts ahead, 1.4 MB all at once."""
    D, F = 2048, 2048
    counts = [rows + 8 * (e % 3) - 3 * (e % 5) for e in range(E)]
    counts[3] = 0
    off, off_d = _off(counts)
    total = off[-1]
    assert (total * (D + F) * 2 > 192 << 20) == (E == 64) and E * 128 >= 1024
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(total + 3, D, generator=g, device=DEV).to(BF)
    dy = torch.randn(total + 3, F, generator=g, device=DEV).to(BF)
    x[total:], dy[total:] = float("nan"), float("nan")
    note(f"{E} experts, {total} rows")
    before = torch.randn(E, F, D, generator=g, device=DEV) if accumulate else None
    got = grouped_gemm_backward_weight(dy, x, off_d,
                                       before.clone() if accumulate else None,
                                       accumulate=accumulate)
    sync_or_fail()
    for e in range(E):
        a, b = off[e], off[e + 1]
        d, xe = dy[a:b].double().t().contiguous(), x[a:b].double()
        want = d @ xe if b > a else torch.zeros(F, D, dtype=torch.float64, device=DEV)
        err = ref.gamma(b - a) * (d.abs() @ xe.abs()) if b > a else torch.zeros_like(want)
        if accumulate:
            want += before[e].double()
        ref.check(got[e], want.cpu(), err.cpu(), ref.U if accumulate else ref.B, f"dw[{e}]")


def test_buffers_past_32_bits():
    """Outputs and rows beyond 4 GiB: the last rows are right."""
    D, F, E = 64, 8192, 2
    R = 280000                                     # 4.6 GB of h
    counts = [R - 40, 33]
    off, off_d = _off(counts)
    total = off[-1]
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(R, D, device=DEV, generator=g).to(BF)
    w = (torch.randn(E, 2 * F, D, device=DEV, generator=g) * D ** -0.5).to(BF)
    note(f"large buffers R={R} F={F}")
    h = gated_grouped_gemm(x, w, off_d)
    dx = grouped_gemm_backward_input(h, w[:, :F].contiguous(), off_d)
    sync_or_fail()
    pick = torch.tensor([0, R // 2, counts[0] - 1, counts[0], total - 1])
    expert = [0, 0, 0, 1, 1]
    for p, e in zip(pick.tolist(), expert):
        xs = x[p:p + 1].cpu()
        want, err, _, _ = ref.gated(xs, w[e:e + 1].cpu(), [0, 1], "silu")
        ref.check(h[p:p + 1], want, err, ref.B, f"row {p}")
        hs = h[p:p + 1].cpu()
        want, mag = ref.linear(hs, w[e:e + 1, :F].transpose(1, 2).contiguous().cpu(), [0, 1])
        ref.check(dx[p:p + 1], want, ref.gamma(F) * mag, ref.B, f"grad row {p}")
    assert (h[total:] == 0).all() and (dx[total:] == 0).all()


def _layer(T, D, F, E, K, seed):
    g = _gen(seed)
    x = torch.randn(T, D, generator=g).to(BF).to(DEV)
    ids = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :K].to(torch.int32)
    ids[torch.rand(T, K, generator=g) < 0.1] = -1
    s = torch.softmax(torch.randn(T, K, generator=g), 1)
    return x, ids.contiguous().to(DEV), s.to(DEV)


def test_layer_training_step():
    """dispatch -> expert_ffn -> combine and back, against the same step with
    every token's experts written out in 64 bits."""
    T, D, F, E, K = 53, 64, 48, 6, 2
    x, ids, s = _layer(T, D, F, E, K, 3)
    w1 = _rand((E, 2 * F, D), 5, D ** -0.5).to(DEV).requires_grad_(True)
    w2 = _rand((E, D, F), 6, F ** -0.5).to(DEV).requires_grad_(True)
    x.requires_grad_(True)
    s.requires_grad_(True)
    dy = _rand((T, D), 7).to(DEV)
    layer = MoeTokenDispatcher(MoeDispatcher(T, D, E, K, backward=True))
    note("layer training step")
    x_e = layer.dispatch(x, s, ids)
    y = layer.combine(expert_ffn(x_e, w1, w2, layer.disp.offsets), s)
    y.backward(dy)
    sync_or_fail()
    ref_in = [t.detach().double().cpu().requires_grad_(True) for t in (x, s, w1, w2)]
    xr, sr, w1r, w2r = ref_in
    rows = []
    for t in range(T):
        acc = torch.zeros(D, dtype=torch.float64)
        for k in range(K):
            e = int(ids[t, k])
            if e >= 0:
                pre = w1r[e] @ xr[t]
                acc = acc + sr[t, k] * (w2r[e] @ (torch.nn.functional.silu(pre[:F]) * pre[F:]))
        rows.append(acc)
    yr = torch.stack(rows)
    yr.backward(dy.double().cpu())
    # Eight bf16 roundings lie on the longest path (pre, h, y_e, g_y_e, dpre,
    # dx_e and the sums' results): each is off by at most B of its value, the
    # values' sums by sqrt of their number; norm-wise 8 B bounds the whole.
    for what, got, want in (("y", y, yr), ("dx", x.grad, xr.grad), ("ds", s.grad, sr.grad),
                            ("dw1", w1.grad, w1r.grad), ("dw2", w2.grad, w2r.grad)):
        diff = (got.detach().double().cpu() - want.detach()).norm()
        assert float(diff) <= 8 * ref.B * float(want.detach().norm()), what


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 37, 600])
def test_layer_in_a_captured_graph(kind, T):
    """layout -> dispatch -> gated product -> down projection -> combine as one
    graph, replayed with other routing and compared with the eager calls."""
    D, F, E, K = 128, 64, 8, 2
    disp = MoeDispatcher(T, D, E, K)
    x, ids, s = _layer(T, D, F, E, K, 1)
    if kind == "bf16":
        w1, w2 = _rand((E, 2 * F, D), 5, D ** -0.5).to(DEV), _rand((E, D, F), 6, F ** -0.5).to(DEV)
    else:
        w1, w2 = _mx(E, 2 * F, D, 5)[2], _mx(E, D, F, 6)[2]

    def step():
        lay = disp.layout(ids)
        dsp = disp.dispatch(x, s, ids, lay.counts)
        h = gated_grouped_gemm(dsp.x_e, w1, lay.offsets)
        y_e = (grouped_gemm_forward if kind == "bf16" else grouped_gemm)(h, w2, lay.offsets)
        return disp.combine(y_e, lay.row_map, s)

    note(f"graph {kind} T={T}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(2, 6):
        nx, nids, ns = _layer(T, D, F, E, K, seed)
        x.copy_(nx), ids.copy_(nids), s.copy_(ns)
        graph.replay()
        got = out.clone()
        sync_or_fail()
        want = step().clone()
        sync_or_fail()
        assert torch.equal(got, want)


def test_gradient_kernels_in_a_captured_graph():
    E, off, off_d, total, R, D, F = _case(5)
    w1, w2 = _rand((E, 2 * F, D), 1, D ** -0.5).to(DEV), _rand((E, D, F), 2, F ** -0.5).to(DEV)
    x, dy = _rand((R, D), 3).to(DEV), _rand((R, D), 4).to(DEV)
    dw = torch.empty(E, 2 * F, D, device=DEV)

    def step():
        pre = torch.empty(R, 2 * F, device=DEV)
        h = gated_grouped_gemm(x, w1, off_d, pre=pre)
        dpre = gated_grouped_gemm_backward(dy, w2, pre, off_d)
        grouped_gemm_backward_weight(dpre, x, off_d, dw)
        return (grouped_gemm_backward_input(dpre, w1, off_d),
                grouped_gemm_backward_weight(dy, h, off_d))

    note("gradient graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        x.copy_(_rand((R, D), 20 + seed)), dy.copy_(_rand((R, D), 30 + seed))
        graph.replay()
        got = [t.clone() for t in (*out, dw)]
        sync_or_fail()
        want = [t.clone() for t in (*step(), dw)]
        sync_or_fail()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals_on_the_device():
    off, off_d = _off([2, 3])
    x, w1 = _rand((5, 32), 1).to(DEV), _rand((2, 64, 32), 2).to(DEV)
    w2 = _rand((2, 32, 32), 3).to(DEV)
    _, _, packed = _mx(2, 64, 32, 4)
    _, _, odd = _mx(2, 24, 32, 4)
    pre, h2 = torch.empty(5, 64, device=DEV), torch.empty(5, 64, dtype=BF, device=DEV)
    value_errors = [
        lambda: gated_grouped_gemm(x[:, :16], w1, off_d),               # strided
        lambda: gated_grouped_gemm(x[:, :16].contiguous(), w1, off_d),  # width
        lambda: gated_grouped_gemm(x, w1[:, :33].contiguous(), off_d),  # odd gate and up
        lambda: gated_grouped_gemm(x, w1, off_d[:2]),                   # offsets
        lambda: gated_grouped_gemm(x, w1, off_d, pre=pre[:4]),
        lambda: gated_grouped_gemm(x, w1, off_d, h2),                   # out width
        lambda: gated_grouped_gemm(x, packed, off_d, pre=pre),
        lambda: gated_grouped_gemm(x, odd, off_d),
        lambda: gated_grouped_gemm(x, packed._replace(k_in=64), off_d),
        lambda: grouped_gemm(x, packed._replace(data=packed.data[:-16]), off_d),
        lambda: grouped_gemm(x, packed, off_d, row_tile=64),
        lambda: grouped_gemm_forward(x, w1.transpose(1, 2), off_d),
        lambda: grouped_gemm_backward_input(x, w1, off_d),              # width 32, not 64
        lambda: gated_grouped_gemm_backward(x, w2, pre[:, :32].contiguous(), off_d),
        lambda: grouped_gemm_backward_weight(x, h2[:4], off_d),
        lambda: grouped_gemm_backward_weight(x, x, off_d, accumulate=True),
        lambda: grouped_gemm_backward_weight(x, x, off_d, w1),
        lambda: expert_ffn(x, w1, w2[:, :, :16].contiguous(), off_d),
        lambda: mxfp4_expert_weights(torch.zeros(1, 8, 8, dtype=torch.uint8, device=DEV),
                                     torch.zeros(1, 8, 1, dtype=torch.uint8, device=DEV)),
    ]
    for i, call in enumerate(value_errors):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    type_errors = [
        lambda: gated_grouped_gemm(x.float(), w1, off_d),
        lambda: gated_grouped_gemm(x, w1, off_d, pre=h2),
        lambda: gated_grouped_gemm_backward(x, w2, h2, off_d),
        lambda: gated_grouped_gemm(x, w1.float(), off_d),
        lambda: gated_grouped_gemm(x, w1, off_d.long()),
        lambda: grouped_gemm(x.half(), packed, off_d),
        lambda: grouped_gemm_backward_weight(x, x, off_d, torch.zeros(2, 32, 32, device=DEV).half()),
        lambda: mxfp4_expert_weights(w1, w1),
    ]
    for i, call in enumerate(type_errors):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"call {i} was not refused")
    from combine_moe_layout_05_amd import MoeError
    flat = torch.zeros(5 * 32 + 8, dtype=BF, device=DEV)
    with pytest.raises(MoeError):                                       # misaligned rows
        gated_grouped_gemm(flat[1:161].view(5, 32), w1, off_d)
    # widths the kernels do not take
    with pytest.raises(MoeError):
        grouped_gemm_forward(_rand((5, 12), 1).to(DEV), _rand((2, 8, 12), 1).to(DEV), off_d)


def test_no_rows_and_one_expert():
    """max_rows = 0 gives empty outputs and zero weight gradients; one expert
    is an ordinary dense block."""
    off_d = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 32, dtype=BF, device=DEV)
    w1, w2 = _rand((2, 64, 32), 2).to(DEV), _rand((2, 24, 32), 3).to(DEV)
    leaves = [t.requires_grad_(True) for t in (x, w1, w2)]
    y = expert_ffn(*leaves, off_d)
    assert tuple(y.shape) == (0, 24)
    y.sum().backward()
    assert tuple(x.grad.shape) == (0, 32)
    assert (w1.grad == 0).all() and (w2.grad == 0).all()
    assert tuple(grouped_gemm(x.detach(), _mx(2, 64, 32, 1)[2], off_d).shape) == (0, 64)


def _captured_step(leaves, off_d, dy):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = expert_ffn(*leaves, off_d)
        y.backward(dy)
    return graph, y


def test_training_step_in_a_captured_graph():
    """Forward and backward in one graph, replayed on new inputs and compared
    with the eager gradients; refused while an eager graph of the same leaves
    from the default stream is alive."""
    off, off_d = _off([40, 0, 90, 7])
    total, D, F = off[-1], 136, 72
    x = _rand((total, D), 1).to(DEV).requires_grad_(True)
    w1 = _rand((4, 2 * F, D), 2, D ** -0.5).to(DEV).requires_grad_(True)
    w2 = _rand((4, D, F), 3, F ** -0.5).to(DEV).requires_grad_(True)
    dy = _rand((total, D), 4).to(DEV)
    leaves = (x, w1, w2)

    def eager():
        copies = [t.detach().clone().requires_grad_(True) for t in leaves]
        y = expert_ffn(*copies, off_d)
        y.backward(dy)
        return [y.detach(), *(t.grad for t in copies)]

    kept = expert_ffn(*leaves, off_d)
    note("capture beside an eager graph: refused")
    with pytest.raises(RuntimeError, match="default stream"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            expert_ffn(*leaves, off_d)
    del kept, graph
    sync_or_fail()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        expert_ffn(*leaves, off_d).backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    for t in leaves:
        t.grad = None
    note("training step graph")
    graph, y = _captured_step(leaves, off_d, dy)
    for seed in range(10, 13):
        with torch.no_grad():
            x.copy_(_rand((total, D), seed)), dy.copy_(_rand((total, D), seed + 50))
        for t in leaves:
            t.grad.zero_()
        graph.replay()
        got = [t.detach().clone() for t in (y, x.grad, w1.grad, w2.grad)]
        sync_or_fail()
        for a, b in zip(got, eager()):
            assert torch.equal(a, b)
        sync_or_fail()


def test_layer_training_step_in_a_captured_graph():
    """dispatch -> expert_ffn -> combine and back in one graph, replayed with
    new rows and new routing, a padded extent included."""
    T, ntpr, D, F, E, K = 53, 58, 64, 48, 6, 2
    x, ids, s = _layer(T, D, F, E, K, 3)
    w1 = _rand((E, 2 * F, D), 5, D ** -0.5).to(DEV).requires_grad_(True)
    w2 = _rand((E, D, F), 6, F ** -0.5).to(DEV).requires_grad_(True)
    dy = _rand((T, D), 7).to(DEV)
    x, s = x.requires_grad_(True), s.requires_grad_(True)
    leaves = (x, s, w1, w2)
    layers = [MoeTokenDispatcher(MoeDispatcher(64, D, E, K, backward=True)) for _ in range(2)]

    def step(layer, x, s, w1, w2):
        x_e = layer.dispatch(x, s, ids, ntpr)
        y = layer.combine(expert_ffn(x_e, w1, w2, layer.disp.offsets), s)
        y.backward(dy)
        return y.detach()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layers[0], *leaves)
    torch.cuda.current_stream().wait_stream(side)
    for t in leaves:
        t.grad = None
    sync_or_fail()
    note("whole layer training step graph")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(layers[0], *leaves)
    for seed in range(20, 24):
        x2, ids2, s2 = _layer(T, D, F, E, K, seed)
        with torch.no_grad():
            x.copy_(x2), ids.copy_(ids2), s.copy_(s2)
        for t in leaves:
            t.grad.zero_()
        graph.replay()
        got = [t.clone() for t in (y, *(t.grad for t in leaves))]
        sync_or_fail()
        copies = [t.detach().clone().requires_grad_(True) for t in leaves]
        want = [step(layers[1], *copies), *(t.grad for t in copies)]
        sync_or_fail()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
