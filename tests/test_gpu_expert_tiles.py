"""GPU tests of the expert products in the forms that many rows take: the large
tiles of the bf16 products, long segments of the weight gradient, and the tiled
4-bit products over many steps. The lists say which form a case runs in;
test_expert_forms.py holds them to it on the CPU."""
import pytest
import torch

import expert_ref as ref
from combine_moe_layout_05_amd import (
    gated_grouped_gemm, gated_grouped_gemm_backward, grouped_gemm, grouped_gemm_backward_input,
    grouped_gemm_backward_weight, grouped_gemm_forward, mxfp4_expert_weights)

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
POISON = 0x7F7F

# Rows of the experts, rows behind them, length of the sums, output features of
# the gated product and of the others.
LARGE = [
    # Last row tiles of one to four 64-row parts; five steps and a part of one;
    # the experts' sums begin at different steps; ragged last feature tiles.
    ([600, 37, 0, 700, 130, 900, 220], 19, 328, 1928, 3800),
    # More than one band of 8 row tiles, last feature tiles of 8 features.
    ([2300, 220, 64, 65], 0, 456, 1544, 3080),
    # Whole steps and whole feature tiles.
    ([300, 520, 0, 256, 512, 700], 5, 512, 1920, 3840),
    # Fewer steps than stages: a part of one, one, one and a part.
    ([257, 1900, 3], 40, 40, 2040, 4088),
    ([1024, 1024, 70], 0, 64, 2048, 4096),
    ([190, 2000, 129], 1, 72, 1992, 3912),
]

# Rows, rows behind, inputs (steps of 128), features (twice as many rows of
# weights if gated). Last row tiles of one to four 16-row blocks.
TILED = [
    (288, 912, 1800),      # 3 steps, the last one partial, in its first half
    (384, 912, 1800),      # 3
    (512, 1008, 1928),     # 4
    (608, 912, 1800),      # 5, partial in the second half
    (640, 1008, 1928),     # 5
    (1120, 912, 1800),     # 9, partial
    (1184, 1008, 1928),    # 10, partial
    (2048, 912, 1800),     # 16
]
TILED_ROWS = [70, 500, 33, 0, 61, 340, 16]
TILED_BEHIND = 5

# Rows, rows behind, k_in, n_out: segments of 2048 rows and more take bands of
# 8 feature tiles, the last one of 2 here and its last tile 8 features wide.
DEEP = [([2100, 0, 3000, 31], 7, 328, 1160), ([2048, 2047], 0, 256, 1024)]


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF)


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


def _case(i):
    counts, behind, red, gated, plain = LARGE[i]
    off, off_d = _off(counts)
    return len(counts), off, off_d, off[-1], off[-1] + behind, red, gated, plain


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_gated_forward(i, name):
    E, off, off_d, total, R, D, F, _ = _case(i)
    note(f"gated E={E} rows={total}/{R} D={D} F={F} {name}")
    x, w = _rows(R, D, total, i), _rand((E, 2 * F, D), 50 + i, 1.5 * D ** -0.5)
    h, err, pre, dpre = ref.gated(x[:total], w, off, name)
    out, pre_d = _poisoned(R, F), torch.full((R, 2 * F), 7.0, device=DEV)
    gated_grouped_gemm(x.to(DEV), w.to(DEV), off_d, out, activation=name, pre=pre_d)
    sync_or_fail()
    ref.check(out[:total], h, err, ref.B, "h")
    ref.check(pre_d[:total], pre, dpre, 0.0, "pre")
    assert _is_poison(out[total:]) and (pre_d[total:] == 7.0).all()


@pytest.mark.parametrize("i", range(len(LARGE)))
def test_plain_forward(i):
    E, off, off_d, total, R, K, _, N = _case(i)
    note(f"forward E={E} rows={total}/{R} K={K} N={N}")
    x, w = _rows(R, K, total, i), _rand((E, N, K), 50 + i, K ** -0.5)
    want, mag = ref.linear(x[:total], w, off)
    out = _poisoned(R, N)
    grouped_gemm_forward(x.to(DEV), w.to(DEV), off_d, out)
    sync_or_fail()
    ref.check(out[:total], want, ref.gamma(K) * mag, ref.B, "out")
    assert _is_poison(out[total:])


@pytest.mark.parametrize("i", range(len(LARGE)))
def test_backward_input(i):
    E, off, off_d, total, R, N, _, K = _case(i)
    note(f"backward input E={E} rows={total}/{R} K={K} N={N}")
    dy, w = _rows(R, N, total, i), _rand((E, N, K), 50 + i, N ** -0.5)
    want, mag = ref.linear(dy[:total], w.transpose(1, 2).contiguous(), off)
    out = _poisoned(R, K)
    grouped_gemm_backward_input(dy.to(DEV), w.to(DEV), off_d, out)
    sync_or_fail()
    ref.check(out[:total], want, ref.gamma(N) * mag, ref.B, "grad x")
    assert _is_poison(out[total:])


def _vanished(dh, u, g, name):
    """What sigmoids below fp32's smallest normal number cost a gradient of the
    gate; the relative bounds of expert_ref hold above it only.

    The sigmoid p(z) is formed as 1 / (1 + exp(-z)) with the hardware's
    reciprocal, which returns 0 in place of a result below 2^-126. So where p <
    2^-126 (and just above it, where the sum may round past 2^126, a factor of 1
    + 2^-22 at most) the computed p is 0 and off by p itself, at most 2^-126 (1 +
    2^-22); elsewhere nothing is added. Since act(g) = g p and act'(g) = p + g p
    (1 - p) dz, act is then off by at most |g| times that and act' by (1 + |g|
    dz) times it, and the results by |dh| and |dh u| times these. 2^-125 in
    place of 2^-126 is room for the error of dh, far below dh itself."""
    z, dz = g, torch.ones_like(g)
    if name == "gelu":
        z = ref.act(name, g)[2]
        dz = 2 * ref.ALPHA * (1 + 3 * ref.BETA * g ** 2)
    lost = torch.where(torch.sigmoid(z) < 2.0 ** -125, 2.0 ** -125, 0.0).double()
    return torch.cat(((dh * u).abs() * lost * (1 + g.abs() * dz), dh.abs() * lost * g.abs()), 1)


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_gated_backward(i, name):
    E, off, off_d, total, R, N, _, F = _case(i)
    note(f"gated backward E={E} rows={total}/{R} N={N} F={F} {name}")
    dy, w = _rows(R, N, total, i), _rand((E, N, F), 50 + i, N ** -0.5)
    pre = torch.randn(R, 2 * F, generator=torch.Generator().manual_seed(90 + i)) * 2.0
    pre[total:] = float("nan")
    want, err = ref.gated_grad(dy[:total], w, pre[:total], off, name)
    dh, _ = ref.linear(dy[:total], w.transpose(1, 2).contiguous(), off)
    err += _vanished(dh, pre[:total, F:].double(), pre[:total, :F].double(), name)
    out = _poisoned(R, 2 * F)
    gated_grouped_gemm_backward(dy.to(DEV), w.to(DEV), pre.to(DEV), off_d, out, activation=name)
    sync_or_fail()
    ref.check(out[:total], want, err, ref.B, "grad pre")
    assert _is_poison(out[total:])


@pytest.mark.parametrize("kind", ["bf16", "fp32", "added"])
@pytest.mark.parametrize("i", range(len(DEEP)))
def test_backward_weight_of_long_segments(i, kind):
    counts, behind, K, N = DEEP[i]
    off, off_d = _off(counts)
    E, total, R = len(counts), off[-1], off[-1] + behind
    note(f"backward weight E={E} rows={total}/{R} K={K} N={N} {kind}")
    dy, x = _rows(R, N, total, i), _rows(R, K, total, 30 + i)
    want, err = ref.wgrad(dy[:total], x[:total], off)
    dtype = BF if kind == "bf16" else torch.float32
    half = ref.B if kind == "bf16" else ref.U
    out = torch.full((E, N, K), float("nan"), dtype=dtype)
    if kind == "added":
        out = torch.randn(E, N, K, generator=torch.Generator().manual_seed(70 + i))
        want = out.double() + want
        err = err + ref.U * want.abs() + ref.U * err
    out = out.to(DEV)
    grouped_gemm_backward_weight(dy.to(DEV), x.to(DEV), off_d, out, accumulate=kind == "added")
    sync_or_fail()
    ref.check(out, want, err, half, "grad w")


def _mx(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    values = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(118, 130, (E, N, K // 32), generator=g, dtype=torch.uint8)
    return (ref.mxfp4_weights(values, scales),
            mxfp4_expert_weights(values.to(DEV), scales.to(DEV)))


@pytest.mark.parametrize("K, F, N", TILED)
def test_mxfp4_forward(K, F, N):
    off, off_d = _off(TILED_ROWS)
    total, R, E = off[-1], off[-1] + TILED_BEHIND, len(TILED_ROWS)
    note(f"mxfp4 E={E} rows={total}/{R} K={K} N={N}")
    w, packed = _mx(E, N, K, K)
    x = _rows(R, K, total, 20)
    want, mag = ref.linear(x[:total], w, off)
    out = _poisoned(R, N)
    grouped_gemm(x.to(DEV), packed, off_d, out)
    sync_or_fail()
    ref.check(out[:total], want, ref.gamma(K) * mag, ref.B, "out")
    assert _is_poison(out[total:])


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("K, F, N", TILED)
def test_mxfp4_gated(K, F, N, name):
    off, off_d = _off(TILED_ROWS)
    total, R, E = off[-1], off[-1] + TILED_BEHIND, len(TILED_ROWS)
    note(f"mxfp4 gated E={E} rows={total}/{R} K={K} F={F} {name}")
    w, packed = _mx(E, 2 * F, K, K)
    x = _rows(R, K, total, 20, 0.2 * K ** -0.5)
    h, err, _, _ = ref.gated(x[:total], w, off, name)
    out = _poisoned(R, F)
    gated_grouped_gemm(x.to(DEV), packed, off_d, out, activation=name)
    sync_or_fail()
    ref.check(out[:total], h, err, ref.B, "h")
    assert _is_poison(out[total:])
