"""GPU tests of rows in 4 bits: quantisation and back, bit for bit, and the
products of 4-bit rows with 4-bit weights against plain 64-bit forms
(layer_ref.py holds the definitions and the derivation of the bounds)."""
import pytest
import torch

import expert_ref
import layer_ref as ref
from combine_moe_layout_05_amd import (
    Mxfp4Rows, dequantize_mxfp4, gated_grouped_gemm, grouped_gemm, mxfp4_expert_weights,
    quantize_mxfp4)

from gpu_util import DEV, note, sync_or_fail

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
POISON = 0x7F7F            # bf16 bits no kernel writes here


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _check_quantized(x):
    """Codes, scales and the way back, bit for bit."""
    values, scales = ref.quantize(x)
    q = quantize_mxfp4(x.to(DEV))
    back = dequantize_mxfp4(q, x.dtype)
    sync_or_fail()
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.values.cpu(), values)
    want = ref.decode(values, scales)
    got = back.cpu().double()
    assert back.dtype == x.dtype and got.shape == x.shape
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (613, 1984), (7, 2880), (2, 5, 96), (1, 7168),
                                   (65, 32)])
def test_quantize(shape, dtype):
    note(f"quantize {shape} {dtype}")
    x = torch.randn(shape, generator=_gen(shape[-1])) * 3
    x *= torch.exp2(torch.randint(-20, 20, shape, generator=_gen(5)).float())
    _check_quantized(x.to(dtype))


def test_every_bf16_number_beside_every_largest_exponent():
    """Each bf16 pattern's magnitude below a block's largest element, for
    every exponent of that element, subnormal ones among them."""
    tops = torch.arange(0, 0x7F80, 0x40, dtype=torch.int32)         # two per exponent
    rows = []
    for top in tops.tolist():
        near = torch.arange(max(top - 0x400, 0), top + 1, dtype=torch.int32)[-31 * 32:]
        near = torch.cat([near, torch.zeros(-len(near) % 31, dtype=torch.int32)]).view(-1, 31)
        rows.append(torch.cat([torch.full((len(near), 1), top, dtype=torch.int32), near], dim=1))
    bits = torch.cat(rows)
    sign = torch.randint(0, 2, bits.shape, generator=_gen(1)).int() << 15
    bits = bits | sign
    x = (bits - ((bits & 0x8000) << 1)).to(torch.int16).view(BF)
    note(f"{x.shape[0]} blocks")
    _check_quantized(x)
    _check_quantized(x.float())


def test_fp32_between_the_numbers():
    """One unit around each middle between two e2m1 numbers."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    x = torch.cat([mid, mid * (1 + 2.0 ** -23), mid * (1 - 2.0 ** -24), torch.zeros(5)])
    x[-1] = 4.0
    x = torch.stack([x * 2.0 ** k for k in range(-120, 120, 7)])
    _check_quantized(x)
    _check_quantized(-x)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_nan_infinity_and_zero_blocks(dtype):
    x = torch.randn(6, 64, generator=_gen(2)).to(dtype)
    x[0, 3], x[1, 40], x[2, 63] = float("nan"), float("inf"), -float("inf")
    x[3] = 0.0
    x[4, :32] = -0.0
    x[5] = torch.finfo(dtype).max
    _check_quantized(x)
    q = quantize_mxfp4(x.to(DEV))
    back = dequantize_mxfp4(q, dtype).cpu()
    assert torch.isnan(back[0, :32]).all() and torch.isfinite(back[0, 32:]).all()
    assert (back[3] == 0).all() and int(q.scales[3, 0]) == 0


def test_all_codes_and_scales_back():
    values = torch.randint(0, 256, (256, 16), generator=_gen(3), dtype=torch.uint8)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1)
    want = ref.decode(values, scales)
    for dtype in (torch.float32, BF):
        got = dequantize_mxfp4(Mxfp4Rows(values.to(DEV), scales.to(DEV)), dtype).cpu().double()
        # 2^127 and 2^126 times 4 or 6 are past the types' largest number.
        big = want.abs() >= 2.0 ** 128
        nan = torch.isnan(want)
        assert torch.equal(got[~big & ~nan], want[~big & ~nan])
        assert torch.isinf(got[big]).all() and torch.isnan(got[nan]).all()


def test_empty_and_many_rows():
    assert quantize_mxfp4(torch.empty(0, 64, device=DEV)).values.shape == (0, 32)
    x = torch.randn(3, 32, generator=_gen(4))
    a, b = quantize_mxfp4(x.to(DEV)), quantize_mxfp4(x.to(DEV)[1:])
    assert torch.equal(a.values[1:], b.values) and torch.equal(a.scales[1:], b.scales)


# ---- Products ----------------------------------------------------------------

# counts, rows behind the last segment, k_in, n_hidden (gated) and n_out (plain)
SHAPES = [
    ([1], 0, 32, 16, 8),                            # one row, one group
    ([1, 0, 1, 1, 0, 0, 1, 2], 26, 256, 64, 200),   # a few rows on many experts
    ([3, 0, 7, 17, 1], 12, 1984, 1008, 1000),       # ragged sums and features
    ([0, 0, 0], 40, 64, 32, 24),                    # no rows at all
    ([int(i % 5 == 0) * (i % 7) for i in range(300)], 5, 96, 48, 40),   # experts > lanes
    # tiles of many rows: whole and partial last ones, odd and even numbers of
    # 128-element halves, one to many steps
    ([700, 3, 500, 0, 333], 21, 32, 672, 1288),
    ([513, 700, 5, 130], 22, 160, 656, 1256),
    ([470, 90, 711, 64], 3, 256, 688, 1304),
    ([16, 700, 31, 47, 350], 0, 288, 832, 1608),
    ([1100, 17], 9, 1312, 800, 1608),
    ([530, 49, 600], 0, 1408, 704, 1336),
    ([64, 1000, 65], 1, 2880, 720, 1400),
    # sums longer than the row scales that LDS holds at a time (7680)
    ([600, 90, 700], 5, 8032, 656, 1256),
    ([300, 1100], 0, 15424, 656, 1256),
    # 128-row tiles; last ones of one to eight 16-row blocks
    ([138, 148, 296, 60, 474, 376, 256], 7, 96, 2064, 4104),
    ([1200, 700, 77], 0, 1312, 2560, 5128),
    ([1500, 1000], 3, 7712, 2048, 4096),
]
TILES_128 = 3              # of these


def _operands(i):
    counts, behind, K, F, N = SHAPES[i]
    off = expert_ref.offsets_of(counts)
    E, R, total = len(counts), off[-1] + behind, off[-1]
    x = ref.quantize(torch.randn(R, K, generator=_gen(i)))
    x[1][total:] = 255                  # what lies behind the segments is not read
    gen = _gen(50 + i)

    def weights(n):
        return (torch.randint(0, 256, (E, n, K // 2), generator=gen, dtype=torch.uint8),
                torch.randint(118, 128, (E, n, K // 32), generator=gen, dtype=torch.uint8))

    return (E, off, total, R, K, F, N, x, weights(2 * F), weights(N),
            torch.tensor(off, dtype=torch.int32, device=DEV))


def _on_gpu(q):
    return Mxfp4Rows(q[0].to(DEV), q[1].to(DEV))


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_products(i):
    E, off, total, R, K, F, N, x, w13, w2, off_d = _operands(i)
    note(f"4-bit rows E={E} rows={total}/{R} K={K} F={F} N={N}")
    rows = _on_gpu(x)
    xd = ref.decode(*x)[:total]
    p13, p2 = mxfp4_expert_weights(*_on_gpu(w13)), mxfp4_expert_weights(*_on_gpu(w2))
    pre, dpre = ref.product(xd, ref.decode(*w13), off)
    for name in ("silu", "gelu"):
        out = torch.full((R, F), POISON, dtype=torch.int16, device=DEV).view(BF)
        assert gated_grouped_gemm(rows, p13, off_d, out, activation=name) is out
        fresh = gated_grouped_gemm(rows, p13, off_d, activation=name)
        sync_or_fail()
        expert_ref.check(out[:total], *ref.gate(pre, dpre, name), ref.B, "h " + name)
        assert (out[total:].view(torch.int16) == POISON).all()
        assert torch.equal(fresh[:total], out[:total])
        assert (fresh[total:].view(torch.int16) == 0).all()
    want, err = ref.product(xd, ref.decode(*w2), off)
    out = torch.full((R, N), POISON, dtype=torch.int16, device=DEV).view(BF)
    assert grouped_gemm(rows, p2, off_d, out) is out
    fresh = grouped_gemm(rows, p2, off_d)
    sync_or_fail()
    expert_ref.check(out[:total], want, err, ref.B, "out")
    assert (out[total:].view(torch.int16) == POISON).all()
    assert torch.equal(fresh[:total], out[:total])
    assert (fresh[total:].view(torch.int16) == 0).all()


@pytest.mark.parametrize("rows", [5, 700])
def test_each_place_alone(rows):
    """One value of a row and one of a weight row other than zero: lane, byte
    and scale of each of a sum's places, exactly."""
    K, N = 544, 40
    gen = _gen(rows)
    values, scales = torch.zeros(rows, K), torch.zeros(rows, K // 32)
    at = torch.randint(0, K, (rows,), generator=gen)
    at[:min(rows, K)] = torch.randperm(K, generator=gen)[:rows]
    x = torch.zeros(rows, K)
    x[torch.arange(rows), at] = 1.5
    xv, _ = ref.quantize(x * 4)
    xs = torch.randint(120, 135, (rows, K // 32), generator=gen, dtype=torch.uint8)
    w = torch.randint(-3, 4, (1, N, K), generator=gen).float() * 2
    w[..., ::32] = 6.0                  # every block with the same scale
    wv, _ = ref.quantize(w)
    ws = torch.randint(120, 135, (1, N, K // 32), generator=gen, dtype=torch.uint8)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    got = grouped_gemm(_on_gpu((xv, xs)), mxfp4_expert_weights(wv.to(DEV), ws.to(DEV)), off)
    want = ref.decode(xv, xs) @ ref.decode(wv, ws)[0].t()
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("rows", [3, 600])
def test_scales_at_the_ends_and_nan(rows):
    K, N = 160, 16
    gen = _gen(9)
    xv = torch.randint(0, 256, (rows, K // 2), generator=gen, dtype=torch.uint8)
    wv = torch.randint(0, 256, (1, N, K // 2), generator=gen, dtype=torch.uint8)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    for a, b in ((0, 254), (254, 0), (0, 127), (1, 160), (100, 100)):
        xs = torch.full((rows, K // 32), a, dtype=torch.uint8)
        ws = torch.full((1, N, K // 32), b, dtype=torch.uint8)
        got = grouped_gemm(_on_gpu((xv, xs)), mxfp4_expert_weights(wv.to(DEV), ws.to(DEV)), off)
        want, err = ref.product(ref.decode(xv, xs), ref.decode(wv, ws), [0, rows])
        # A product below fp32's normal numbers may come out as zero.
        err = err + K * 2.0 ** -126
        assert ((got.cpu().double() - want).abs()
                <= err + ref.B * got.cpu().double().abs() + 2.0 ** -133).all(), (a, b)
    xs = torch.full((rows, K // 32), 127, dtype=torch.uint8)
    ws = torch.full((1, N, K // 32), 127, dtype=torch.uint8)
    for group in range(K // 32):
        one = xs.clone()
        one[1, group] = 255
        got = grouped_gemm(_on_gpu((xv, one)), mxfp4_expert_weights(wv.to(DEV), ws.to(DEV)), off)
        nan = torch.isnan(got).cpu()
        assert nan[1].all() and int(nan.sum()) == N, group
        one = ws.clone()
        one[0, 5, group] = 255
        got = grouped_gemm(_on_gpu((xv, xs)), mxfp4_expert_weights(wv.to(DEV), one.to(DEV)), off)
        nan = torch.isnan(got).cpu()
        assert nan[:, 5].all() and int(nan.sum()) == rows, group


def test_captured_chain():
    """Quantisation, gated product, quantisation and the down projection in a
    graph, replayed with other rows and other offsets."""
    E, R, D, F = 6, 300, 256, 160
    gen = _gen(12)
    w13 = quantize_mxfp4((torch.randn(E, 2 * F, D, generator=gen) * D ** -0.5).to(DEV))
    w2 = quantize_mxfp4((torch.randn(E, D, F, generator=gen) * F ** -0.5).to(DEV))
    p13, p2 = mxfp4_expert_weights(*w13), mxfp4_expert_weights(*w2)
    x = torch.zeros(R, D, dtype=BF, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)

    def chain():
        h = gated_grouped_gemm(quantize_mxfp4(x), p13, off)
        return grouped_gemm(quantize_mxfp4(h), p2, off)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = chain()
    for seed in range(4):
        x.copy_(torch.randn(R, D, generator=_gen(seed)).to(BF))
        cut = torch.sort(torch.randint(0, R - 7, (E,), generator=_gen(seed)))[0].int()
        off[1:].copy_(cut)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, chain()), seed
        assert (got[int(cut[-1]):] == 0).all() and torch.isfinite(got).all()
