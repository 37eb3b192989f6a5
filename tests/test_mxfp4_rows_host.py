"""CPU tests of the host side of 4-bit rows: every refusal happens before
anything is enqueued, and the rule that chooses the products' form."""
import ctypes as C

import pytest
import torch

import combine_moe_layout_05_amd as moe
import test_gpu_mxfp4_rows as gpu
from combine_moe_layout_05_amd import _lib as L

P = 1 << 56                # a device address that is never dereferenced; buffers lie P apart
OK, BAD = L.MOE_OK, L.MOE_ERR_INVALID_ARG
MAX = L.MOE_MAX_GEMM_WIDTH

QUANT = dict(x=P, dtype=L.MOE_BF16, rows=0, width=64, values=2 * P, scales=3 * P, stream=None)
BACK = dict(values=2 * P, scales=3 * P, dtype=L.MOE_F32, rows=0, width=64, x=P, stream=None)
PLAIN = dict(values=P, scales=2 * P, w=3 * P, offsets=4 * P, E=4, rows=0, k=64, n=32, out=5 * P,
             flags=1, stream=None)
GATED = dict(values=P, scales=2 * P, w=3 * P, offsets=4 * P, E=4, rows=0, k=64, n=32, act=0,
             out=5 * P, flags=9, stream=None)


@pytest.fixture(scope="module")
def lib():
    return L.load()


def test_quantisation_refusals(lib):
    for fn, args in ((lib.moe_quantize_mxfp4, QUANT), (lib.moe_dequantize_mxfp4, BACK)):
        assert fn(*args.values()) == OK
        for key, value in [("dtype", 2), ("rows", -1), ("width", 0), ("width", 16), ("width", 48),
                           ("width", MAX + 32), ("rows", 1 << 30)]:
            assert fn(*dict(args, **{key: value}).values()) == BAD, (key, value)
        args = dict(args, rows=4)
        for key in ("x", "values", "scales"):
            assert fn(*dict(args, **{key: None}).values()) == BAD, key
        for key in ("x", "values"):
            assert fn(*dict(args, **{key: args[key] + 8}).values()) == BAD, key
    args = dict(QUANT, rows=4)
    for bad in (dict(values=P), dict(values=P + 4 * 64 * 2 - 16), dict(scales=P + 511),
                dict(scales=2 * P), dict(scales=2 * P + 127), dict(values=3 * P)):
        assert lib.moe_quantize_mxfp4(*dict(args, **bad).values()) == BAD, bad
    args = dict(BACK, rows=4)
    for bad in (dict(x=2 * P), dict(x=2 * P - 16), dict(x=3 * P), dict(x=2 * P + 112)):
        assert lib.moe_dequantize_mxfp4(*dict(args, **bad).values()) == BAD, bad


@pytest.mark.parametrize("name, args", [("moe_grouped_gemm_mxfp4_rows", PLAIN),
                                        ("moe_gated_grouped_gemm_mxfp4_rows", GATED)])
def test_product_refusals(lib, name, args):
    fn = getattr(lib, name)
    assert fn(*args.values()) == OK
    bad = [("E", 0), ("E", L.MOE_MAX_EXPERTS + 1), ("rows", -1), ("rows", 1 << 31), ("k", 0),
           ("k", 48), ("k", MAX + 32), ("n", 0), ("n", 20), ("n", MAX + 8), ("flags", 2),
           ("flags", 4)]
    if "act" in args:
        bad += [("act", 2), ("act", -1), ("n", 24), ("n", MAX // 2 + 16)]
    for key, value in bad:
        assert fn(*dict(args, **{key: value}).values()) == BAD, (key, value)
    args = dict(args, rows=8)
    for key in ("values", "scales", "w", "offsets", "out"):
        assert fn(*dict(args, **{key: None}).values()) == BAD, key
    for key, by in (("values", 8), ("w", 8), ("offsets", 2), ("out", 8)):
        assert fn(*dict(args, **{key: args[key] + by}).values()) == BAD, key
    out = 8 * 32 * 2
    for key, size in (("values", 8 * 32), ("scales", 16), ("offsets", 20),
                      ("w", 4 * (4 if "act" in args else 2) * 1088)):
        for at in (args[key], args[key] + (size - 1) // 16 * 16, args[key] + 16 - out):
            assert fn(*dict(args, out=at).values()) == BAD, (key, at)
    # past the work-items of a launch
    assert fn(*dict(args, E=1, rows=(1 << 31) - 1, k=32, n=16).values()) == BAD
    assert fn(*dict(args, E=1024, rows=8192, k=32, n=MAX // 2).values()) == BAD


class _Cuda(torch.Tensor):
    """A CPU tensor that says it is on a GPU: what the checks see."""
    is_cuda = property(lambda self: True)


def _fake(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Cuda)


def test_binding_refusals(monkeypatch):
    from combine_moe_layout_05_amd import experts, moe as core
    calls = []
    monkeypatch.setattr(core, "_call", lambda *a: calls.append(a))
    monkeypatch.setattr(experts, "_call", lambda *a: calls.append(a))
    with pytest.raises(ValueError, match="must be on a GPU"):
        moe.quantize_mxfp4(torch.zeros(2, 32))
    for x, error in ((_fake(2, 32, dtype=torch.float16), TypeError),
                     (_fake(2, 48, dtype=torch.float32), ValueError),
                     (_fake(32, 2, dtype=torch.float32).t(), ValueError),
                     (_fake(2, 0, dtype=torch.float32), ValueError)):
        with pytest.raises(error):
            moe.quantize_mxfp4(x)
    rows = moe.Mxfp4Rows(_fake(8, 32), _fake(8, 2))
    with pytest.raises(TypeError, match="dtype must be"):
        moe.dequantize_mxfp4(rows, torch.float16)
    for bad in (moe.Mxfp4Rows(_fake(8, 32), _fake(8, 4)), moe.Mxfp4Rows(_fake(8, 24), _fake(8, 2)),
                moe.Mxfp4Rows(_fake(8, 32), _fake(7, 2))):
        with pytest.raises(ValueError, match="shapes"):
            moe.dequantize_mxfp4(bad)
    packed = moe.Mxfp4ExpertWeights(_fake(4 * 2 * 1088), 4, 32, 64)
    off, i32 = _fake(5, dtype=torch.int32), torch.int32
    assert moe.grouped_gemm(rows, packed, off).shape == (8, 32)
    assert moe.gated_grouped_gemm(rows, packed, off).shape == (8, 16)
    n = len(calls)
    w = _fake(4, 32, 64, dtype=torch.bfloat16)
    for call in (moe.grouped_gemm, moe.gated_grouped_gemm):
        with pytest.raises(TypeError, match="weights packed"):
            call(rows, w, off)
        with pytest.raises(ValueError, match="shapes"):
            call(moe.Mxfp4Rows(_fake(8, 16), _fake(8, 1)), packed, off)
        with pytest.raises(ValueError, match="shapes"):
            call(rows, packed, _fake(4, dtype=i32))
        with pytest.raises(TypeError, match="offsets must be"):
            call(rows, packed, _fake(5, dtype=torch.int64))
        with pytest.raises(ValueError, match="packed weights must hold"):
            call(rows, packed._replace(data=_fake(64)), off)
        with pytest.raises(ValueError, match="out must be"):
            call(rows, packed, off, _fake(8, 24, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="row_tile"):
        moe.grouped_gemm(rows, packed, off, row_tile=64)
    with pytest.raises(ValueError, match="no backward"):
        moe.gated_grouped_gemm(rows, packed, off, pre=_fake(8, 32, dtype=torch.float32))
    with pytest.raises(ValueError, match="multiple of 16"):
        moe.gated_grouped_gemm(rows, moe.Mxfp4ExpertWeights(_fake(4 * 2 * 1088), 4, 24, 64), off)
    assert len(calls) == n


def test_both_forms_are_tested(lib):
    rule = getattr(lib, "_ZN3moe18expert_mx4_streamsEill")
    rule.argtypes, rule.restype = [C.c_int32, C.c_int64, C.c_int64], C.c_bool
    few, many = gpu.SHAPES[:5], gpu.SHAPES[5:]
    for shapes, streams in ((few, True), (many, False)):
        for counts, behind, K, F, N in shapes:
            rows = sum(counts) + behind
            assert rule(len(counts), rows, N) == rule(len(counts), rows, 2 * F) == streams
    tile = getattr(lib, "_ZN3moe20expert_mx4_tile_rowsEbili")
    tile.argtypes, tile.restype = [C.c_bool, C.c_int32, C.c_int64, C.c_int32], C.c_int
    for i, (counts, behind, K, F, N) in enumerate(many):
        E, rows = len(counts), sum(counts) + behind
        want = 128 if i >= len(many) - gpu.TILES_128 else 64
        assert tile(False, E, rows, N) == tile(True, E, rows, F) == want, i
    large = many[-gpu.TILES_128:]
    assert {-(-(c % 128) // 16) for counts, *_ in large for c in counts} >= {0, 1, 2, 3, 4, 6, 8}
    assert any(K > 7680 for _, _, K, _, _ in large)
    # whole and partial sums of odd and even numbers of 128-element halves, and
    # last row tiles of one to four 16-row blocks
    assert {(-(-K // 128) % 2, K % 128 != 0) for _, _, K, _, _ in many} == {
        (0, False), (0, True), (1, False), (1, True)}
    assert {-(-(c % 64) // 16) for counts, *_ in many for c in counts if c % 64} == {1, 2, 3, 4}


def test_forward_mode_is_refused(monkeypatch):
    from combine_moe_layout_05_amd import experts
    calls = []
    monkeypatch.setattr(experts, "_call", lambda *a: calls.append(a))
    x = _fake(2, 32, dtype=torch.float32)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError, match="quantize_mxfp4 has no forward-mode"):
            moe.quantize_mxfp4(dual)
        assert not calls
        moe.quantize_mxfp4(x)
    moe.quantize_mxfp4(x)
    assert len(calls) == 2
