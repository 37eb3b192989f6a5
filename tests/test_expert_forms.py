"""CPU tests of the rules that choose an expert product's form: the GPU tests'
cases run in the forms that they are there for."""
import ctypes as C

import pytest

import test_gpu_expert_tiles as tiles
from combine_moe_layout_05_amd import _lib as L

PLAIN, GATED, INPUT_GRAD, GATED_GRAD = range(4)      # the library's ExpertOp


@pytest.fixture(scope="module")
def rules():
    """The library's own rules, by their C++ names."""
    lib = L.load()

    def rule(name, *types):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = types, C.c_bool
        return fn

    i32, i64 = C.c_int32, C.c_int64
    return dict(small=rule("_ZN3moe17expert_small_tileENS_8ExpertOpEili", C.c_int, i32, i64, i32),
                bf16=rule("_ZN3moe19expert_streams_bf16El", i64),
                mxfp4=rule("_ZN3moe20expert_streams_mxfp4Eill", i32, i64, i64))


@pytest.mark.parametrize("counts, behind, red, gated, plain", tiles.LARGE)
def test_large_tiles(rules, counts, behind, red, gated, plain):
    E, rows = len(counts), sum(counts) + behind
    assert not rules["bf16"](rows)
    for op in (PLAIN, GATED, INPUT_GRAD, GATED_GRAD):
        assert not rules["small"](op, E, rows, gated if op == GATED else plain), op


def test_large_tiles_leave_every_number_of_64_row_parts():
    for list_ in (tiles.LARGE, tiles.LARGE[:1]):
        last = {-(-(c % 256) // 64) for counts, *_ in list_ for c in counts if c % 256}
        assert last == {1, 2, 3, 4}


@pytest.mark.parametrize("K, F, N", tiles.TILED)
def test_tiled_4_bit_products(rules, K, F, N):
    E, rows = len(tiles.TILED_ROWS), sum(tiles.TILED_ROWS) + tiles.TILED_BEHIND
    assert not rules["mxfp4"](E, rows, 2 * F) and not rules["mxfp4"](E, rows, N)


def test_tiled_4_bit_products_cover_the_loop():
    """More steps than the three stages, odd and even numbers of them, whole
    and partial last ones, and last row tiles of one to four 16-row blocks."""
    kinds = {(-(-K // 128) % 2, K % 128 != 0) for K, _, _ in tiles.TILED if K > 3 * 128}
    assert kinds == {(0, False), (0, True), (1, False), (1, True)}
    assert {-(-(c % 64) // 16) for c in tiles.TILED_ROWS if c % 64} == {1, 2, 3, 4}


def test_long_segments_of_the_weight_gradient():
    for counts, _, K, N in tiles.DEEP:
        assert any(c >= 2048 for c in counts) and -(-N // 128) >= 8


def test_both_forms_are_chosen(rules):
    """The rules answer differently on either side of their limits."""
    assert rules["bf16"](64) and not rules["bf16"](65)
    assert rules["small"](GATED, 128, 4096, 2048) and not rules["small"](GATED, 128, 4097, 2048)
    assert rules["small"](GATED, 1, 2048, 2048) and not rules["small"](GATED, 1, 2049, 2048)
    assert rules["mxfp4"](128, 1024, 4096) and not rules["mxfp4"](128, 1025, 4096)
