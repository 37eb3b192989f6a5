"""CPU tests of the host side of the whole layer for a few tokens: every
refusal happens before anything is enqueued."""
import pytest
import torch

import combine_moe_layout_05_amd as moe
from combine_moe_layout_05_amd import _lib as L

P = 1 << 56                # a device address that is never dereferenced; buffers lie P apart
OK, BAD = L.MOE_OK, L.MOE_ERR_INVALID_ARG
MAX = L.MOE_MAX_GEMM_WIDTH

CALL = dict(x=P, scores=2 * P, ids=3 * P, T=0, K=8, w1=4 * P, w2=5 * P, layout=0, E=16, hidden=64,
            n_hidden=32, act=0, ws=6 * P, bytes=1 << 40, y=7 * P, stream=None)


@pytest.fixture(scope="module")
def lib():
    return L.load()


@pytest.mark.parametrize("layout", [L.MOE_WEIGHTS_ROW_MAJOR, L.MOE_WEIGHTS_MXFP4])
def test_sizes(lib, layout):
    fn, args = lib.moe_few_tokens_layer, dict(CALL, layout=layout)
    assert fn(*args.values()) == OK
    bad = [("T", -1), ("T", 65), ("K", 0), ("K", 17), ("layout", 1), ("layout", 3), ("E", 0),
           ("E", 1025), ("hidden", 0), ("hidden", 12), ("hidden", MAX + 32), ("n_hidden", 0),
           ("n_hidden", 20), ("n_hidden", MAX // 2 + 32), ("act", 2)]
    if layout == L.MOE_WEIGHTS_MXFP4:
        bad += [("hidden", 72), ("n_hidden", 40)]
        # more weights than a packing launch takes
        assert fn(*dict(args, E=1024, hidden=MAX, n_hidden=MAX // 2).values()) == BAD
    for key, value in bad:
        assert fn(*dict(args, **{key: value}).values()) == BAD, (key, value)
    # past the work-items of a launch
    assert fn(*dict(args, T=64, E=1024, hidden=32, n_hidden=MAX // 2).values()) == BAD


def test_workspace(lib):
    size = lib.moe_few_tokens_workspace_bytes
    assert size(1, 8, 2048) == 8 * 2048 * 4 and size(0, 1, 8) == 0
    assert size(512, 1, 8) == 512 * 512 and size(513, 1, 8) == -1
    for bad in [(-1, 8, 64), (65, 8, 64), (1, 0, 64), (1, 17, 64), (1, 8, 12), (1, 8, MAX)]:
        assert size(*bad) == -1, bad
    fn, args = lib.moe_few_tokens_layer, dict(CALL, T=4)
    assert fn(*dict(args, bytes=4 * 8 * 128 * 4 - 1).values()) == L.MOE_ERR_WORKSPACE
    assert fn(*dict(args, bytes=-1).values()) == L.MOE_ERR_WORKSPACE


def test_pointers(lib):
    fn, args = lib.moe_few_tokens_layer, dict(CALL, T=4)
    for key in ("x", "scores", "ids", "w1", "w2", "ws", "y"):
        assert fn(*dict(args, **{key: None}).values()) == BAD, key
        by = 2 if key in ("scores", "ids") else 8
        assert fn(*dict(args, **{key: args[key] + by}).values()) == BAD, key
    sizes = dict(x=4 * 64 * 2, scores=128, ids=128, w1=16 * 64 * 64 * 2, w2=16 * 64 * 32 * 2,
                 ws=4 * 8 * 128 * 4)
    for key, size in sizes.items():
        for at in (args[key], args[key] + size - 16, args[key] + 16 - 4 * 64 * 2):
            assert fn(*dict(args, y=at).values()) == BAD, key
            if key != "ws":
                assert fn(*dict(args, ws=at).values()) == BAD, key


class _Cuda(torch.Tensor):
    """A CPU tensor that says it is on a GPU: what the checks see."""
    is_cuda = property(lambda self: True)


def _fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Cuda)


def test_binding_refusals(monkeypatch):
    from combine_moe_layout_05_amd import layer
    calls = []
    monkeypatch.setattr(layer, "_call", lambda *a: calls.append(a))
    T, E, K, D, F = 4, 3, 2, 64, 32
    good = dict(x=_fake(T, D), s=_fake(T, K, dtype=torch.float32),
                i=_fake(T, K, dtype=torch.int32), w1=_fake(E, 2 * F, D), w2=_fake(E, D, F))
    p1 = moe.Mxfp4ExpertWeights(_fake(E * 4 * 1088, dtype=torch.uint8), E, 2 * F, D)
    p2 = moe.Mxfp4ExpertWeights(_fake(E * 4 * 1088, dtype=torch.uint8), E, D, F)
    assert moe.moe_layer(*good.values()).shape == (T, D)
    # the workspace the binding gives is what the library asks for
    size = L.load().moe_few_tokens_workspace_bytes
    assert calls[0][-2] == size(T, K, F)
    for f in (8, 128, 136, 2048):
        moe.moe_layer(*dict(good, w1=_fake(E, 2 * f, D), w2=_fake(E, D, f)).values())
        assert calls[-1][-2] == size(T, K, f)
    assert moe.moe_layer(*dict(good, w1=p1, w2=p2).values()).shape == (T, D)
    n = len(calls)
    i32, f32 = torch.int32, torch.float32
    for error, match, more in [
            (TypeError, "x_TD must be", dict(x=_fake(T, D, dtype=f32))),
            (TypeError, "topk_scores_TK must be", dict(s=_fake(T, K))),
            (TypeError, "topk_expert_ids_TK must be", dict(i=_fake(T, K, dtype=torch.int64))),
            (ValueError, "contiguous", dict(x=_fake(D, T).t())),
            (ValueError, "shapes", dict(s=_fake(T + 1, K, dtype=f32))),
            (ValueError, "shapes", dict(i=_fake(T, K + 1, dtype=i32))),
            (ValueError, "shapes", dict(w1=_fake(E, F, D))),
            (ValueError, "shapes", dict(w1=_fake(E + 1, 2 * F, D))),
            (ValueError, "shapes", dict(w2=_fake(E, D + 8, F))),
            (TypeError, "both", dict(w1=p1)),
            (TypeError, "both", dict(w2=p2)),
            (ValueError, "shapes", dict(w1=p2, w2=p1)),
            (ValueError, "packed weights must hold", dict(
                w1=p1._replace(data=_fake(64, dtype=torch.uint8)), w2=p2)),
            (ValueError, "at most 512 slots", dict(
                x=_fake(257, D), s=_fake(257, K, dtype=f32), i=_fake(257, K, dtype=i32)))]:
        with pytest.raises(error, match=match):
            moe.moe_layer(*dict(good, **more).values())
    with pytest.raises(ValueError, match="activation"):
        moe.moe_layer(*good.values(), activation="relu")
    with pytest.raises(ValueError, match="must be on a GPU"):
        moe.moe_layer(*dict(good, x=torch.zeros(T, D, dtype=torch.bfloat16)).values())
    assert len(calls) == n


def test_forward_mode_is_refused(monkeypatch):
    from combine_moe_layout_05_amd import layer
    calls = []
    monkeypatch.setattr(layer, "_call", lambda *a: calls.append(a))
    T, E, K, D, F = 4, 3, 2, 64, 32
    i = _fake(T, K, dtype=torch.int32)
    good = [_fake(T, D), _fake(T, K, dtype=torch.float32), i, _fake(E, 2 * F, D), _fake(E, D, F)]
    with torch.autograd.forward_ad.dual_level():
        for k in (0, 1, 3, 4):
            args = list(good)
            args[k] = torch.autograd.forward_ad.make_dual(good[k], torch.ones_like(good[k]))
            with pytest.raises(NotImplementedError, match="moe_layer has no forward-mode"):
                moe.moe_layer(*args)
        assert not calls
        assert moe.moe_layer(*good).shape == (T, D)
    assert moe.moe_layer(*good).shape == (T, D) and len(calls) == 2
