"""What the feed-forward calls refuse before anything is launched, in the binding (with stand-ins of
CUDA tensors) and at the C ABI, and the sizes they report without a GPU."""

import ctypes

import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from matrix_aware_optimizers_gb300 import _abi
from test_experts_binding_cpu import BF16, F32, I32, U8, Stand, Stream, calls  # noqa: F401

I8 = torch.int8
FAKE = 0x10000  # never dereferenced: the calls below fail validation, or only report sizes

FFN = dict(X=Stand((40, 64), BF16), up=Stand((2, 96, 64), BF16), down=Stand((2, 72, 48), BF16),
           offsets=Stand((3,), I32), counts=Stand((2,), I32))
CALLS = {
    "gated_ffn": (mao.gated_ffn, dict(FFN, out=Stand((40, 72), BF16), Z=Stand((40, 96), BF16), ws=Stand((1 << 20,), U8)), {}),
    "gated_ffn_backward": (
        mao.gated_ffn_backward,
        dict(FFN, dY=Stand((40, 72), BF16), Z=Stand((40, 96), BF16), dX=Stand((40, 64), F32),
             dup=Stand((2, 96, 64), F32), ddown=Stand((2, 72, 48), BF16), ws=Stand((1 << 20,), U8)), {}),
    "int8_quantize": (mao.int8_quantize, dict(X=Stand((40, 256), BF16)), dict(gate="silu")),
    "int8_quantize list": (lambda a, b, **o: mao.int8_quantize([a, b], **o),
                           dict(a=Stand((40, 256)), b=Stand((40, 256))), {}),
    "int8_quantize out": (lambda X, a, b, **o: mao.int8_quantize(X, out=(a, b), **o),
                          dict(X=Stand((40, 256)), a=Stand((40, 256), I8), b=Stand((40,))), {}),
    "int8_product": (
        mao.int8_product,
        dict(A=Stand((40, 256), I8), a_scales=Stand((40,)), B=Stand((2, 128, 256), I8), b_scales=Stand((2, 128)),
             offsets=Stand((3,), I32), counts=Stand((2,), I32), out=Stand((40, 128), BF16), ws=Stand((512,), U8)), {}),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(calls, name):  # noqa: F811
    call, tensors, rest = CALLS[name]
    call(**tensors, **rest)
    assert len(calls) == 1 and calls[0][1][-1] == 32
    call(**tensors, **rest, stream=Stream(0))
    assert len(calls) == 2 and calls[1][1][-1] == 64
    for which in tensors:
        with pytest.raises(ValueError):
            call(**dict(tensors, **{which: tensors[which].on(1)}), **rest)
    with pytest.raises(ValueError):
        call(**{k: t.on(1) for k, t in tensors.items()}, **rest)
    with pytest.raises(ValueError):
        call(**tensors, **rest, stream=Stream(1))
    assert len(calls) == 2


@pytest.mark.parametrize("change", [
    dict(X=Stand((40, 64), F32)), dict(up=Stand((2, 96, 64), F32)), dict(down=Stand((2, 72, 48), F32)),
    dict(up=Stand((2, 95, 64), BF16)), dict(up=Stand((2, 96, 63), BF16)), dict(up=Stand((3, 96, 64), BF16)),
    dict(up=Stand((96, 64), BF16)), dict(down=Stand((72, 48), BF16)), dict(down=Stand((1, 2, 72, 48), BF16)),
    dict(offsets=Stand((3,), F32)), dict(offsets=Stand((1,), I32)), dict(counts=Stand((3,), I32)),
    dict(counts=Stand((2,), F32)), dict(offsets=None), dict(ws=Stand((1 << 20,), U8, -1)), dict(act="relu"),
    dict(act=None), dict(X=Stand((40, 64), BF16, -1))])
def test_blocks_that_do_not_fit_are_refused(calls, change):  # noqa: F811
    for name in ("gated_ffn", "gated_ffn_backward"):
        call, tensors, rest = CALLS[name]
        with pytest.raises(ValueError):
            call(**dict(tensors, **change))
    assert not calls


def test_types_and_shapes_of_codes_are_refused(calls):  # noqa: F811
    call, tensors, rest = CALLS["int8_product"]
    for change in (dict(A=Stand((40, 256), U8)), dict(A=Stand((1, 40, 256), I8)), dict(a_scales=Stand((41,))),
                   dict(a_scales=Stand((40,), BF16)), dict(B=Stand((128, 256), BF16)), dict(b_scales=Stand((2, 127))),
                   dict(counts=Stand((1,), I32)), dict(offsets=None), dict(out_dtype=torch.float16, out=None)):
        with pytest.raises(ValueError):
            call(**dict(tensors, **change))
    for X, opts in ((Stand((4, 7)), dict(gate="silu")), (Stand((4, 8)), dict(gate="tanh")), ([], {}),
                    (Stand((4, 8), I8), {}), (Stand((4, 8)), dict(out=(Stand((4, 8), U8), Stand((4,)))))):
        with pytest.raises(ValueError):
            mao.int8_quantize(X, **opts)
    with pytest.raises(ValueError):
        mao.gated_ffn(Stand((4, 64), BF16), Stand((96, 64), BF16), Stand((72, 48), BF16), out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mao.gated_ffn_backward(Stand((4, 72), BF16), Stand((4, 64), BF16), Stand((96, 64), BF16), Stand((72, 48), BF16),
                               Stand((4, 96), BF16), grad_dtype=torch.float16)
    for save in (torch.float16, "bf16", 1):
        with pytest.raises(ValueError):
            mao.gated_ffn(Stand((4, 64), BF16), Stand((96, 64), BF16), Stand((72, 48), BF16), save=save)
    assert not calls


def mat(rows, cols, dtype=_abi.MAO_BF16, ld=None, data=FAKE, reserved=0):
    return _abi.MaoMat(data, rows, cols, cols if ld is None else ld, dtype, reserved)


def codes(rows, cols, ld=None, count=1, data=FAKE, scales=FAKE, reserved=0):
    return _abi.MaoInt8(data, scales, rows, cols, -(-cols // 16) * 16 if ld is None else ld, count, reserved)


def test_block_arguments_rejected_before_any_launch(lib):
    off, bad = ctypes.c_void_p(FAKE), _abi.MAO_ERR_INVALID_ARG

    def fwd(X=mat(9, 64), up=mat(96, 64), down=mat(72, 48), act=0, offsets=None, counts=None, groups=1,
            Z=None, Y=mat(9, 72)):
        return lib.gated_ffn(X, up, down, act, offsets, counts, groups, Z, Y, ctypes.c_void_p(FAKE), 1 << 30, None)

    F, I = _abi.MAO_F32, _abi.MAO_I8
    for kw in (dict(X=None), dict(up=None), dict(down=None), dict(Y=None), dict(act=-1), dict(act=3), dict(groups=0),
               dict(groups=2), dict(counts=off), dict(X=mat(9, 64, F)), dict(up=mat(96, 64, F)), dict(X=mat(9, 64, I)),
               dict(up=mat(97, 64)), dict(up=mat(96, 65)), dict(down=mat(72, 47)), dict(down=mat(0, 48)),
               dict(Y=mat(9, 71)), dict(Y=mat(8, 72)), dict(Z=mat(9, 95)), dict(Z=mat(9, 96, I)), dict(X=mat(-1, 64)),
               dict(X=mat(9, 64, ld=63)), dict(X=mat(9, 64, data=None)), dict(Y=mat(9, 72, reserved=1)),
               dict(groups=2, offsets=off, down=mat(73, 48), up=mat(192, 64))):
        assert fwd(**kw) == bad, kw
    assert fwd(offsets=ctypes.c_void_p(FAKE + 2)) == _abi.MAO_ERR_MISALIGNED
    assert fwd(X=mat(9, 64, data=FAKE + 1)) == _abi.MAO_ERR_MISALIGNED
    assert fwd(groups=1025, offsets=off) == _abi.MAO_ERR_UNSUPPORTED
    assert fwd(X=mat(2 ** 31, 64), Y=mat(2 ** 31, 72)) == _abi.MAO_ERR_UNSUPPORTED
    assert fwd(X=mat(9, 64, ld=2 ** 40)) == _abi.MAO_ERR_UNSUPPORTED

    def bwd(dY=mat(9, 72), X=mat(9, 64), up=mat(96, 64), down=mat(72, 48), Z=mat(9, 96), act=0, dX=None, dup=None,
            ddown=None):
        return lib.gated_ffn_backward(dY, X, up, down, Z, act, None, None, 1, dX, dup, ddown, ctypes.c_void_p(FAKE),
                                      1 << 30, None)

    for kw in (dict(dY=None), dict(Z=None), dict(dY=mat(9, 73)), dict(dY=mat(9, 72, F)), dict(Z=mat(9, 97)),
               dict(dX=mat(9, 63)), dict(dup=mat(95, 64)), dict(ddown=mat(72, 49)), dict(dX=mat(9, 64, I)), dict(act=7)):
        assert bwd(**kw) == bad, kw


def test_int8_arguments_rejected_before_any_launch(lib):
    bad, off = _abi.MAO_ERR_INVALID_ARG, ctypes.c_void_p(FAKE)

    def quantize(X=mat(9, 64, _abi.MAO_F32), batch=1, stride=0, gated=0, act=0, out=codes(9, 64)):
        return lib.int8_quantize(X, batch, stride, gated, act, out, None)

    for kw in (dict(X=None), dict(out=None), dict(batch=0), dict(stride=-1), dict(gated=1), dict(out=codes(8, 64)),
               dict(out=codes(9, 63)), dict(out=codes(9, 64, ld=72)), dict(out=codes(9, 64, count=2)),
               dict(out=codes(9, 64, data=None)), dict(out=codes(9, 64, scales=None)), dict(out=codes(9, 64, reserved=1)),
               dict(X=mat(9, 64, _abi.MAO_I8)), dict(gated=1, act=3, out=codes(9, 32))):
        assert quantize(**kw) == bad, kw
    assert quantize(out=codes(9, 64, data=FAKE + 8)) == _abi.MAO_ERR_MISALIGNED
    assert quantize(out=codes(9, 64, scales=FAKE + 2)) == _abi.MAO_ERR_MISALIGNED

    def product(A=codes(9, 64), B=codes(48, 64), D=mat(9, 48), offsets=None, counts=None, groups=1):
        return lib.int8_product(A, B, D, offsets, counts, groups, None, 0, None)

    for kw in (dict(A=None), dict(B=None), dict(D=None), dict(A=codes(9, 65)), dict(B=codes(47, 64)), dict(D=mat(8, 48)),
               dict(A=codes(9, 64, count=2)), dict(groups=2), dict(groups=2, offsets=off), dict(counts=off),
               dict(B=codes(0, 64), D=mat(9, 0)), dict(D=mat(9, 48, _abi.MAO_I8))):
        assert product(**kw) == bad, kw
    assert product(offsets=off, groups=1025, B=codes(48, 64, count=1025)) == _abi.MAO_ERR_UNSUPPORTED


def test_sizes_without_a_gpu(lib):
    """Workspaces hold the intermediate rows, and copies of operands whose rows are not aligned."""
    H = lambda rows, n: rows * n * 2  # noqa: E731
    size = lambda X, up, down, g=1, grouped=0: lib.gated_ffn_workspace_bytes(X, up, down, g, grouped)  # noqa: E731
    plain = size(mat(1000, 64), mat(96, 64), mat(72, 48))
    assert plain >= H(1000, 48)
    assert size(mat(1000, 64, ld=65), mat(96, 64), mat(72, 48)) >= plain + H(1000, 64)
    assert size(mat(1000, 64, data=FAKE + 2), mat(96, 64), mat(72, 48)) >= plain + H(1000, 64)
    assert size(mat(0, 64), mat(96, 64), mat(72, 48)) == 0
    assert size(mat(9, 64), mat(96, 63), mat(72, 48)) == 0
    assert size(mat(1024, 64), mat(8 * 96, 64), mat(8 * 72, 48), 8, 1) == H(1024, 48)
    back = lib.gated_ffn_backward_workspace_bytes(mat(1000, 72), mat(1000, 64), mat(96, 64), mat(72, 48), 1, 0)
    assert back >= 3 * H(1000, 48)
    few, more = (lib.int8_product_workspace_bytes(codes(n, 64), codes(48, 64), 0) for n in (16, 17))
    assert few == 0 and more >= 17 * 64 * 2
