"""What the expert-layer calls of the Python binding refuse before the library is called, with
stand-ins of CUDA tensors (no GPU, nothing is launched)."""

import pytest
import torch

import matrix_aware_optimizers_gb300 as mao

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
E4M3 = torch.float8_e4m3fn


class Stand:
    """A contiguous tensor of a shape and type on a CUDA device, or (device -1) on the host."""

    def __init__(self, shape, dtype=F32, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.is_cuda = device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        st = torch.empty(self.shape, device="meta").stride()
        return st if i is None else st[i]

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def get_device(self):
        return self.index

    def on(self, device):
        return Stand(self.shape, self.dtype, device)


class Stream:
    def __init__(self, device):
        self.cuda_stream, self.device_index = 64, device


class Library:
    """Sizes from the library itself; calls are noted and succeed."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name == "expert_rows":
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def calls(lib, monkeypatch):
    """Calls that reach the library; the current device is 0, new tensors are stand-ins."""
    fake = Library(lib)
    monkeypatch.setattr(mao, "lib", lambda: fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 32, raising=False)

    def out(t, shape, dtype, name, like, stream):
        if t is None:
            t = Stand((shape,) if isinstance(shape, int) else shape, dtype, like.index)
        return t, t.data_ptr()

    monkeypatch.setattr(mao, "_out", out)
    return fake.calls


# Each call with its tensors by name; the rest of its arguments.
CALLS = {
    "fp8_quantize": (mao.fp8_quantize, dict(X=Stand((40, 256), BF16), rows=Stand((9,), I32)), dict(blocks="row")),
    "fp8_quantize stacked": (mao.fp8_quantize, dict(X=Stand((3, 40, 256))), dict(blocks="tile")),
    "fp8_quantize out": (
        lambda X, a, b, **o: mao.fp8_quantize(X, out=(a, b), **o),
        dict(X=Stand((40, 256)), a=Stand((40, 256), E4M3), b=Stand((40, 2), U8)), dict(blocks="row")),
    "fp8_quantize list": (
        lambda a, b, **o: mao.fp8_quantize([a, b], **o), dict(a=Stand((40, 256)), b=Stand((40, 256))),
        dict(blocks="col")),
    "fp8_product": (
        mao.fp8_product,
        dict(A=Stand((40, 256), E4M3), a_scales=Stand((40, 2), U8), B=Stand((2, 128, 256), E4M3),
             b_scales=Stand((2, 1, 2), U8), offsets=Stand((3,), I32), out=Stand((40, 128), BF16),
             ws=Stand((512,), U8)), dict(form="nt")),
    "expert_route": (
        mao.expert_route, dict(logits=Stand((5, 16)), bias=Stand((16,)), weights=Stand((5, 2)), ids=Stand((5, 2), I32)),
        dict(top_k=2)),
    "expert_route_backward": (
        mao.expert_route_backward,
        dict(logits=Stand((5, 16)), ids=Stand((5, 2), I32), dweights=Stand((5, 2)), dlogits=Stand((5, 16))), {}),
    "expert_plan": (mao.expert_plan, dict(ids=Stand((5000, 2), I32), ws=Stand((1 << 20,), U8)), dict(experts=8)),
    "expert_combine": (
        mao.expert_combine,
        dict(Z=Stand((256, 40)), row_of=Stand((5, 2), I32), weights=Stand((5, 2)), out=Stand((5, 40))), {}),
    "expert_combine_backward": (
        mao.expert_combine_backward,
        dict(dY=Stand((5, 40)), Z=Stand((256, 40)), row_of=Stand((5, 2), I32), slot_of=Stand((256,), I32),
             weights=Stand((5, 2)), dZ=Stand((256, 40)), dweights=Stand((5, 2))), {}),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(calls, name):
    """The library launches on the current device: a tensor or a stream of another is an error."""
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


class Gaps(Stand):
    def is_contiguous(self):
        return False

    def on(self, device):
        return Gaps(self.shape, self.dtype, device)


@pytest.mark.parametrize("name", ["fp8_product", "expert_plan"])
def test_workspaces_on_the_host_or_with_gaps_are_refused(calls, name):
    call, tensors, rest = CALLS[name]
    for ws in (Stand((1 << 20,), U8, -1), Gaps((1 << 20,), U8)):
        with pytest.raises(ValueError):
            call(**dict(tensors, ws=ws), **rest)
    assert not calls


def test_unknown_kinds_of_scores_are_refused(calls):
    """With ValueError, as the other calls refuse an unknown kind."""
    x, ids, g = Stand((5, 16)), Stand((5, 2), I32), Stand((5, 2))
    for opts in (dict(score="tanh"), dict(score=None), dict(group_score="mean"), dict(group_score=2)):
        with pytest.raises(ValueError):
            mao.expert_route(x, 2, **opts)
    with pytest.raises(ValueError):
        mao.expert_route_backward(x, ids, g, score="tanh")
    assert not calls


def test_no_matrices_to_quantise_are_refused(calls):
    for X in ([], ()):
        with pytest.raises(ValueError):
            mao.fp8_quantize(X, "row")
    assert not calls


@pytest.mark.parametrize("copies", [0, -1, 2 ** 31, 2 ** 32 + 1])
def test_copies_that_no_row_number_reaches_are_refused(calls, copies):
    """Passed on in 32 bits, 2^32 + 1 copies would be taken for one."""
    with pytest.raises(ValueError):
        mao.fp8_quantize(Stand((40, 256)), "row", rows=Stand((9,), I32), copies=copies)
    assert not calls


class Watched(Stand):
    """Counts the looks at its shape and strides, which cost a real tensor about 0.3 us each."""

    def __init__(self, *args):
        self.seen = dict(shape=0, stride=0)
        super().__init__(*args)

    def __getattribute__(self, name):
        if name in ("shape", "stride", "dim"):
            self.seen["stride" if name == "stride" else "shape"] += 1
        return super().__getattribute__(name)


def test_a_matrix_is_looked_at_once():
    """One descriptor per matrix and step: a step of many matrices makes over a thousand."""
    t = Watched((4, 8))
    t.stride = lambda i=None: (8, 1) if i is None else (8, 1)[i]
    t.seen.update(shape=0, stride=0)
    m = mao._mat(t)
    assert (m.rows, m.cols, m.ld) == (4, 8, 8)
    assert t.seen == dict(shape=1, stride=1)


@pytest.mark.parametrize("shape,strides,ld", [((4, 8), (8, 1), 8), ((4, 8), (11, 1), 11), ((1, 8), (0, 1), 8),
                                              ((1, 8), (3, 1), 8), ((4, 1), (1, 1), 1), ((4, 8), (7, 1), None),
                                              ((4, 8), (0, 1), None), ((4, 8), (1, 4), None), ((4,), (1,), None),
                                              ((2, 4, 8), (32, 8, 1), None)])
def test_descriptors_of_matrices(shape, strides, ld):
    t = Stand(shape)
    t.stride = lambda i=None: strides if i is None else strides[i]
    if ld is None:
        with pytest.raises(ValueError):
            mao._mat(t)
    else:
        m = mao._mat(t)
        assert (m.data, m.rows, m.cols, m.ld, m.dtype) == (0x10000,) + shape + (ld, 0)
