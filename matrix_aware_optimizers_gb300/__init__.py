"""GB300 (sm_103a) Muon / Sign-Muon optimizer step behind a C ABI (libmao.so).

This module only marshals PyTorch CUDA tensors into the C ABI of include/mao.h;
every stage of the step runs in the library's CUDA kernels. There is no CPU or
PyTorch fallback: if libmao.so is missing, the calls raise.

Functions (same names as the C ABI):
  muon_momentum_update(M, G, mu)                     M <- mu*M + G
  ns_workspace_bytes(X, compute)                     workspace size for ns_orthogonalize
  ns_orthogonalize(inp, out, steps, coeffs, ...)     Newton–Schulz polar factor (+ packed signs)
  muon_step(W, M, G, mu, lr, ...)                    momentum + Newton–Schulz + update, fused
  muon_step_host(W, M, G, mu, lr, g_host, ...)      muon_step with host gradients / weights
  sign_muon_step(W, M, G, words, vote, mu, lr, ...)  momentum + NS signs + vote + update
  ns_orthogonalize_blockwise(inp, out, block, ...)   Newton–Schulz of every block on its own
  sign_pack_bits(U, bits)                            sign + 1-bit pack
  majority_vote_packed(bits, nbits, vote)            vote over workers' packed signs
  sign_int8(U, s)                                    sign as int8 +-1 (all-reduce variant)
  majority_vote_int8(s, n, sum, s_bar, vote)         int8 SUM over workers + threshold
  apply_update(W, lr, vote=..., U=...)               W <- W - lr*D
  dion_step(X, M, G, Q, mu, lr, ...)                 one Dion step (low-rank, error feedback)
  fp8_quantize(X, blocks, ...)                       8-bit codes with a scale per block of 128
  fp8_product(A, a_scales, B, b_scales, form, ...)   products of 8-bit matrices, grouped rows
  expert_route(logits, top_k, ...)                   choice and weights of each token's experts
  expert_route_backward(logits, ids, dweights, ...)  gradient of the logits
  expert_plan(ids, experts)                          places of the copies among the experts' rows
  expert_combine(Z, row_of, weights)                 weighted sum of a token's expert outputs
  expert_combine_backward(dY, Z, row_of, ...)        its gradients
  sync_status()                                      stream sync + device error word
"""

import ctypes
import functools

import torch

from . import _abi
from ._abi import MaoError  # noqa: F401

# Default Newton–Schulz coefficients (a, b, c): the quintic used by Muon.
QUINTIC = (3.4445, -4.7750, 2.0315)

_DT = {torch.float32: _abi.MAO_F32, torch.bfloat16: _abi.MAO_BF16, torch.int8: _abi.MAO_I8}
_COMPUTE = {"f32": _abi.MAO_F32, "bf16": _abi.MAO_BF16,
            torch.float32: _abi.MAO_F32, torch.bfloat16: _abi.MAO_BF16}


def lib():
    return _abi.load()


def _as_list(x):
    if x is None:
        return None
    return list(x) if isinstance(x, (list, tuple)) else [x]


class PackedSigns:
    """A rows x cols sign matrix held as packed words (int32 tensor of ceil(rows*cols/32)
    words, header layout), usable as an ns_orthogonalize input."""

    def __init__(self, words, rows, cols):
        if not words.is_cuda or words.dtype != torch.int32 or not words.is_contiguous():
            raise ValueError("words must be a contiguous int32 CUDA tensor")
        if words.numel() < packed_words(rows, cols):
            raise ValueError("too few words for a %d x %d sign matrix" % (rows, cols))
        self.words, self.shape = words, (int(rows), int(cols))
        self.device = words.device


def _mat(t, allow_none=False, like=None):
    if isinstance(t, PackedSigns):
        R, C = t.shape
        return _abi.MaoMat(t.words.data_ptr(), R, C, C, _abi.MAO_SIGN1, 0)
    if t is None:
        if not allow_none:
            raise ValueError("tensor required")
        return _abi.MaoMat(None, like.shape[0], like.shape[1], like.shape[1], _abi.MAO_F32, 0)
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    shape, st = t.shape, t.stride()  # one look at each: steps of many matrices come here often
    if len(shape) != 2 or st[1] != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    (rows, cols), ld = shape, st[0]
    if ld < cols:
        if rows > 1:
            raise ValueError("expected a tensor whose rows do not overlap")
        ld = cols
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError("dtype must be float32, bfloat16 or int8")
    return _abi.MaoMat(t.data_ptr(), rows, cols, ld, dt, 0)


def _mats(ts, allow_none=False, like=None):
    arr = (_abi.MaoMat * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = _mat(t, allow_none, like[i] if like is not None else None)
    return arr


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def muon_momentum_update(M, G, mu, stream=None):
    """M <- mu*M + G for each (M, G) pair (one fp32 FMA per element, rounded to M's dtype)."""
    Ms, Gs = _as_list(M), _as_list(G)
    st = lib().muon_momentum_update(_mats(Ms), _mats(Gs), len(Ms), float(mu), _stream(stream))
    _abi.check("muon_momentum_update", st)


def ns_workspace_bytes(X, compute="bf16"):
    Xs = _as_list(X)
    arr = (_abi.MaoMat * len(Xs))()
    for i, x in enumerate(Xs):
        shape = x.shape if hasattr(x, "shape") else x
        arr[i] = _abi.MaoMat(None, shape[0], shape[1], shape[1], _abi.MAO_F32, 0)
    n = lib().ns_workspace_bytes(arr, len(Xs), _COMPUTE[compute])
    if n == 0:
        raise ValueError("invalid shapes for ns_workspace_bytes")
    return int(n)


def workspace(X, compute="bf16", device=None):
    """A device buffer of ns_workspace_bytes(X) bytes (256-byte aligned by the allocator)."""
    n = ns_workspace_bytes(X, compute)
    dev = device if device is not None else torch.device("cuda")
    return torch.empty(n, dtype=torch.uint8, device=dev)


def ns_orthogonalize(inp, out, steps=5, coeffs=QUINTIC, eps=1e-7, compute="bf16",
                     sign_bits=None, ws=None, stream=None):
    """Newton–Schulz orthogonalisation of each input into out (and/or packed signs).

    coeffs: one (a, b, c) triple for every step, or a list of `steps` triples.
    out entries may be None when sign_bits (int32 tensors of ceil(R*C/32) words) are given.
    """
    ins = _as_list(inp)
    outs = _as_list(out) if out is not None else [None] * len(ins)
    co = list(coeffs)
    if len(co) == 3 and not isinstance(co[0], (list, tuple)):
        flat, stride = [float(c) for c in co], 0
    else:
        if len(co) != steps:
            raise ValueError("need one coefficient triple per step")
        flat, stride = [float(c) for t in co for c in t], 3
    carr = (ctypes.c_float * len(flat))(*flat)
    bits = _as_list(sign_bits)
    barr = None
    if bits is not None:
        barr = (ctypes.c_void_p * len(bits))(*[b.data_ptr() if b is not None else None for b in bits])
    if ws is None:
        ws = workspace(ins, compute, ins[0].device)
    st = lib().ns_orthogonalize(
        _mats(ins), _mats(outs, allow_none=True, like=ins), len(ins), int(steps), carr, stride,
        float(eps), _COMPUTE[compute], barr, ctypes.c_void_p(ws.data_ptr()), ws.numel(),
        _stream(stream))
    _abi.check("ns_orthogonalize", st)


def muon_step(W, M, G, mu, lr, steps=5, coeffs=QUINTIC, eps=1e-7, compute="bf16", ws=None,
              W_out=None, stream=None):
    """One whole Muon step: M <- mu*M + G, U = Newton-Schulz(M), W' = W - lr*U into W_out
    (W itself when W_out is None).

    U is never stored: the last product updates W from U's fp32 values. The workspace is
    that of ns_orthogonalize(M) (workspace(M, "bf16", device)).
    """
    Ws, Ms, Gs = _as_list(W), _as_list(M), _as_list(G)
    Wo = _as_list(W_out) if W_out is not None else None
    if not (len(Ws) == len(Ms) == len(Gs)) or (Wo is not None and len(Wo) != len(Ws)):
        raise ValueError("W, M, G (and W_out) need the same number of matrices")
    carr, stride = _coeff_args(coeffs, steps)
    if ws is None:
        ws = workspace(Ms, compute, Ms[0].device)
    st = lib().muon_step(_mats(Ws), _mats(Ms), _mats(Gs), _mats(Wo) if Wo is not None else None,
                         len(Ws), float(mu), float(lr),
                         int(steps), carr, stride, float(eps), _COMPUTE[compute],
                         ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(stream))
    _abi.check("muon_step", st)


def muon_step_host(W, M, G, mu, lr, g_host, g_dev, w_host, w_dev, steps=5, coeffs=QUINTIC,
                   eps=1e-7, compute="bf16", ws=None, W_out=None, stream=None, wait_event=None,
                   record_event=None):
    """muon_step with host data: g_host (pinned CPU tensor) is copied into g_dev (the device
    tensor whose storage holds G) before the step, and w_dev (the device tensor holding the
    new weights) into w_host (pinned CPU tensor) after it, all on `stream`; wait_event /
    record_event (torch.cuda.Event) order the step's compute across streams."""
    Ws, Ms, Gs = _as_list(W), _as_list(M), _as_list(G)
    Wo = _as_list(W_out) if W_out is not None else None
    if g_host.is_cuda or w_host.is_cuda or not g_dev.is_cuda or not w_dev.is_cuda:
        raise ValueError("g_host / w_host must be host tensors and g_dev / w_dev device tensors")
    gb = g_host.numel() * g_host.element_size()
    wb = w_dev.numel() * w_dev.element_size()
    if g_dev.numel() * g_dev.element_size() != gb or w_host.numel() * w_host.element_size() != wb:
        raise ValueError("host and device buffers of different sizes")
    carr, stride = _coeff_args(coeffs, steps)
    if ws is None:
        ws = workspace(Ms, compute, Ms[0].device)
    if record_event is not None and not record_event.cuda_event:
        record_event.record(stream)  # a torch event exists only once recorded
    ev = lambda e: ctypes.c_void_p(e.cuda_event if e is not None else None)  # noqa: E731
    st = lib().muon_step_host(
        _mats(Ws), _mats(Ms), _mats(Gs), _mats(Wo) if Wo is not None else None, len(Ws),
        float(mu), float(lr), int(steps), carr, stride, float(eps), _COMPUTE[compute],
        ctypes.c_void_p(ws.data_ptr()), ws.numel(), ctypes.c_void_p(g_host.data_ptr()),
        ctypes.c_void_p(g_dev.data_ptr()), gb, ctypes.c_void_p(w_host.data_ptr()),
        ctypes.c_void_p(w_dev.data_ptr()), wb, _stream(stream), ev(wait_event), ev(record_event))
    _abi.check("muon_step_host", st)


class PreparedCall:
    """A library call whose arguments were marshalled once: calling the object repeats the
    call with the same tensors (which must keep their storage), scalars and stream. For
    training loops whose step is short enough that building the arguments on the host each
    time would cost more than the GPU work."""

    def __init__(self, name, args, keep):
        self._fn = getattr(lib(), name)
        self._name = name
        self._args = args
        self._keep = keep  # the tensors and ctypes objects the arguments point into

    def __call__(self):
        _abi.check(self._name, self._fn(*self._args))


def sign_muon_step(W, M, G, words, vote, mu, lr, steps=5, coeffs=QUINTIC, eps=1e-7,
                   compute="bf16", ws=None, stream=None, prepare=False):
    """One whole Sign-Muon step: momentum of every worker, Newton-Schulz with the packed
    signs into words[m] (int32 tensor [W_n][stride]), the majority vote into `vote` and
    W <- W - lr * vote; the same results as the four separate calls. With prepare=True the
    call is not made: a PreparedCall that makes it (on `stream`, or the stream current now)
    is returned."""
    Ms, Gs = _as_list(M), _as_list(G)
    if len(Ms) != len(Gs) or words.dim() != 2 or words.shape[0] != len(Ms) or \
            words.stride(1) != 1 or words.dtype != torch.int32:
        raise ValueError("need one M and G per worker and int32 words [W_n][stride]")
    carr, stride = _coeff_args(coeffs, steps)
    if ws is None:
        ws = workspace(Ms, compute, Ms[0].device)
    wm, ma, ga = _mat(W), _mats(Ms), _mats(Gs)
    args = (ctypes.byref(wm), ma, ga, len(Ms), ctypes.c_void_p(words.data_ptr()), words.stride(0),
            ctypes.c_void_p(vote.data_ptr()), float(mu), float(lr), int(steps), carr, stride,
            float(eps), _COMPUTE[compute], ctypes.c_void_p(ws.data_ptr()), ws.numel(),
            _stream(stream))
    if prepare:
        return PreparedCall("sign_muon_step", args, (W, Ms, Gs, words, vote, ws, wm, ma, ga, carr))
    _abi.check("sign_muon_step", lib().sign_muon_step(*args))


def _coeff_args(coeffs, steps):
    co = list(coeffs)
    if len(co) == 3 and not isinstance(co[0], (list, tuple)):
        flat, stride = [float(c) for c in co], 0
    else:
        if len(co) != steps:
            raise ValueError("need one coefficient triple per step")
        flat, stride = [float(c) for t in co for c in t], 3
    return (ctypes.c_float * len(flat))(*flat), stride


def ns_blockwise_workspace_bytes(X, block, compute="bf16"):
    Xs = _as_list(X)
    arr = (_abi.MaoMat * len(Xs))()
    for i, x in enumerate(Xs):
        shape = x.shape if hasattr(x, "shape") else x
        arr[i] = _abi.MaoMat(None, shape[0], shape[1], shape[1], _abi.MAO_F32, 0)
    n = lib().ns_blockwise_workspace_bytes(arr, len(Xs), int(block[0]), int(block[1]),
                                           _COMPUTE[compute])
    if n == 0:
        raise ValueError("invalid shapes or block for ns_blockwise_workspace_bytes")
    return int(n)


def ns_orthogonalize_blockwise(inp, out, block, steps=5, coeffs=QUINTIC, eps=1e-7,
                               compute="bf16", ws=None, stream=None):
    """Newton–Schulz of every (block[0] x block[1]) block of each input on its own."""
    ins, outs = _as_list(inp), _as_list(out)
    carr, stride = _coeff_args(coeffs, steps)
    if ws is None:
        n = ns_blockwise_workspace_bytes(ins, block, compute)
        ws = torch.empty(n, dtype=torch.uint8, device=ins[0].device)
    st = lib().ns_orthogonalize_blockwise(
        _mats(ins), _mats(outs), len(ins), int(block[0]), int(block[1]), int(steps), carr, stride,
        float(eps), _COMPUTE[compute], ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(stream))
    _abi.check("ns_orthogonalize_blockwise", st)


def packed_words(rows, cols):
    return (rows * cols + 31) // 32


def sign_pack_bits(U, bits=None, stream=None):
    if bits is None:
        bits = torch.empty(packed_words(*U.shape), dtype=torch.int32, device=U.device)
    st = lib().sign_pack_bits(ctypes.byref(_mat(U)), ctypes.c_void_p(bits.data_ptr()), _stream(stream))
    _abi.check("sign_pack_bits", st)
    return bits


def majority_vote_packed(bits, nbits, vote=None, stream=None):
    """bits: int32 tensor [W_n][stride] of packed worker signs; returns the packed vote."""
    if bits.dim() != 2 or bits.stride(1) != 1:
        raise ValueError("bits must be [n_workers][stride] with unit stride")
    if vote is None:
        vote = torch.empty((nbits + 31) // 32, dtype=torch.int32, device=bits.device)
    st = lib().majority_vote_packed(ctypes.c_void_p(bits.data_ptr()), bits.shape[0], bits.stride(0),
                                    int(nbits), ctypes.c_void_p(vote.data_ptr()), _stream(stream))
    _abi.check("majority_vote_packed", st)
    return vote


def sign_int8(U, s=None, stream=None):
    """int8 signs of U (-1 where U < 0, else +1), row-major R x C."""
    if s is None:
        s = torch.empty(U.shape, dtype=torch.int8, device=U.device)
    st = lib().sign_int8(ctypes.byref(_mat(U)), ctypes.c_void_p(s.data_ptr()), _stream(stream))
    _abi.check("sign_int8", st)
    return s


def majority_vote_int8(s, n, sum=None, s_bar=None, vote=None, stream=None):
    """Integer SUM of workers' int8 signs, then the threshold vote.

    s: int8 tensor [W_n][stride] (stride >= n, unit inner stride). Each of sum / s_bar
    (int8, n entries) and vote (int32, ceil(n/32) words) is a tensor to fill, True to
    allocate, or None to skip. Returns (sum, s_bar, vote).
    """
    if s.dim() != 2 or s.stride(1) != 1 or s.dtype != torch.int8:
        raise ValueError("s must be an int8 [n_workers][stride] tensor with unit stride")

    def alloc(x, count, dt):
        if x is True:
            return torch.empty(count, dtype=dt, device=s.device)
        return x if x is not None and x is not False else None

    sum = alloc(sum, n, torch.int8)
    s_bar = alloc(s_bar, n, torch.int8)
    vote = alloc(vote, packed_words(1, n), torch.int32)
    ptr = lambda x: ctypes.c_void_p(x.data_ptr() if x is not None else None)  # noqa: E731
    st = lib().majority_vote_int8(ptr(s), s.shape[0], s.stride(0), int(n), ptr(sum), ptr(s_bar),
                                  ptr(vote), _stream(stream))
    _abi.check("majority_vote_int8", st)
    return sum, s_bar, vote


def apply_update(W, lr, vote=None, U=None, stream=None):
    """W <- W - lr*D with D the packed vote (+1/-1) or the matrix U."""
    Ws = _as_list(W)
    varr = None
    uarr = None
    if vote is not None:
        vs = _as_list(vote)
        varr = (ctypes.c_void_p * len(vs))(*[v.data_ptr() for v in vs])
    if U is not None:
        uarr = _mats(_as_list(U))
    st = lib().apply_update(_mats(Ws), varr, uarr, len(Ws), float(lr), _stream(stream))
    _abi.check("apply_update", st)


def dion_workspace_bytes(shapes, rank):
    """Workspace bytes of one dion_step call over matrices of the given (m, n) shapes."""
    arr = (_abi.MaoMat * len(shapes))()
    for i, sh in enumerate(shapes):
        arr[i] = _abi.MaoMat(None, sh[0], sh[1], sh[1], _abi.MAO_F32, 0)
    n = lib().dion_workspace_bytes(arr, len(shapes), int(rank))
    if n == 0:
        raise ValueError("invalid shapes or rank for dion_workspace_bytes")
    return int(n)


def _q_mat(q):
    if not q.is_cuda or q.dtype != torch.float32 or q.dim() != 2 or q.stride(1) != 1:
        raise ValueError("Q must be a 2-D float32 CUDA tensor with unit column stride")
    return _abi.MaoMat(q.data_ptr(), q.shape[0], q.shape[1], max(q.stride(0), q.shape[1]),
                       _abi.MAO_F32, 0)


def dion_step(X, M, G, Q, mu, lr, P_out=None, ws=None, stream=None, X_out=None):
    """One Dion step for each (X, M, G, Q), any mix of shapes, one rank: X and M updated in
    place, Q replaced by the new right factor (n x r, float32). P_out: optional float32
    tensors (m x r, contiguous) receiving the final P. X_out: optional tensors of X's shapes
    and dtypes receiving the new X (X is then only read)."""
    Xs, Ms, Gs, Qs = _as_list(X), _as_list(M), _as_list(G), _as_list(Q)
    rank = Qs[0].shape[1]
    if any(q.shape[1] != rank for q in Qs):
        raise ValueError("one rank per call")
    qarr = (_abi.MaoMat * len(Qs))()
    for k, q in enumerate(Qs):
        qarr[k] = _q_mat(q)
    parr = None
    if P_out is not None:
        Ps = _as_list(P_out)
        parr = (ctypes.c_void_p * len(Ps))(*[p.data_ptr() if p is not None else None for p in Ps])
    if ws is None:
        ws = torch.empty(dion_workspace_bytes([tuple(x.shape) for x in Xs], rank),
                         dtype=torch.uint8, device=Xs[0].device)
    xo = None
    if X_out is not None:
        Xos = _as_list(X_out)
        if len(Xos) != len(Xs):
            raise ValueError("X_out needs one tensor per X")
        xo = _mats(Xos)
    st = lib().dion_step(_mats(Xs), _mats(Ms), _mats(Gs), qarr, xo, parr, len(Xs), int(rank),
                         float(mu), float(lr), _abi.MAO_BF16, ctypes.c_void_p(ws.data_ptr()),
                         ws.numel(), _stream(stream))
    _abi.check("dion_step", st)


# ---------------------------------------------------------------- expert layers

_BLOCKS = {"row": _abi.MAO_BLOCKS_ROW, "col": _abi.MAO_BLOCKS_COL, "tile": _abi.MAO_BLOCKS_TILE}
_KINDS = {"row": ("row",), "col": ("col",), "tile": ("tile",), "both": ("row", "col")}
_FORM = {"nt": _abi.MAO_NT, "nn": _abi.MAO_NN, "tn": _abi.MAO_TN}
_SCORE = {"softmax": _abi.MAO_SCORE_SOFTMAX, "sigmoid": _abi.MAO_SCORE_SIGMOID}
_GROUP_SCORE = {"max": _abi.MAO_GROUP_MAX, "top2": _abi.MAO_GROUP_TOP2}


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream`: allocated there, so that its memory is reused
    only after that stream's work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_strided(shape, strides, dtype, device, stream):
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


_FLOATS = {torch.float32: _abi.MAO_F32, torch.bfloat16: _abi.MAO_BF16}


def _desc(t, dims=2):
    """_mat of a float32 or bfloat16 matrix, with as few calls as it takes; with dims = 3 of the
    first of stacked matrices."""
    shape, st = t.shape, t.stride()
    if len(shape) != dims or (st[-1] != 1 and shape[-1] > 1) or not t.is_cuda:
        raise ValueError("expected a %d-D CUDA tensor with unit column stride" % dims)
    rows, cols, ld = shape[-2], shape[-1], st[-2]
    if ld < cols:
        if rows > 1:
            raise ValueError("expected a tensor whose rows do not overlap")
        ld = cols
    dt = _FLOATS.get(t.dtype)
    if dt is None:
        raise ValueError("dtype must be float32 or bfloat16")
    return _abi.MaoMat(t.data_ptr(), rows, cols, ld, dt, 0)


def _raw_stream(stream, *operands):
    """The handle of a call's stream, by default the current one. The library launches on the
    current device, so its operands (None: not given) and its stream have to be there. (These calls
    may be as short as a kernel launch, so the handle is fetched without a Stream object.)"""
    device = torch._C._cuda_getDevice()
    for t in operands:
        if t is not None and t.get_device() != device:
            raise ValueError("expected tensors of the current CUDA device, %d" % device)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError("expected a stream of the current CUDA device, %d" % device)
    return stream.cuda_stream


def _dense_ptr(t, dtype, shape, name):
    """Device pointer of a contiguous tensor of the given type and shape (None: NULL)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA tensor of shape %s"
                         % (name, dtype, tuple(shape)))
    return t.data_ptr()


def _out(t, shape, dtype, name, like, stream):
    """An output of a call: t, checked, or a new tensor; and its device pointer."""
    if t is not None:
        return t, _dense_ptr(t, dtype, shape, name)
    t = torch.empty(shape, dtype=dtype, device=like.device) if stream is None else \
        _empty(shape, dtype, like.device, stream)
    return t, t.data_ptr()


def _buffer(ws):
    """Device pointer and bytes of a caller's workspace."""
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _scale_shape(rows, cols, blocks):
    br = 1 if blocks == "row" else 128
    bc = 1 if blocks == "col" else 128
    return -(-rows // br), -(-cols // bc)


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _fp8(codes, scales, blocks, name):
    """MaoFp8 of a code tensor [R, C] or [B, R, C] and its scale bytes."""
    shape, sshape = codes.shape, scales.shape
    if codes.dtype not in _CODES or scales.dtype != torch.uint8:
        raise ValueError("%s: codes are float8_e4m3fn and scales uint8 tensors" % name)
    if not codes.is_cuda or not scales.is_cuda or len(shape) not in (2, 3) or \
            len(sshape) != len(shape):
        raise ValueError("%s: CUDA tensors of two or three dimensions" % name)
    rows, cols = shape[-2], shape[-1]
    count = shape[0] if len(shape) == 3 else 1
    sr, sc = _scale_shape(rows, cols, blocks)
    if sshape[-2] != sr or sshape[-1] != sc or (len(shape) == 3 and sshape[0] != count):
        raise ValueError("%s: scales of shape %s do not fit %s blocks of %s"
                         % (name, tuple(sshape), blocks, tuple(shape)))
    st, sst = codes.stride(), scales.stride()
    if (st[-1] != 1 and cols > 1) or (sst[-1] != 1 and sc > 1):
        raise ValueError("%s: expected unit column stride" % name)
    # the row stride of a single row may be anything
    ld = st[-2] if rows > 1 else -(-cols // 16) * 16
    sld = sst[-2] if sr > 1 else sc
    if count > 1 and rows:
        if rows == 1:
            ld = st[0]
        if sr == 1:
            sld = sst[0]
        if st[0] != rows * ld or sst[0] != sr * sld:
            raise ValueError("%s: stacked matrices follow each other without gaps" % name)
    return _abi.MaoFp8(codes.data_ptr(), scales.data_ptr(), rows, cols, ld, sld, count,
                       _BLOCKS[blocks])


def fp8_quantize(X, blocks, rows=None, copies=1, out=None, stream=None):
    """Codes (float8_e4m3fn) and scale bytes of X in 8-bit floating point, with a
    power-of-two scale 2^(byte - 127) for each block of 128.

    X: a float32 or bfloat16 matrix [R, C], stacked matrices [B, R, C], or a list of B
    matrices of one shape. blocks: "row" (128 columns of a row), "col" (128 rows of a column),
    "tile" (128 x 128) or "both" (row and col, in one pass). Returns (codes, scales), or with
    "both" (row codes, row scales, col codes, col scales), stacked as X is; code rows are 16-byte
    aligned. rows: int32 tensor of source rows (one matrix X): row i of the result is row
    rows[i] // copies of X, or zeros where rows[i] < 0. out: a tuple of tensors to fill.
    """
    many = isinstance(X, (list, tuple))
    if many and not X:
        raise ValueError("no matrices")
    x0 = X[0] if many else X
    stacked = many or x0.dim() == 3
    if many:
        mats, batch, stride = _mats(list(X)), len(X), 0
        R, C = x0.shape
    elif stacked:
        batch, R, C = x0.shape
        if batch == 0:
            raise ValueError("no matrices")
        m = _desc(x0, 3)
        stride = x0.stride(0) if batch > 1 else 0
        if batch > 1 and stride < 1:
            raise ValueError("stacked matrices need a positive stride")
        mats = ctypes.byref(m)
    else:
        m = _desc(x0)
        mats, batch, stride = ctypes.byref(m), 1, 0
        R, C = m.rows, m.cols
    index, n_index = None, 0
    if rows is None:
        copies = 0
    else:
        if batch != 1:
            raise ValueError("rows go with a single matrix")
        if not 1 <= copies < 2 ** 31:
            raise ValueError("copies must be at least 1 and below 2^31")
        n_index = R = rows.numel()
        index = _dense_ptr(rows, torch.int32, rows.shape, "rows")
    kinds = _KINDS.get(blocks)
    if kinds is None:
        raise ValueError("blocks must be row, col, tile or both")
    desc = {}
    if out is None:
        out, wide = [], (C + 15) // 16 * 16
        for k in kinds:
            sr, sc = _scale_shape(R, C, k)
            size, ssize, strides = (R, C), (sr, sc), (wide, 1)
            if stacked:
                size, ssize, strides = (batch, R, C), (batch, sr, sc), (R * wide, wide, 1)
            if wide == C:
                codes, cp = _out(None, size, torch.float8_e4m3fn, "", x0, stream)
            else:  # rows start at multiples of 16 bytes
                codes = _empty_strided(size, strides, torch.float8_e4m3fn, x0.device, stream)
                cp = codes.data_ptr()
            scales, sp = _out(None, ssize, torch.uint8, "", x0, stream)
            desc[k] = ctypes.byref(_abi.MaoFp8(cp, sp, R, C, wide, sc, batch, _BLOCKS[k]))
            out += (codes, scales)
    else:
        if len(out) != 2 * len(kinds):
            raise ValueError("out needs codes and scales for each kind of blocks")
        for i, k in enumerate(kinds):
            desc[k] = ctypes.byref(_fp8(out[2 * i], out[2 * i + 1], k, k))
    st = lib().fp8_quantize(mats, batch, stride, index, n_index, copies, desc.get("row"),
                            desc.get("col"), desc.get("tile"),
                            _raw_stream(stream, rows, *(X if many else (X,)), *out))
    if st:
        _abi.check("fp8_quantize", st)
    return tuple(out)


def fp8_product(A, a_scales, B, b_scales, form, offsets=None, out=None, out_dtype=torch.bfloat16,
                accumulate=False, ws=None, stream=None):
    """Product of 8-bit matrices (fp8_quantize's codes and scales) with fp32 sums, over groups
    of rows.

    form "nt": out[t, n] = sum_k A[t, k] B[g, n, k]   A in row blocks, B in tiles
         "nn": out[t, k] = sum_n A[t, n] B[g, n, k]   A in row blocks, B in tiles
         "tn": out[g, n, k] = sum_t A[t, n] B[t, k]   A and B in column blocks
    offsets: int32 tensor of groups + 1 row numbers (expert_plan's; for "tn" multiples of
    128): g is the group of row t, and "tn" sums over the rows of group g. None: one group, and
    B may then be [N, K]. out: a float32 or bfloat16 tensor to fill, or with accumulate to add
    to; by default a new one of out_dtype. Rows without a group become zero. ws: a uint8
    buffer for products without groups whose sum is split (fp8_product_workspace_bytes);
    allocated when needed.
    """
    if form not in _FORM:
        raise ValueError("form must be nt, nn or tn")
    tn = form == "tn"
    if A.dim() != 2 or (tn and B.dim() != 2):
        raise ValueError("A (and for tn B) must be a matrix")
    a = _fp8(A, a_scales, "col" if tn else "row", "A")
    b = _fp8(B, b_scales, "col" if tn else "tile", "B")
    if offsets is None:
        groups, off = 1, None
    else:
        groups = offsets.numel() - 1
        off = _dense_ptr(offsets, torch.int32, (groups + 1,), "offsets")
    shape = (groups, a.cols, b.cols) if tn else (a.rows, b.rows if form == "nt" else b.cols)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if out_dtype not in _FLOATS:
            raise ValueError("out_dtype must be float32 or bfloat16")
        out, op = _out(None, shape, out_dtype, "", A, stream)
        d = _abi.MaoMat(op, groups * a.cols if tn else a.rows, shape[-1], shape[-1],
                        _FLOATS[out_dtype], 0)
    else:
        if tuple(out.shape) != shape and not (tn and groups == 1 and tuple(out.shape) == shape[1:]):
            raise ValueError("out must have shape %s" % (shape,))
        flat = out
        if out.dim() == 3:
            if groups > 1 and out.stride(0) != a.cols * out.stride(1):
                raise ValueError("the groups' matrices follow each other without gaps")
            flat = out.as_strided((groups * a.cols, b.cols), (out.stride(1), out.stride(2)))
        d = _desc(flat)
    ra, rb = ctypes.byref(a), ctypes.byref(b)
    wptr, wbytes = None, 0
    if ws is not None:
        wptr, wbytes = _buffer(ws)
    elif off is None:
        wbytes = lib().fp8_product_workspace_bytes(ra, rb, _FORM[form])
        if wbytes:
            ws, wptr = _out(None, wbytes, torch.uint8, "", A, stream)
    st = lib().fp8_product(ra, rb, ctypes.byref(d), _FORM[form], off, groups,
                           bool(accumulate), wptr, wbytes,
                           _raw_stream(stream, A, a_scales, B, b_scales, offsets, out, ws))
    if st:
        _abi.check("fp8_product", st)
    return out


def expert_route(logits, top_k, score="softmax", bias=None, groups=1, keep_groups=None,
                 group_score="top2", renorm=True, scale=1.0, weights=None, ids=None, stream=None):
    """The top_k experts of each token: (weights float32 [T, top_k], ids int32 [T, top_k]).

    score: "softmax" or "sigmoid" of the logits [T, E] (float32 or bfloat16). bias: float32 [E],
    added to the scores for choosing only. groups, keep_groups, group_score ("max" or
    "top2"): only experts of the best runs of E / groups are chosen. renorm: the chosen scores
    are divided by their sum. Masked experts (logit -inf) are never chosen; ids -1 with
    weight 0 fill the places that are left.
    """
    kind, run = _SCORE.get(score), _GROUP_SCORE.get(group_score)
    if kind is None or run is None:
        raise ValueError("score must be softmax or sigmoid, group_score max or top2")
    m = _desc(logits)
    shape = (m.rows, top_k)
    weights, wp = _out(weights, shape, torch.float32, "weights", logits, stream)
    ids, ip = _out(ids, shape, torch.int32, "ids", logits, stream)
    st = lib().expert_route(
        ctypes.byref(m), _dense_ptr(bias, torch.float32, (m.cols,), "bias"), top_k, kind,
        groups, groups if keep_groups is None else keep_groups, run,
        bool(renorm), scale, wp, ip, _raw_stream(stream, logits, bias, weights, ids))
    if st:
        _abi.check("expert_route", st)
    return weights, ids


def expert_route_backward(logits, ids, dweights, score="softmax", renorm=True, scale=1.0,
                          dlogits=None, stream=None):
    """Gradient of expert_route's weights with respect to the logits (dlogits: of the logits'
    shape and dtype unless given)."""
    kind = _SCORE.get(score)
    if kind is None:
        raise ValueError("score must be softmax or sigmoid")
    m = _desc(logits)
    shape = ids.shape
    if len(shape) != 2 or shape[0] != m.rows:
        raise ValueError("ids must be [T, top_k]")
    if dlogits is None:
        dlogits, dp = _out(None, logits.shape, logits.dtype, "", logits, stream)
        d = _abi.MaoMat(dp, m.rows, m.cols, m.cols, m.dtype, 0)
    else:
        d = _desc(dlogits)
    st = lib().expert_route_backward(
        ctypes.byref(m), _dense_ptr(ids, torch.int32, shape, "ids"),
        _dense_ptr(dweights, torch.float32, shape, "dweights"), shape[1], kind,
        bool(renorm), scale, ctypes.byref(d), _raw_stream(stream, logits, ids, dweights, dlogits))
    if st:
        _abi.check("expert_route_backward", st)
    return dlogits


def expert_rows(n, experts):
    """Rows that always hold n copies in the experts' padded runs."""
    return int(lib().expert_rows(int(n), int(experts)))


class ExpertPlan:
    """Where the tokens' copies go (expert_plan): counts [E], offsets [E + 1], row_of [T, k]
    (-1: dropped) and slot_of [rows] (the copy t * k + j in each row, -1 in padding rows)."""

    __slots__ = ("counts", "offsets", "row_of", "slot_of")

    def __init__(self, counts, offsets, row_of, slot_of):
        self.counts, self.offsets, self.row_of, self.slot_of = counts, offsets, row_of, slot_of


@functools.lru_cache(maxsize=256)
def _plan_sizes(n, experts):
    """(rows, workspace bytes or 0 where none is needed) of a plan."""
    nb = lib().expert_plan_workspace_bytes(n, experts)
    if nb == 0:
        raise ValueError("expert_plan takes up to 2^24 copies and 1 to 1024 experts")
    return expert_rows(n, experts), nb if n > 4096 else 0


def expert_plan(ids, experts, ws=None, stream=None):
    """Places of the copies ids [T, top_k] (int32; entries outside 0 .. experts - 1 are dropped):
    each expert's copies, in the order of the tokens, in a run of rows that starts at a
    multiple of 128. Returns an ExpertPlan."""
    n, experts = ids.numel(), int(experts)
    p_ids = _dense_ptr(ids, torch.int32, ids.shape, "ids")
    rows, nb = _plan_sizes(n, experts)
    i32 = torch.int32
    counts, p_counts = _out(None, experts, i32, "", ids, stream)
    offsets, p_off = _out(None, experts + 1, i32, "", ids, stream)
    row_of, p_row = _out(None, ids.shape, i32, "", ids, stream)
    slot_of, p_slot = _out(None, rows, i32, "", ids, stream)
    wptr = None
    if ws is not None:
        wptr, nb = _buffer(ws)
    elif nb:
        ws, wptr = _out(None, nb, torch.uint8, "", ids, stream)
    st = lib().expert_plan(p_ids, n, experts, p_counts, p_off, p_row, p_slot, rows, wptr, nb,
                           _raw_stream(stream, ids, ws))
    if st:
        _abi.check("expert_plan", st)
    return ExpertPlan(counts, offsets, row_of, slot_of)


def expert_combine(Z, row_of, weights=None, out=None, stream=None):
    """y[t] = sum_j weights[t, j] Z[row_of[t, j]] (entries below 0 are skipped; weights None:
    all 1), summed in fp32; out: of Z's dtype unless given."""
    shape = row_of.shape
    T, k = shape
    z = _desc(Z)
    if out is None:
        out, yp = _out(None, (T, z.cols), Z.dtype, "", Z, stream)
        y = _abi.MaoMat(yp, T, z.cols, z.cols, z.dtype, 0)
    else:
        y = _desc(out)
    st = lib().expert_combine(
        ctypes.byref(z), _dense_ptr(row_of, torch.int32, shape, "row_of"),
        _dense_ptr(weights, torch.float32, shape, "weights"), T, k, ctypes.byref(y),
        _raw_stream(stream, Z, row_of, weights, out))
    if st:
        _abi.check("expert_combine", st)
    return out


def expert_combine_backward(dY, Z, row_of, slot_of, weights=None, dZ=None, dweights=None,
                            stream=None):
    """Gradients (dZ of Z's shape and dtype unless given, dweights float32 [T, k]) of
    expert_combine."""
    shape = row_of.shape
    T, k = shape
    dy, z = _desc(dY), _desc(Z)
    if dy.rows != T:
        raise ValueError("dY needs one row per token")
    if dZ is None:
        dZ, dp = _out(None, Z.shape, Z.dtype, "", Z, stream)
        d = _abi.MaoMat(dp, z.rows, z.cols, z.cols, z.dtype, 0)
    else:
        d = _desc(dZ)
    dweights, wp = _out(dweights, shape, torch.float32, "dweights", Z, stream)
    st = lib().expert_combine_backward(
        ctypes.byref(dy), ctypes.byref(z), _dense_ptr(row_of, torch.int32, shape, "row_of"),
        _dense_ptr(slot_of, torch.int32, (z.rows,), "slot_of"),
        _dense_ptr(weights, torch.float32, shape, "weights"), k, ctypes.byref(d), wp,
        _raw_stream(stream, dY, Z, row_of, slot_of, weights, dZ, dweights))
    if st:
        _abi.check("expert_combine_backward", st)
    return dZ, dweights


def set_wait_limit(ns):
    """Bound (ns) of every device-side wait of the tensor-core kernels; 0 gives up at once."""
    lib().mao_set_wait_limit(int(ns))


def get_wait_limit():
    return int(lib().mao_get_wait_limit())


def sync_status(stream=None):
    st = lib().mao_sync_status(_stream(stream))
    _abi.check("mao_sync_status", st)


def launch_count():
    """Kernels libmao has launched in this process."""
    return int(lib().mao_launch_count())


PROFILE_TAGS = {0: "tc", 1: "dion_setup", 2: "dion_stage", 3: "dion_gram", 4: "dion_chol",
                5: "dion_split", 6: "dion_norm", 7: "ns_small"}


def profile_begin(max_launches):
    """Record CUDA events around each tensor-core product launch and each Dion CUDA-core
    kernel launch (benchmarking)."""
    _abi.check("mao_profile_begin", lib().mao_profile_begin(int(max_launches)))


def profile_end(max_out=1 << 20):
    """Stop recording; returns the per-launch durations in milliseconds."""
    buf = (ctypes.c_float * max_out)()
    n = lib().mao_profile_end(buf, max_out)
    if n < 0:
        raise MaoError("mao_profile_end", _abi.MAO_ERR_CUDA)
    return [buf[i] for i in range(min(n, max_out))]


def profile_end_tagged(max_out=1 << 20):
    """Stop recording; returns (milliseconds, tag name) per recorded launch."""
    buf = (ctypes.c_float * max_out)()
    tags = (ctypes.c_int32 * max_out)()
    n = lib().mao_profile_end_tagged(buf, tags, max_out)
    if n < 0:
        raise MaoError("mao_profile_end_tagged", _abi.MAO_ERR_CUDA)
    return [(buf[i], PROFILE_TAGS.get(tags[i], str(tags[i]))) for i in range(min(n, max_out))]


def profile_span_begin(max_spans):
    """Record one CUDA event pair around each Newton–Schulz call's run of tensor-core products
    (benchmarking; the products keep overlapping one another's set-up)."""
    _abi.check("mao_profile_span_begin", lib().mao_profile_span_begin(int(max_spans)))


def profile_span_end(max_out=1 << 16):
    """Stop recording; returns the recorded spans in milliseconds."""
    buf = (ctypes.c_float * max_out)()
    n = lib().mao_profile_span_end(buf, max_out)
    if n < 0:
        raise MaoError("mao_profile_span_end", _abi.MAO_ERR_CUDA)
    return [buf[i] for i in range(min(n, max_out))]
