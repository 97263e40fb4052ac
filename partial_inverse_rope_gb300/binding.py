"""ctypes binding of ``libinvrope.so`` (the C ABI declared in ``include/invrope.h``,
``include/latent_attn.h``, ``include/kv_pages.h`` and ``include/rope.h``).

Argument marshalling only: each function checks that torch tensors have the
dtype / device / layout the C ABI expects, allocates outputs with torch when
the caller passes none, and forwards raw device pointers, sizes and the
current CUDA stream. All arithmetic runs in the library's kernels. There is no
fallback: if the library is not built, the first call raises.

Ordinary calls of the serving operators (tensors as they are asked for, outputs
allocated, or given to a step of pages, the current stream) go through a compiled
module, ``_calls.so``, which leaves all others to the functions here.
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

# INVROPE_LIBRARY selects another build of the same library (e.g. the
# debug-bounds build, libinvrope_debug.so); it must export the same symbols.
_LIB_PATH = os.environ.get("INVROPE_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                             "libinvrope.so")
_lib = None
_calls = None  # the compiled calls, once the library is loaded

INVROPE_OK = 0
INVROPE_ERR_INVALID_ARG = 1
INVROPE_ERR_UNSUPPORTED = 2
INVROPE_ERR_WORKSPACE = 3
INVROPE_ERR_CUDA = 4
INVROPE_ERR_DEVICE = 5

# name -> (restype, argtypes); mirrors the headers under include/
_SIGNATURES = {
    "invrope_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "invrope_last_cuda_error": (ctypes.c_int, []),
    "invrope_postmix_fwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "invrope_postmix_bwd_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "invrope_postmix_bwd": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "invrope_postmix_bwd_noalloc": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "invrope_postmix_fwd_ex": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "invrope_postmix_bwd_ex": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "kv_idx_local_to_global": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "kv_idx_local_to_global_i64": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "invrope_take_device_fault": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int)]),
    "invrope_watchdog_selftest": (ctypes.c_int, [ctypes.c_int64, ctypes.POINTER(ctypes.c_int)]),
    "invrope_debug_occupy_next_slot": (ctypes.c_int, [ctypes.c_int, ctypes.c_ulonglong]),
    "kv_latent_row_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "kv_latent_write": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "kv_latent_read": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "latent_attn_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "invrope_latent_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "latent_attn_decode": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "latent_attn_sparse": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p]),
    "kv_pages_advance": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]),
    "kv_idx_local_to_slots": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
        ctypes.c_void_p]),
    "rope_freqs": (ctypes.c_int, [
        ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
        ctypes.c_void_p, ctypes.c_void_p]),
    "rope_apply": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
        ctypes.c_double, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
}

KV_LATENT_BF16 = 0
KV_LATENT_E4M3 = 1
KV_LATENT_E2M1 = 4

ROPE_SCALE_NONE = 0
ROPE_SCALE_LINEAR = 1
ROPE_SCALE_NTK = 2
ROPE_SCALE_YARN = 3
ROPE_MAX_TENSORS = 4

INVROPE_WATCHDOG_SELFTEST_CODE = 0x60A
INVROPE_FAULT_SCHED_BUSY_FWD = 0x5C1
INVROPE_FAULT_SCHED_BUSY_REMAP = 0x5C2
INVROPE_FAULT_SCHED_BUSY_BWD = 0x5C3


class InvropeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().invrope_status_string(status).decode()
        if status == INVROPE_ERR_CUDA:
            msg += f" (cudaError {lib().invrope_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load ``libinvrope.so`` once; raise if it has not been built."""
    global _lib, _calls
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -m partial_inverse_rope_gb300.build` (there is no CPU fallback)")
        handle = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
        _calls = _compiled_calls(handle)
    return _lib


def _compiled_calls(handle):
    """The module of ``csrc/calls.cpp`` over the library's functions; None where it was not built."""
    try:
        from . import _calls as calls
    except ImportError:
        return None
    names = ("kv_pages_advance", "kv_idx_local_to_slots", "rope_apply", "kv_latent_row_bytes", "kv_latent_write",
             "kv_latent_read", "invrope_latent_workspace_bytes", "latent_attn_decode", "latent_attn_sparse")
    calls.bind(*[ctypes.cast(getattr(handle, n), ctypes.c_void_p).value for n in names])
    return calls


def _made(got, what):
    """What a compiled call gave, once it has given something: its result, or its status as an error."""
    if type(got) is int:
        _check(got, what)
    return got


def _check(status: int, what: str):
    if status != INVROPE_OK:
        raise InvropeError(status, what)


def _stream_handle(device, stream):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _empty(shape, dtype, device, stream):
    """An uninitialised tensor that belongs to ``stream`` (None: the current
    one): its memory is free on the stream the kernels write it on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def invrope_postmix_fwd(O, M, pos0: int, nope: int, pe: int, theta: float = 10000.0,
                        Y=None, stream=None):
    """``Y[s,g,:] = sum_h M[g,h] invrope_{pos0+s}(O[s,h,:])``; returns ``Y`` (bf16)."""
    _need(O, "O", torch.bfloat16, 3)
    _need(M, "M", torch.float32, 2)
    sq, nh, d = O.shape
    if tuple(M.shape) != (nh, nh):
        raise ValueError(f"M must be [{nh}, {nh}]")
    if Y is None:
        Y = torch.empty_like(O)
    else:
        _need(Y, "Y", torch.bfloat16, 3)
        if Y.shape != O.shape:
            raise ValueError("Y must have O's shape")
    st = lib().invrope_postmix_fwd(O.data_ptr(), M.data_ptr(), Y.data_ptr(), sq, nh, nope, pe,
                                   int(pos0), float(theta), _stream_handle(O.device, stream))
    _check(st, "invrope_postmix_fwd")
    return Y


def invrope_postmix_bwd_workspace_bytes(sq: int, nh: int, nope: int, pe: int) -> int:
    """Workspace bytes the backward needs on the current device (0 if the shape is invalid)."""
    return int(lib().invrope_postmix_bwd_workspace_bytes(int(sq), int(nh), int(nope), int(pe)))


def invrope_postmix_bwd(dY, O, M, pos0: int, nope: int, pe: int, theta: float = 10000.0,
                        dO=None, dM=None, workspace=None, stream=None):
    """Backward of the fused postmix; returns ``(dO bf16, dM fp32)``."""
    _need(dY, "dY", torch.bfloat16, 3)
    _need(O, "O", torch.bfloat16, 3)
    _need(M, "M", torch.float32, 2)
    sq, nh, d = O.shape
    if dY.shape != O.shape or tuple(M.shape) != (nh, nh):
        raise ValueError("dY must match O and M must be [nh, nh]")
    if dO is None:
        dO = torch.empty_like(O)
    if dM is None:
        dM = torch.empty(nh, nh, dtype=torch.float32, device=O.device)
    _need(dO, "dO", torch.bfloat16, 3)
    _need(dM, "dM", torch.float32, 2)
    if workspace is None:
        nbytes = invrope_postmix_bwd_workspace_bytes(sq, nh, nope, pe)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=O.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().invrope_postmix_bwd(dY.data_ptr(), O.data_ptr(), M.data_ptr(), dO.data_ptr(),
                                   dM.data_ptr(), workspace.data_ptr(), ws_bytes, sq, nh, nope, pe,
                                   int(pos0), float(theta), _stream_handle(O.device, stream))
    _check(st, "invrope_postmix_bwd")
    return dO, dM


def _mix_and_positions(M, positions, sq, nh, group_size, device):
    """Check the [nh/gs, gs, gs] mix and the optional int32 [sq] positions."""
    gs = nh if group_size is None else int(group_size)
    if gs < 1 or nh % gs:
        raise ValueError("group_size must divide nh")
    want = (nh // gs, gs, gs) if group_size is not None else (nh, nh)
    _need(M, "M", torch.float32, len(want))
    if tuple(M.shape) != want:
        raise ValueError(f"M must be {list(want)}")
    if positions is not None:
        _need(positions, "positions", torch.int32, 1)
        if positions.shape[0] != sq or positions.device != device:
            raise ValueError("positions must be int32 [sq] on the tensors' device")
    return gs, (positions.data_ptr() if positions is not None else None)


def invrope_postmix_fwd_ex(O, M, nope: int, pe: int, positions=None, pos0: int = 0,
                           theta: float = 10000.0, group_size=None, Y=None, stream=None):
    """Forward with an optional grouped mix (``M`` = [nh/gs, gs, gs] when
    ``group_size`` is given) and optional int32 per-row ``positions`` (row s
    sits at ``pos0 + positions[s]``, else ``pos0 + s``); returns ``Y``."""
    _need(O, "O", torch.bfloat16, 3)
    sq, nh, d = O.shape
    gs, pos_ptr = _mix_and_positions(M, positions, sq, nh, group_size, O.device)
    if Y is None:
        Y = torch.empty_like(O)
    else:
        _need(Y, "Y", torch.bfloat16, 3)
        if Y.shape != O.shape:
            raise ValueError("Y must have O's shape")
    st = lib().invrope_postmix_fwd_ex(O.data_ptr(), M.data_ptr(), Y.data_ptr(), sq, nh, gs, nope, pe,
                                      pos_ptr, int(pos0), float(theta), _stream_handle(O.device, stream))
    _check(st, "invrope_postmix_fwd_ex")
    return Y


def invrope_postmix_bwd_ex(dY, O, M, nope: int, pe: int, positions=None, pos0: int = 0,
                           theta: float = 10000.0, group_size=None, dO=None, dM=None,
                           workspace=None, stream=None):
    """Backward of :func:`invrope_postmix_fwd_ex`; returns ``(dO bf16, dM fp32)``
    with ``dM`` shaped like ``M``."""
    _need(dY, "dY", torch.bfloat16, 3)
    _need(O, "O", torch.bfloat16, 3)
    sq, nh, d = O.shape
    if dY.shape != O.shape:
        raise ValueError("dY must match O")
    gs, pos_ptr = _mix_and_positions(M, positions, sq, nh, group_size, O.device)
    if dO is None:
        dO = torch.empty_like(O)
    if dM is None:
        dM = torch.empty(M.shape, dtype=torch.float32, device=O.device)
    _need(dO, "dO", torch.bfloat16, 3)
    _need(dM, "dM", torch.float32, M.dim())
    if dM.shape != M.shape:
        raise ValueError("dM must have M's shape")
    if workspace is None:
        nbytes = invrope_postmix_bwd_workspace_bytes(sq, nh, nope, pe)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=O.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().invrope_postmix_bwd_ex(dY.data_ptr(), O.data_ptr(), M.data_ptr(), dO.data_ptr(),
                                      dM.data_ptr(), workspace.data_ptr(), ws_bytes, sq, nh, gs, nope, pe,
                                      pos_ptr, int(pos0), float(theta), _stream_handle(O.device, stream))
    _check(st, "invrope_postmix_bwd_ex")
    return dO, dM


def invrope_postmix_bwd_noalloc(dY, O, M, pos0: int, nope: int, pe: int, dO, dM,
                                theta: float = 10000.0, stream=None):
    """Backward without a workspace, for callers that may not allocate device
    memory on their call path: the library's own fixed scratch array
    (``INVROPE_NOALLOC_SCRATCH_BYTES``) holds the dM partials. ``dO`` and
    ``dM`` must be given (this wrapper allocates nothing either). Calls that
    overlap on the GPU share that array and must be ordered."""
    _need(dY, "dY", torch.bfloat16, 3)
    _need(O, "O", torch.bfloat16, 3)
    _need(M, "M", torch.float32, 2)
    _need(dO, "dO", torch.bfloat16, 3)
    _need(dM, "dM", torch.float32, 2)
    sq, nh, d = O.shape
    if dY.shape != O.shape or dO.shape != O.shape or tuple(M.shape) != (nh, nh) \
            or tuple(dM.shape) != (nh, nh):
        raise ValueError("dY/dO must match O; M and dM must be [nh, nh]")
    st = lib().invrope_postmix_bwd_noalloc(dY.data_ptr(), O.data_ptr(), M.data_ptr(), dO.data_ptr(),
                                           dM.data_ptr(), sq, nh, nope, pe, int(pos0), float(theta),
                                           _stream_handle(O.device, stream))
    _check(st, "invrope_postmix_bwd_noalloc")
    return dO, dM


def kv_idx_local_to_global(idx, sq: int, seqlen_kv: int, out=None, stream=None):
    """``out = idx < 0 ? idx : idx + (row // sq) * seqlen_kv`` on an int32 ``[rows, topk]`` table."""
    _need(idx, "idx", torch.int32, 2)
    rows, topk = idx.shape
    if out is None:
        out = torch.empty_like(idx)
    else:
        _need(out, "out", torch.int32, 2)
        if out.shape != idx.shape:
            raise ValueError("out must match idx")
    st = lib().kv_idx_local_to_global(idx.data_ptr(), out.data_ptr(), rows, topk, int(sq),
                                      int(seqlen_kv), _stream_handle(idx.device, stream))
    _check(st, "kv_idx_local_to_global")
    return out


def kv_idx_local_to_global_i64(idx, sq: int, seqlen_kv: int, out=None, stream=None):
    """The same remap on an int64 ``[rows, topk]`` table (64-bit wrap)."""
    _need(idx, "idx", torch.int64, 2)
    rows, topk = idx.shape
    if out is None:
        out = torch.empty_like(idx)
    else:
        _need(out, "out", torch.int64, 2)
        if out.shape != idx.shape:
            raise ValueError("out must match idx")
    st = lib().kv_idx_local_to_global_i64(idx.data_ptr(), out.data_ptr(), rows, topk, int(sq),
                                          int(seqlen_kv), _stream_handle(idx.device, stream))
    _check(st, "kv_idx_local_to_global_i64")
    return out


_C_INTS = ("page_size", "nope", "pe")


def _fits(**numbers):
    """Numbers that go into the library as C ints, which ctypes would cut to 32 or 64 bits."""
    for name, v in numbers.items():
        most = 2**31 if name in _C_INTS else 2**63
        if not -most <= v < most:
            raise ValueError(f"{name} must be below 2**{most.bit_length() - 1}, got {v}")


def _kept(v, bits=32):
    """A number for the library that keeps it out of range where it is (ctypes would cut it
    to another one)."""
    return min(max(int(v), -2**(bits - 1)), 2**(bits - 1) - 1)


def kv_latent_row_bytes(nope: int, pe: int, fmt: int) -> int:
    """Bytes of one cache row (0 if the shape is invalid); ``fmt`` is
    ``KV_LATENT_BF16``, ``KV_LATENT_E4M3`` or ``KV_LATENT_E2M1``."""
    return int(lib().kv_latent_row_bytes(_kept(nope), _kept(pe), _kept(fmt)))


def kv_latent_empty(num_pages: int, page_size: int, nope: int, pe: int, fmt: int = KV_LATENT_BF16, device="cuda"):
    """A cache of ``num_pages`` pages: bf16 ``[num_pages, page_size, nope+pe]``,
    or uint8 ``[num_pages, page_size, row bytes]`` for ``KV_LATENT_E4M3`` and
    ``KV_LATENT_E2M1``. Its contents are undefined until they are written. The tensor itself
    carries its format, its views and copies do not: of those, the width of a row tells it."""
    nbytes = kv_latent_row_bytes(nope, pe, fmt)
    if nbytes == 0:
        raise ValueError(f"no cache row for nope={nope}, pe={pe}, fmt={fmt}")
    if fmt != KV_LATENT_BF16:
        cache = torch.empty(num_pages, page_size, nbytes, dtype=torch.uint8, device=device)
    else:
        cache = torch.empty(num_pages, page_size, nbytes // 2, dtype=torch.bfloat16, device=device)
    cache._kv_latent_fmt = int(fmt)
    return cache


def _is(t, dtype, ndim):
    return t.dtype is dtype and t.dim() == ndim and t.is_cuda and t.is_contiguous()


@functools.lru_cache(maxsize=64)
def _row_width(nope, pe, fmt):
    return kv_latent_row_bytes(nope, pe, fmt) // (2 if fmt == KV_LATENT_BF16 else 1)


_FORMATS = {KV_LATENT_BF16: "bf16", KV_LATENT_E4M3: "e4m3", KV_LATENT_E2M1: "e2m1"}


def _cache(cache, nope, pe, fmt=None):
    """Check a cache tensor against the channel split; returns its format: ``fmt``, or what
    the tensor carries (:func:`kv_latent_empty`), or what dtype and width tell: bf16 rows are
    the values, uint8 rows the e4m3 layout or the narrower e2m1 one. Widths alone do not tell
    them apart between splits: 448 + 64 channels in e2m1 are as wide as 224 + 64 in e4m3."""
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a torch.Tensor")
    _fits(nope=nope, pe=pe)
    if fmt is not None and fmt not in _FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt}")
    carried = getattr(cache, "_kv_latent_fmt", None)
    if fmt is None:
        fmt = carried
    elif carried is not None and carried != fmt:
        raise ValueError(f"the cache is {_FORMATS[carried]}, fmt says {_FORMATS[fmt]}")
    dtype = (torch.bfloat16 if cache.dtype is torch.bfloat16 else torch.uint8) if fmt is None else \
        (torch.bfloat16 if fmt == KV_LATENT_BF16 else torch.uint8)
    if not _is(cache, dtype, 3):
        _need(cache, "cache", dtype, 3)
    if fmt is None:
        fmt = KV_LATENT_BF16 if dtype is torch.bfloat16 else KV_LATENT_E4M3
        width = _row_width(nope, pe, fmt)
        if cache.shape[2] != width and fmt == KV_LATENT_E4M3 and cache.shape[2] == _row_width(nope, pe, KV_LATENT_E2M1):
            return KV_LATENT_E2M1
    else:
        width = _row_width(nope, pe, fmt)
    if width and cache.shape[2] != width:  # width 0: the library says why the split is refused
        raise ValueError(f"cache rows must be {width} wide for nope={nope}, pe={pe} in {_FORMATS[fmt]}, got {cache.shape[2]}")
    return fmt


def _call_device(cache, stream):
    """The device of a call: the cache's, which has to be the current one (where the
    library launches) and the stream's."""
    index = cache.get_device()
    current = torch._C._cuda_getDevice()
    if index != current:
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{current}")
    if stream is not None and stream.device_index != index:
        raise ValueError(f"stream must be of cuda:{index}, got cuda:{stream.device_index}")
    return index


def _same_device(index, **tensors):
    for name, t in tensors.items():
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _raw_stream(index, stream):
    """The stream's handle; the current stream's where none is given."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def kv_latent_write(cache, x, slots, nope: int, pe: int, stream=None, fmt=None):
    """``cache[slots[i]] = x[i]`` for bf16 vectors ``x`` [n, nope+pe] and int32
    ``slots`` [n] (slot = page * page_size + place in the page), quantising them
    where the cache has 8 or 4 bits; slots out of range store nothing. ``fmt`` says the
    cache's format where the tensor was not made by :func:`kv_latent_empty` (without it the
    width of a row does). Returns ``cache``."""
    if stream is None and _calls is not None:
        got = _calls.latent_write(cache, x, slots, nope, pe, fmt)
        if got is not None:
            return _made(got, "kv_latent_write")
    fmt = _cache(cache, nope, pe, fmt)
    if not (isinstance(x, torch.Tensor) and _is(x, torch.bfloat16, 2)):
        _need(x, "x", torch.bfloat16, 2)
    if not (isinstance(slots, torch.Tensor) and _is(slots, torch.int32, 1)):
        _need(slots, "slots", torch.int32, 1)
    n, d = x.shape
    if d != nope + pe or slots.shape[0] != n:
        raise ValueError(f"x must be [n, {nope + pe}] and slots [n]")
    index = _call_device(cache, stream)
    _same_device(index, x=x, slots=slots)
    pages, size, _ = cache.shape
    st = lib().kv_latent_write(x.data_ptr(), slots.data_ptr(), cache.data_ptr(), n, pages * size, nope, pe, fmt,
                               _raw_stream(index, stream))
    _check(st, "kv_latent_write")
    return cache


def kv_latent_read(cache, slots, nope: int, pe: int, out=None, stream=None, fmt=None):
    """The bf16 vectors [n, nope+pe] that the cache holds at int32 ``slots`` [n]
    (zeros for a slot out of range). ``fmt`` as in :func:`kv_latent_write`."""
    if stream is None and out is None and _calls is not None:
        got = _calls.latent_read(cache, slots, nope, pe, fmt)
        if got is not None:
            return _made(got, "kv_latent_read")
    fmt = _cache(cache, nope, pe, fmt)
    if not (isinstance(slots, torch.Tensor) and _is(slots, torch.int32, 1)):
        _need(slots, "slots", torch.int32, 1)
    n = slots.shape[0]
    index = _call_device(cache, stream)
    if out is None:
        out = _empty((n, nope + pe), torch.bfloat16, cache.device, stream)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (n, nope + pe):
            raise ValueError(f"out must be [{n}, {nope + pe}]")
    _same_device(index, slots=slots, out=out)
    pages, size, _ = cache.shape
    st = lib().kv_latent_read(cache.data_ptr(), slots.data_ptr(), out.data_ptr(), n, pages * size, nope, pe, fmt,
                              _raw_stream(index, stream))
    _check(st, "kv_latent_read")
    return out


def latent_attn_workspace_bytes(rows: int, nh: int, max_tokens: int, nope: int, pe: int) -> int:
    """Workspace bytes the attention needs on the current device (0: none)."""
    return int(lib().latent_attn_workspace_bytes(_kept(rows, 64), _kept(nh), _kept(max_tokens, 64), _kept(nope), _kept(pe)))


def invrope_latent_workspace_bytes(rows: int, nh: int, max_tokens: int, nope: int, pe: int, fmt: int) -> int:
    """Workspace bytes with which the attention over a cache of format ``fmt`` cuts short rows
    the finest: for ``KV_LATENT_E2M1`` more than it asks for."""
    return int(lib().invrope_latent_workspace_bytes(_kept(rows, 64), _kept(nh), _kept(max_tokens, 64), _kept(nope), _kept(pe),
                                                    _kept(fmt)))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index, rows, nh, max_tokens, nope, pe, fmt):  # of the current device, `index`
    if fmt == KV_LATENT_E2M1:
        return invrope_latent_workspace_bytes(rows, nh, max_tokens, nope, pe, fmt)
    return latent_attn_workspace_bytes(rows, nh, max_tokens, nope, pe)


def _attn_io(q, cache, nope, pe, max_tokens, O, lse, workspace, stream, fmt, **tables):
    """Checks and outputs common to the two attention calls."""
    fmt = _cache(cache, nope, pe, fmt)
    if not (isinstance(q, torch.Tensor) and _is(q, torch.bfloat16, 3)):
        _need(q, "q", torch.bfloat16, 3)
    rows, nh, d = q.shape
    if d != nope + pe:
        raise ValueError(f"q must be [rows, nh, {nope + pe}]")
    index, device = _call_device(cache, stream), cache.device
    if O is None:
        O = _empty((rows, nh, d), torch.bfloat16, device, stream)
    else:
        _need(O, "O", torch.bfloat16, 3)
        if O.shape != q.shape:
            raise ValueError("O must have q's shape")
        tables["O"] = O
    if lse is None:
        lse = _empty((rows, nh), torch.float32, device, stream)
    else:
        _need(lse, "lse", torch.float32, 2)
        if tuple(lse.shape) != (rows, nh):
            raise ValueError(f"lse must be [{rows}, {nh}]")
        tables["lse"] = lse
    if workspace is None:
        nbytes = _workspace_bytes(index, rows, nh, max_tokens, nope, pe, fmt)
        if nbytes:
            workspace = _empty((nbytes,), torch.uint8, device, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    else:
        tables["workspace"] = workspace
        nbytes = workspace.numel() * workspace.element_size()
    _same_device(index, q=q, **tables)
    return fmt, O, lse, (workspace.data_ptr() if workspace is not None else None), nbytes, workspace, \
        _raw_stream(index, stream)


def latent_attn_decode(q, cache, page_table, lens, nope: int, pe: int, scale=None, O=None, lse=None,
                       workspace=None, stream=None, fmt=None):
    """Attention of one new token a row over its pages of the latent cache, which
    are keys and values of every head: ``q`` bf16 [rows, nh, nope+pe],
    ``page_table`` int32 [rows, max_pages], ``lens`` int32 [rows] tokens a row.
    ``scale`` defaults to ``(nope+pe) ** -0.5``. Returns ``(O bf16, lse fp32 [rows, nh])``;
    a row with nothing to attend to gives zeros and -inf. ``fmt`` as in :func:`kv_latent_write`."""
    if stream is None and O is None and lse is None and workspace is None and lens is not None and _calls is not None:
        got = _calls.attn(q, cache, page_table, lens, nope, pe, scale, fmt)
        if got is not None:
            return _made(got, "latent_attn_decode")
    for t, name, ndim in ((page_table, "page_table", 2), (lens, "lens", 1)):
        if not (isinstance(t, torch.Tensor) and _is(t, torch.int32, ndim)):
            _need(t, name, torch.int32, ndim)
    max_pages = page_table.shape[1]
    fmt, O, lse, ws, ws_bytes, workspace, handle = _attn_io(
        q, cache, nope, pe, max_pages * cache.shape[1], O, lse, workspace, stream, fmt, page_table=page_table,
        lens=lens)
    rows, nh, d = q.shape
    if page_table.shape[0] != rows or lens.shape[0] != rows:
        raise ValueError(f"page_table must be [{rows}, max_pages] and lens [{rows}]")
    pages, size, _ = cache.shape
    st = lib().latent_attn_decode(q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), lens.data_ptr(), O.data_ptr(),
                                  lse.data_ptr(), ws, ws_bytes, rows, nh, nope, pe, fmt, pages, size, max_pages,
                                  d ** -0.5 if scale is None else float(scale), handle)
    _check(st, "latent_attn_decode")
    return O, lse


def latent_attn_sparse(q, cache, idx, nope: int, pe: int, scale=None, O=None, lse=None, workspace=None, stream=None,
                       fmt=None):
    """The same attention over the cache slots that ``idx`` int32 [rows, topk]
    selects for each row (the flat-global table of :func:`kv_idx_local_to_global`;
    entries out of range, such as -1 padding, are left out). ``fmt`` as in
    :func:`kv_latent_write`."""
    if stream is None and O is None and lse is None and workspace is None and _calls is not None:
        got = _calls.attn(q, cache, idx, None, nope, pe, scale, fmt)
        if got is not None:
            return _made(got, "latent_attn_sparse")
    if not (isinstance(idx, torch.Tensor) and _is(idx, torch.int32, 2)):
        _need(idx, "idx", torch.int32, 2)
    rows, topk = idx.shape
    fmt, O, lse, ws, ws_bytes, workspace, handle = _attn_io(
        q, cache, nope, pe, topk, O, lse, workspace, stream, fmt, idx=idx)
    if q.shape[0] != rows:
        raise ValueError("idx must have a row for each of q's")
    nh, d = q.shape[1:]
    pages, size, _ = cache.shape
    st = lib().latent_attn_sparse(q.data_ptr(), cache.data_ptr(), idx.data_ptr(), O.data_ptr(), lse.data_ptr(), ws,
                                  ws_bytes, rows, nh, nope, pe, fmt, pages * size, topk,
                                  d ** -0.5 if scale is None else float(scale), handle)
    _check(st, "latent_attn_sparse")
    return O, lse


def kv_pages_empty(b: int, max_pages: int, num_pages: int, device="cuda"):
    """``(state, page_table, queue)`` of ``b`` empty sequences over a pool of ``num_pages``
    free pages, of which a sequence has up to ``max_pages``: int32 [b + 2], [b, max_pages]
    and [num_pages]. ``state[:b]`` are the sequences' lengths."""
    state = torch.zeros(b + 2, dtype=torch.int32, device=device)
    state[b + 1] = num_pages
    return (state, torch.full((b, max_pages), -1, dtype=torch.int32, device=device),
            torch.arange(num_pages, dtype=torch.int32, device=device))


def _int32(t, name, ndim):
    if not (isinstance(t, torch.Tensor) and _is(t, torch.int32, ndim)):
        _need(t, name, torch.int32, ndim)


def kv_pages_advance(state, page_table, queue, new_tokens, page_size: int, max_tokens: int, state_out=None, out=None,
                     stream=None):
    """One step of the sequences of :func:`kv_pages_empty`: ``new_tokens`` int32 [b] asks
    for that many further tokens of each (a negative number ends it and gives its pages
    back). Pages go from ``queue`` into ``page_table``; ``state`` becomes the state after
    the step, or ``state_out`` does. Returns int32 ``(slots, positions, rows, starts,
    granted)`` of ``max_tokens``, ``max_tokens``, ``max_tokens``, b + 1 and b entries (in the
    tensors of ``out``, if given): the tokens asked for, one sequence after the other, with
    their slots (-1 where the sequence got nothing, and behind the last token), positions
    and sequences, where each sequence's begin, and how many it got."""
    if out is not None:
        out = tuple(out)
    if stream is None and _calls is not None:
        got = _calls.pages_advance(state, page_table, queue, new_tokens, page_size, max_tokens, state_out, out)
        if got is not None:
            return _made(got, "kv_pages_advance")
    _int32(state, "state", 1)
    _int32(page_table, "page_table", 2)
    _int32(queue, "queue", 1)
    _int32(new_tokens, "new_tokens", 1)
    _fits(page_size=page_size, max_tokens=max_tokens)
    b, max_pages = page_table.shape
    if state.shape[0] != b + 2 or new_tokens.shape[0] != b:
        raise ValueError(f"state must be [{b + 2}] and new_tokens [{b}]")
    index = _call_device(state, stream)
    tensors = {"page_table": page_table, "queue": queue, "new_tokens": new_tokens}
    if state_out is None:
        state_out = state
    else:
        _int32(state_out, "state_out", 1)
        if state_out.shape[0] != b + 2:
            raise ValueError(f"state_out must be [{b + 2}]")
        tensors["state_out"] = state_out
    if out is None:
        if max_tokens < 0:
            raise ValueError("max_tokens must not be negative")
        # (one allocation: the parts are as a caller would allocate them, but for their alignment)
        out = _empty((3 * max_tokens + 2 * b + 1,), torch.int32, state.device, stream).split(
            (max_tokens, max_tokens, max_tokens, b + 1, b))
    else:
        for t, name, size in zip(out, ("slots", "positions", "rows", "starts", "granted"),
                                 (max_tokens, max_tokens, max_tokens, b + 1, b), strict=True):
            _int32(t, name, 1)
            if t.shape[0] != size:
                raise ValueError(f"{name} must be [{size}]")
            tensors[name] = t
    _same_device(index, **tensors)
    slots, positions, rows, starts, granted = out
    st = lib().kv_pages_advance(state.data_ptr(), state_out.data_ptr(), page_table.data_ptr(), queue.data_ptr(),
                                new_tokens.data_ptr(), slots.data_ptr(), positions.data_ptr(), rows.data_ptr(),
                                starts.data_ptr(), granted.data_ptr(), b, max_pages, queue.shape[0], int(page_size),
                                int(max_tokens), _raw_stream(index, stream))
    _check(st, "kv_pages_advance")
    return out


def kv_idx_local_to_slots(idx, page_table, lens, page_size: int, num_pages: int, sq: int = 1, seq=None, out=None,
                          stream=None):
    """The cache slots (int32 [rows, topk], -1: none) of token numbers ``idx`` int32 [rows,
    topk] within each row's sequence, through its pages: row r is of sequence ``seq[r]``
    (int32 [rows]), or ``r // sq``. Negative numbers and those at or beyond the sequence's
    length ``lens[s]`` give -1. ``out`` may be ``idx``."""
    if stream is None and out is None and _calls is not None:
        got = _calls.idx_local_to_slots(idx, page_table, lens, page_size, num_pages, sq, seq)
        if got is not None:
            return _made(got, "kv_idx_local_to_slots")
    _int32(idx, "idx", 2)
    _int32(page_table, "page_table", 2)
    _int32(lens, "lens", 1)
    _fits(page_size=page_size, num_pages=num_pages, sq=sq)
    rows, topk = idx.shape
    seqs, max_pages = page_table.shape
    if lens.shape[0] != seqs:
        raise ValueError(f"lens must be [{seqs}]")
    index = _call_device(idx, stream)
    tensors = {"page_table": page_table, "lens": lens}
    if seq is not None:
        _int32(seq, "seq", 1)
        if seq.shape[0] != rows:
            raise ValueError(f"seq must be [{rows}]")
        tensors["seq"] = seq
    if out is None:
        out = _empty((rows, topk), torch.int32, idx.device, stream)
    else:
        _int32(out, "out", 2)
        if out.shape != idx.shape:
            raise ValueError("out must match idx")
        tensors["out"] = out
    _same_device(index, **tensors)
    st = lib().kv_idx_local_to_slots(idx.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
                                     seq.data_ptr() if seq is not None else None, out.data_ptr(), rows, topk, int(sq), seqs,
                                     max_pages, int(num_pages), int(page_size), _raw_stream(index, stream))
    _check(st, "kv_idx_local_to_slots")
    return out


def rope_freqs(pe: int, theta: float = 10000.0, scaling: int = ROPE_SCALE_NONE, factor: float = 1.0,
               original: float = 4096.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Frequencies of ``pe / 2`` rotary pairs (radians a position, float64 on the host) and
    the amplitude that goes with them, for :func:`rope_apply`; ``scaling`` is one of
    ``ROPE_SCALE_NONE``, ``_LINEAR``, ``_NTK`` and ``_YARN``, ``original`` the number of
    positions that the frequencies were made for."""
    pe = min(int(pe), 2**31 - 2)
    freqs = torch.empty(pe // 2 if 0 < pe <= 512 else 0, dtype=torch.float64)  # the library says why it refuses others
    amplitude = ctypes.c_double(0.0)
    st = lib().rope_freqs(max(pe, -1), float(theta), _kept(scaling), float(factor), float(original), float(beta_fast),
                          float(beta_slow), freqs.data_ptr() or None, ctypes.byref(amplitude))
    _check(st, "rope_freqs")
    return freqs, amplitude.value


_ROPE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_rope_tensor = struct.Struct("PPqqqqqqq").pack  # RopeTensor


def _rope_pair(x, out, pe, offset, index, dtype, n):
    """RopeTensor of one tensor and its output, both [n, heads, d] or [n, d]."""
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor for each x")
    if out.dtype != dtype or x.dtype != dtype or out.shape != x.shape:
        raise ValueError("tensors of one call must have one type, and an output its input's shape")
    if x.get_device() != index or out.get_device() != index:
        raise ValueError(f"x and out must be on cuda:{index}, got {x.device} and {out.device}")
    if x.dim() == 3:
        rows, heads, d = x.shape
        (x_row, x_head, x_c), (out_row, out_head, out_c) = x.stride(), out.stride()
    elif x.dim() == 2:
        (rows, d), heads, x_head, out_head = x.shape, 1, 0, 0
        (x_row, x_c), (out_row, out_c) = x.stride(), out.stride()
    else:
        raise ValueError(f"x must be [n, heads, d] or [n, d], got {tuple(x.shape)}")
    if rows != n:
        raise ValueError("tensors of one call must have the same rows")
    if d > 1 and (x_c != 1 or out_c != 1):
        raise ValueError("the last axis of x and out must be contiguous")
    return _rope_tensor(x.data_ptr(), out.data_ptr(), heads, d, d - pe if offset is None else offset,
                        x_row, x_head, out_row, out_head)


def rope_apply(x, freqs, positions=None, pos0: int = 0, offset=None, amplitude: float = 1.0, interleaved: bool = False,
               inverse: bool = False, out=None, stream=None):
    """Rotary positions on ``pe = 2 * len(freqs)`` channels of each head of ``x`` [n, heads, d]
    (or [n, d]; bf16, fp16 or fp32, any strides with a contiguous last axis), from channel
    ``offset`` (default: the last ``pe``); row r is at ``pos0 + positions[r]`` (int32 [n]), else
    ``pos0 + r``. Pairs are (i, i + pe/2), or ``interleaved`` (2i, 2i + 1); they are multiplied by
    ``amplitude`` and turned by the angle, with ``inverse`` by its negative, which is the
    gradient of the call without. ``x`` may be a list of up to four tensors with the same rows,
    which takes one launch where they have one layout. Returns the outputs, new ones or ``out``, which may be ``x`` itself."""
    if stream is None and out is None and _calls is not None:
        got = _calls.rope(x, freqs, positions, pos0, offset, amplitude, interleaved, inverse)
        if got is not None:
            return _made(got, "rope_apply")
    many = not isinstance(x, torch.Tensor)
    xs = x if many else (x,)
    outs = out if many or out is None else (out,)
    if not 1 <= len(xs) <= ROPE_MAX_TENSORS or not all(isinstance(t, torch.Tensor) for t in xs):
        raise ValueError(f"x must be a tensor or 1 to {ROPE_MAX_TENSORS} of them")
    first = xs[0]
    dtype = _ROPE_TYPES.get(first.dtype)
    if dtype is None:
        raise TypeError(f"x must be bf16, fp16 or fp32, got {first.dtype}")
    if not first.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if not (isinstance(freqs, torch.Tensor) and freqs.dtype is torch.float64 and freqs.dim() == 1 and not freqs.is_cuda
            and freqs.is_contiguous()):
        raise ValueError("freqs must be a contiguous float64 vector on the host")
    index = _call_device(first, stream)
    _fits(pos0=pos0, offset=offset or 0)
    if outs is None:
        outs = [_empty(t.shape, t.dtype, t.device, stream) for t in xs]
    elif isinstance(outs, torch.Tensor) or len(outs) != len(xs):
        raise ValueError("out must hold a tensor for each of x")
    n, pe = first.shape[0] if first.dim() else 0, 2 * freqs.shape[0]
    tensors = b"".join([_rope_pair(t, o, pe, offset, index, first.dtype, n) for t, o in zip(xs, outs)])
    if positions is None:
        where = None
    else:
        _int32(positions, "positions", 1)
        if positions.shape[0] != n:
            raise ValueError(f"positions must be [{n}]")
        _same_device(index, positions=positions)
        where = positions.data_ptr()
    st = lib().rope_apply(tensors, len(xs), freqs.data_ptr(), where, int(pos0), n, _kept(pe), float(amplitude), dtype, bool(interleaved),
                          bool(inverse), _raw_stream(index, stream))
    _check(st, "rope_apply")
    return outs if many else outs[0]


def invrope_take_device_fault() -> int:
    """Synchronise, then return and clear the kernels' watchdog code (0 = no fault)."""
    v = ctypes.c_int(0)
    _check(lib().invrope_take_device_fault(ctypes.byref(v)), "invrope_take_device_fault")
    return v.value


def invrope_debug_occupy_next_slot(which: str, owner: int) -> None:
    """Test hook: mark the work-counter slot the next eager ``"fwd"`` or
    ``"remap"`` launch will take as held by launch tag ``owner``."""
    code = {"fwd": 0, "remap": 1}[which]
    _check(lib().invrope_debug_occupy_next_slot(code, int(owner)), "invrope_debug_occupy_next_slot")


def invrope_watchdog_selftest(limit_us: int = 50000) -> int:
    """Run one bounded wait that must expire; returns the recorded watchdog code."""
    v = ctypes.c_int(0)
    _check(lib().invrope_watchdog_selftest(int(limit_us), ctypes.byref(v)), "invrope_watchdog_selftest")
    return v.value
