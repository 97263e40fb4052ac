"""ctypes binding of ``libinvrope.so`` (the C ABI declared in ``include/invrope.h``
and ``include/latent_attn.h``).

Argument marshalling only: each function checks that torch tensors have the
dtype / device / layout the C ABI expects, allocates outputs with torch when
the caller passes none, and forwards raw device pointers, sizes and the
current CUDA stream. All arithmetic runs in the library's kernels. There is no
fallback: if the library is not built, the first call raises.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

# INVROPE_LIBRARY selects another build of the same library (e.g. the
# debug-bounds build, libinvrope_debug.so); it must export the same symbols.
_LIB_PATH = os.environ.get("INVROPE_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                             "libinvrope.so")
_lib = None

INVROPE_OK = 0
INVROPE_ERR_INVALID_ARG = 1
INVROPE_ERR_UNSUPPORTED = 2
INVROPE_ERR_WORKSPACE = 3
INVROPE_ERR_CUDA = 4
INVROPE_ERR_DEVICE = 5

# name -> (restype, argtypes); mirrors include/invrope.h and include/latent_attn.h
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
}

KV_LATENT_BF16 = 0
KV_LATENT_E4M3 = 1

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
    global _lib
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
    return _lib


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


def kv_latent_row_bytes(nope: int, pe: int, fmt: int) -> int:
    """Bytes of one cache row (0 if the shape is invalid); ``fmt`` is
    ``KV_LATENT_BF16`` or ``KV_LATENT_E4M3``."""
    return int(lib().kv_latent_row_bytes(int(nope), int(pe), int(fmt)))


def kv_latent_empty(num_pages: int, page_size: int, nope: int, pe: int, fmt: int = KV_LATENT_BF16, device="cuda"):
    """A cache of ``num_pages`` pages: bf16 ``[num_pages, page_size, nope+pe]``,
    or uint8 ``[num_pages, page_size, row bytes]`` for ``KV_LATENT_E4M3``.
    Its contents are undefined until they are written."""
    nbytes = kv_latent_row_bytes(nope, pe, fmt)
    if nbytes == 0:
        raise ValueError(f"no cache row for nope={nope}, pe={pe}, fmt={fmt}")
    if fmt == KV_LATENT_E4M3:
        return torch.empty(num_pages, page_size, nbytes, dtype=torch.uint8, device=device)
    return torch.empty(num_pages, page_size, nbytes // 2, dtype=torch.bfloat16, device=device)


def _is(t, dtype, ndim):
    return t.dtype is dtype and t.dim() == ndim and t.is_cuda and t.is_contiguous()


@functools.lru_cache(maxsize=64)
def _row_width(nope, pe, fmt):
    return kv_latent_row_bytes(nope, pe, fmt) // (1 if fmt == KV_LATENT_E4M3 else 2)


def _cache(cache, nope, pe):
    """Check a cache tensor against the channel split; returns its format. The
    dtype tells it: bf16 rows are the values, uint8 rows the e4m3 layout."""
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a torch.Tensor")
    fmt = KV_LATENT_BF16 if cache.dtype is torch.bfloat16 else KV_LATENT_E4M3
    dtype = torch.uint8 if fmt == KV_LATENT_E4M3 else torch.bfloat16
    if not _is(cache, dtype, 3):
        _need(cache, "cache", dtype, 3)
    width = _row_width(nope, pe, fmt)
    if width and cache.shape[2] != width:  # width 0: the library says why the split is refused
        raise ValueError(f"cache rows must be {width} wide for nope={nope}, pe={pe}, got {cache.shape[2]}")
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


def kv_latent_write(cache, x, slots, nope: int, pe: int, stream=None):
    """``cache[slots[i]] = x[i]`` for bf16 vectors ``x`` [n, nope+pe] and int32
    ``slots`` [n] (slot = page * page_size + place in the page), quantising them
    where the cache is 8-bit; slots out of range store nothing. Returns ``cache``."""
    fmt = _cache(cache, nope, pe)
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


def kv_latent_read(cache, slots, nope: int, pe: int, out=None, stream=None):
    """The bf16 vectors [n, nope+pe] that the cache holds at int32 ``slots`` [n]
    (zeros for a slot out of range)."""
    fmt = _cache(cache, nope, pe)
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
    return int(lib().latent_attn_workspace_bytes(int(rows), int(nh), int(max_tokens), int(nope), int(pe)))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index, rows, nh, max_tokens, nope, pe):
    return latent_attn_workspace_bytes(rows, nh, max_tokens, nope, pe)  # of the current device, `index`


def _attn_io(q, cache, nope, pe, max_tokens, O, lse, workspace, stream, **tables):
    """Checks and outputs common to the two attention calls."""
    fmt = _cache(cache, nope, pe)
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
        nbytes = _workspace_bytes(index, rows, nh, max_tokens, nope, pe)
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
                       workspace=None, stream=None):
    """Attention of one new token a row over its pages of the latent cache, which
    are keys and values of every head: ``q`` bf16 [rows, nh, nope+pe],
    ``page_table`` int32 [rows, max_pages], ``lens`` int32 [rows] tokens a row.
    ``scale`` defaults to ``(nope+pe) ** -0.5``. Returns ``(O bf16, lse fp32 [rows, nh])``;
    a row with nothing to attend to gives zeros and -inf."""
    for t, name, ndim in ((page_table, "page_table", 2), (lens, "lens", 1)):
        if not (isinstance(t, torch.Tensor) and _is(t, torch.int32, ndim)):
            _need(t, name, torch.int32, ndim)
    max_pages = page_table.shape[1]
    fmt, O, lse, ws, ws_bytes, workspace, handle = _attn_io(
        q, cache, nope, pe, max_pages * cache.shape[1], O, lse, workspace, stream, page_table=page_table, lens=lens)
    rows, nh, d = q.shape
    if page_table.shape[0] != rows or lens.shape[0] != rows:
        raise ValueError(f"page_table must be [{rows}, max_pages] and lens [{rows}]")
    pages, size, _ = cache.shape
    st = lib().latent_attn_decode(q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), lens.data_ptr(), O.data_ptr(),
                                  lse.data_ptr(), ws, ws_bytes, rows, nh, nope, pe, fmt, pages, size, max_pages,
                                  d ** -0.5 if scale is None else float(scale), handle)
    _check(st, "latent_attn_decode")
    return O, lse


def latent_attn_sparse(q, cache, idx, nope: int, pe: int, scale=None, O=None, lse=None, workspace=None, stream=None):
    """The same attention over the cache slots that ``idx`` int32 [rows, topk]
    selects for each row (the flat-global table of :func:`kv_idx_local_to_global`;
    entries out of range, such as -1 padding, are left out)."""
    if not (isinstance(idx, torch.Tensor) and _is(idx, torch.int32, 2)):
        _need(idx, "idx", torch.int32, 2)
    rows, topk = idx.shape
    fmt, O, lse, ws, ws_bytes, workspace, handle = _attn_io(
        q, cache, nope, pe, topk, O, lse, workspace, stream, idx=idx)
    if q.shape[0] != rows:
        raise ValueError("idx must have a row for each of q's")
    nh, d = q.shape[1:]
    pages, size, _ = cache.shape
    st = lib().latent_attn_sparse(q.data_ptr(), cache.data_ptr(), idx.data_ptr(), O.data_ptr(), lse.data_ptr(), ws,
                                  ws_bytes, rows, nh, nope, pe, fmt, pages * size, topk,
                                  d ** -0.5 if scale is None else float(scale), handle)
    _check(st, "latent_attn_sparse")
    return O, lse


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
