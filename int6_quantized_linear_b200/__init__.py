"""Python binding of ``libqlinear.so``: the B200 weight-only quantized linear layer.

Argument marshalling only -- every step of the computation runs in the
library's CUDA kernels.  Functions carry the C entry points' names
(``include/qlinear.h``), take ``torch.Tensor`` arguments on a CUDA device,
pass their data pointers and the current CUDA stream, and raise
``QLinearError`` on a non-OK status.  There is no CPU fallback: if the library
is missing, the first call raises.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from dataclasses import dataclass

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlinear.so")

QL_OK, QL_ERR_NULL, QL_ERR_SHAPE, QL_ERR_ALIGN, QL_ERR_RANGE, QL_ERR_UNSUPPORTED, QL_ERR_CUDA, \
    QL_ERR_TIMEOUT = range(8)
FORMATS = {"int4": 1, "int6": 2, "affine": 3, "int6p": 4}  # int6p: int6 codes in planar storage
QL_OUT_F32, QL_OUT_BF16 = 0, 1
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1, "gelu": 2}


class QLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class ql_desc(C.Structure):
    _fields_ = [("fmt", C.c_int32), ("bits", C.c_int32), ("group", C.c_int32), ("reserved", C.c_int32),
                ("N", C.c_int64), ("K", C.c_int64)]


class ql_packed(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("gmeta", C.c_void_p), ("steps", C.c_void_p)]


ql_packed_const = ql_packed  # same layout, const in C


class ql_unpacked(C.Structure):
    _fields_ = [("q", C.c_void_p), ("meta0", C.c_void_p), ("meta1", C.c_void_p), ("step0", C.c_void_p),
                ("step1", C.c_void_p)]


ql_unpacked_out = ql_unpacked


class ql_saved8(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("exps", C.c_void_p)]


ql_saved8_const = ql_saved8

_lib = None

# (name, argtypes) of every entry point declared in include/qlinear.h
_SIGNATURES = {
    "qlinear_version": ([], C.c_int32),
    "qlinear_status_string": ([C.c_int], C.c_char_p),
    "qlinear_packed_bytes": ([C.POINTER(ql_desc), C.POINTER(C.c_size_t), C.POINTER(C.c_size_t),
                              C.POINTER(C.c_size_t)], C.c_int),
    "qlinear_pack": ([C.POINTER(ql_desc), C.POINTER(ql_unpacked), C.POINTER(ql_packed), C.c_void_p], C.c_int),
    "qlinear_unpack": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.POINTER(ql_unpacked), C.c_void_p], C.c_int),
    "qlinear_dequant": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int32, C.c_void_p], C.c_int),
    "qlinear_gemv_workspace_bytes": ([C.POINTER(ql_desc), C.c_int64, C.POINTER(C.c_size_t)], C.c_int),
    "qlinear_gemv": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                      C.c_size_t, C.c_void_p], C.c_int),
    "qlinear_gemm_workspace_bytes": ([C.POINTER(ql_desc), C.c_int64, C.POINTER(C.c_size_t)], C.c_int),
    "qlinear_gemm": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                      C.c_size_t, C.c_void_p], C.c_int),
    "qlinear_gemm_noalloc": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_void_p,
                              C.c_void_p], C.c_int),
    "qlinear_sync_status": ([C.c_void_p], C.c_int),
    "qlinear_set_withhold_copies": ([C.c_int32], C.c_int),
    "qlinear_gemv_bias": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_void_p,
                           C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p], C.c_int),
    "qlinear_gemm_bias": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_void_p,
                           C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p], C.c_int),
    "qlinear_concat_n": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.POINTER(ql_desc), C.POINTER(ql_packed),
                          C.POINTER(ql_packed), C.c_void_p], C.c_int),
    "qlinear_quantize_meta": ([C.POINTER(ql_desc), C.c_void_p, C.c_void_p, C.POINTER(ql_unpacked), C.c_void_p],
                              C.c_int),
    "qlinear_saved8_bytes": ([C.c_int64, C.c_int64, C.POINTER(C.c_size_t), C.POINTER(C.c_size_t)], C.c_int),
    "qlinear_save8": ([C.c_void_p, C.c_int64, C.c_int64, C.POINTER(ql_saved8), C.c_void_p], C.c_int),
    "qlinear_restore8": ([C.POINTER(ql_saved8), C.c_int64, C.c_int64, C.c_void_p, C.c_void_p], C.c_int),
    "qlinear_gated_workspace_bytes": ([C.POINTER(ql_desc), C.c_int64, C.POINTER(C.c_size_t)], C.c_int),
    "qlinear_gated": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_int32, C.c_void_p,
                       C.POINTER(ql_saved8), C.c_void_p, C.c_size_t, C.c_void_p], C.c_int),
    "qlinear_gemm_dx_workspace_bytes": ([C.POINTER(ql_desc), C.c_int64, C.POINTER(C.c_size_t)], C.c_int),
    "qlinear_gemm_dx": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                         C.c_size_t, C.c_void_p], C.c_int),
    "qlinear_gated_backward": ([C.POINTER(ql_desc), C.POINTER(ql_packed), C.POINTER(ql_saved8), C.c_void_p,
                                C.c_int64, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p],
                               C.c_int),
}


def lib():
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run __graft_entry__.build() or python -m int6_quantized_linear_b200._build)")
        L = C.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().qlinear_status_string(status).decode()


def _check(status: int, where: str):
    if status != QL_OK:
        raise QLinearError(status, where)


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


@dataclass(frozen=True)
class Desc:
    """A quantized weight matrix's format and shape (mirrors ``ql_desc``)."""
    fmt: str
    N: int
    K: int
    bits: int = 0
    group: int = 0

    def c(self) -> ql_desc:
        return ql_desc(FORMATS[self.fmt], self.bits, self.group, 0, self.N, self.K)


def qlinear_version() -> int:
    return lib().qlinear_version()


def qlinear_packed_bytes(desc: Desc):
    c, g, s = C.c_size_t(), C.c_size_t(), C.c_size_t()
    d = desc.c()
    _check(lib().qlinear_packed_bytes(C.byref(d), C.byref(c), C.byref(g), C.byref(s)), "qlinear_packed_bytes")
    return c.value, g.value, s.value


def alloc_packed(desc: Desc, device="cuda"):
    """Allocate (uninitialised) packed buffers for ``desc`` as uint8 tensors."""
    import torch
    c, g, s = qlinear_packed_bytes(desc)
    return (torch.empty(c, dtype=torch.uint8, device=device), torch.empty(g, dtype=torch.uint8, device=device),
            torch.empty(max(s, 16), dtype=torch.uint8, device=device))


def qlinear_pack(desc: Desc, q, meta0, meta1, step0, step1, codes, gmeta, steps, stream=None):
    d = desc.c()
    u = ql_unpacked(_ptr(q), _ptr(meta0), _ptr(meta1), _ptr(step0), _ptr(step1))
    o = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_pack(C.byref(d), C.byref(u), C.byref(o), _stream(stream)), "qlinear_pack")


def qlinear_unpack(desc: Desc, codes, gmeta, steps, q, meta0=None, meta1=None, step0=None, step1=None,
                   stream=None):
    d = desc.c()
    i = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    o = ql_unpacked(_ptr(q), _ptr(meta0), _ptr(meta1), _ptr(step0), _ptr(step1))
    _check(lib().qlinear_unpack(C.byref(d), C.byref(i), C.byref(o), _stream(stream)), "qlinear_unpack")


def qlinear_dequant(desc: Desc, codes, gmeta, steps, out, out_dtype: int, stream=None):
    d = desc.c()
    w = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_dequant(C.byref(d), C.byref(w), _ptr(out), out_dtype, _stream(stream)),
           "qlinear_dequant")


def qlinear_quantize_meta(desc: Desc, scale, zero, meta0, meta1, step0, step1, stream=None):
    """Float per-group metadata (float32 CUDA tensors) -> codes and fp16 step bits in the given
    output tensors (int4: sc, zc u8 [N][K/32], ss, zs [N][K/256] 16-bit; int6: sc i8 [N][K/16],
    st [N][K/256]; pass None for the unused ones).  Out-of-domain inputs show up as QL_ERR_RANGE
    from qlinear_sync_status()."""
    d = desc.c()
    o = ql_unpacked(None, _ptr(meta0), _ptr(meta1), _ptr(step0), _ptr(step1))
    _check(lib().qlinear_quantize_meta(C.byref(d), _ptr(scale), _ptr(zero), C.byref(o), _stream(stream)),
           "qlinear_quantize_meta")


def qlinear_gemv_workspace_bytes(desc: Desc, M: int) -> int:
    d = desc.c()
    n = C.c_size_t()
    _check(lib().qlinear_gemv_workspace_bytes(C.byref(d), M, C.byref(n)), "qlinear_gemv_workspace_bytes")
    return n.value


def alloc_gemv_workspace(desc: Desc, M: int, device="cuda"):
    import torch
    return torch.empty(qlinear_gemv_workspace_bytes(desc, M), dtype=torch.uint8, device=device)


def qlinear_gemv(desc: Desc, codes, gmeta, steps, x, M: int, y, workspace=None, stream=None):
    """``workspace``: a uint8 CUDA tensor of at least qlinear_gemv_workspace_bytes(desc, M) bytes;
    allocated here when omitted."""
    if workspace is None:
        workspace = alloc_gemv_workspace(desc, M, x.device)
    d = desc.c()
    w = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_gemv(C.byref(d), C.byref(w), _ptr(x), M, _ptr(y), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream)), "qlinear_gemv")


def qlinear_gemv_bias(desc: Desc, codes, gmeta, steps, x, M: int, bias, y, workspace=None, stream=None):
    """qlinear_gemv with a bf16 [N] bias added before the rounding to bf16."""
    if workspace is None:
        workspace = alloc_gemv_workspace(desc, M, x.device)
    d = desc.c()
    w = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_gemv_bias(C.byref(d), C.byref(w), _ptr(x), M, _ptr(bias), _ptr(y), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "qlinear_gemv_bias")


def qlinear_concat_n(desc_a: Desc, packed_a, desc_b: Desc, packed_b, out, stream=None):
    """Stack two packed layers along N into ``out`` = (codes, gmeta, steps) of the stacked layer."""
    da, db = desc_a.c(), desc_b.c()
    wa = ql_packed(*[_ptr(t) for t in packed_a])
    wb = ql_packed(*[_ptr(t) for t in packed_b])
    o = ql_packed(*[_ptr(t) for t in out])
    _check(lib().qlinear_concat_n(C.byref(da), C.byref(wa), C.byref(db), C.byref(wb), C.byref(o), _stream(stream)),
           "qlinear_concat_n")


def qlinear_gemm_workspace_bytes(desc: Desc, M: int) -> int:
    d = desc.c()
    n = C.c_size_t()
    _check(lib().qlinear_gemm_workspace_bytes(C.byref(d), M, C.byref(n)), "qlinear_gemm_workspace_bytes")
    return n.value


def alloc_gemm_workspace(desc: Desc, M: int, device="cuda"):
    """Allocate a workspace for qlinear_gemm (torch allocations are 256-byte aligned)."""
    import torch
    return torch.empty(qlinear_gemm_workspace_bytes(desc, M), dtype=torch.uint8, device=device)


def qlinear_gemm(desc: Desc, codes, gmeta, steps, x, M: int, y, workspace=None, stream=None):
    """``workspace``: a uint8 CUDA tensor of at least qlinear_gemm_workspace_bytes(desc, M) bytes;
    allocated here when omitted."""
    if workspace is None:
        workspace = alloc_gemm_workspace(desc, M, x.device)
    d = desc.c()
    w = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_gemm(C.byref(d), C.byref(w), _ptr(x), M, _ptr(y), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream)), "qlinear_gemm")


def qlinear_gemm_bias(desc: Desc, codes, gmeta, steps, x, M: int, bias, y, workspace=None, stream=None):
    """qlinear_gemm with a bf16 [N] bias added before the rounding to bf16."""
    if workspace is None:
        workspace = alloc_gemm_workspace(desc, M, x.device)
    d = desc.c()
    w = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_gemm_bias(C.byref(d), C.byref(w), _ptr(x), M, _ptr(bias), _ptr(y), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "qlinear_gemm_bias")


def qlinear_gemm_noalloc(desc: Desc, codes, gmeta, steps, x, M: int, y, stream=None):
    """qlinear_gemm without a workspace argument, for callers that may not allocate device memory:
    the library uses its own fixed 32 MiB device array (shared by every call on the device, so calls
    must not overlap on the GPU).  Raises QLinearError(QL_ERR_RANGE) when the problem needs more."""
    d = desc.c()
    w = ql_packed(_ptr(codes), _ptr(gmeta), _ptr(steps))
    _check(lib().qlinear_gemm_noalloc(C.byref(d), C.byref(w), _ptr(x), M, _ptr(y), _stream(stream)),
           "qlinear_gemm_noalloc")


# ---- gated feed-forward block, 8-bit checkpoints, input gradients ------------------------------------------
# These calls check their tensors before the library sees a pointer: contiguous CUDA tensors of one device, of
# the type and at least the size that the call reads or writes.  They run on that device (also when it is not
# the current one), on its current stream or on `stream`.  A decode step is a few microseconds of GPU time, so
# what depends on the layer and M alone is worked out once.

def _refuse(where: str, t, dtype, numel: int):
    if t is None:
        raise QLinearError(QL_ERR_NULL, where)
    if not t.is_cuda or (t.dtype == dtype and t.is_contiguous() and t.numel() >= numel):
        raise QLinearError(QL_ERR_UNSUPPORTED, f"{where}: tensors must be on one CUDA device")
    raise QLinearError(QL_ERR_SHAPE, f"{where}: expected a contiguous {dtype} tensor of at least {numel} elements, "
                                     f"got {t.dtype} of shape {tuple(t.shape)}")


def _ptr_of(where: str, t, dtype, numel: int, dev: int) -> int:
    """The address of a contiguous CUDA tensor of the given type, size and device; anything else is refused."""
    if t is None or t.dtype != dtype or t.numel() < numel or not t.is_contiguous() or t.get_device() != dev:
        _refuse(where, t, dtype, numel)
    return t.data_ptr()


def _device_of(where: str, t) -> int:
    if t is None or not t.is_cuda:
        raise QLinearError(QL_ERR_NULL if t is None else QL_ERR_UNSUPPORTED, f"{where}: tensors must be on one CUDA device")
    return t.get_device()


def _buffer_of(where: str, t, nbytes: int, dev: int) -> int:
    """The address of a contiguous CUDA buffer of any type with at least nbytes bytes (0: an unused one)."""
    if nbytes == 0:
        return 0 if t is None else t.data_ptr()
    if t is None:
        raise QLinearError(QL_ERR_NULL, where)
    if t.get_device() != dev:
        raise QLinearError(QL_ERR_UNSUPPORTED, f"{where}: tensors must be on one CUDA device")
    if t.nbytes < nbytes or not t.is_contiguous():
        raise QLinearError(QL_ERR_SHAPE, f"{where}: expected a contiguous buffer of at least {nbytes} bytes")
    return t.data_ptr()


def _packed_of(where: str, sizes, codes, gmeta, steps, dev: int) -> ql_packed:
    return ql_packed(_buffer_of(where, codes, sizes[0], dev), _buffer_of(where, gmeta, sizes[1], dev),
                     _buffer_of(where, steps, sizes[2], dev))


def _activation(where: str, act: str) -> int:
    a = ACTIVATIONS.get(act)
    if a is None:
        raise QLinearError(QL_ERR_UNSUPPORTED, f"{where}: unknown activation {act!r}")
    return a


def _bytes_for(name: str, desc: Desc, M: int) -> int:
    d, n = desc.c(), C.c_size_t()
    _check(getattr(lib(), name)(C.byref(d), M, C.byref(n)), name)
    return n.value


@functools.lru_cache(maxsize=4096)
def _layer_plan(bytes_name: str, desc: Desc, M: int):
    """(C descriptor, its reference, packed sizes, workspace bytes) of a layer at M tokens."""
    need = _bytes_for(bytes_name, desc, M)
    d = desc.c()
    return d, C.byref(d), qlinear_packed_bytes(desc), need


@functools.lru_cache(maxsize=4096)
def _saved8_sizes(rows: int, cols: int):
    c, e = C.c_size_t(), C.c_size_t()
    _check(lib().qlinear_saved8_bytes(rows, cols, C.byref(c), C.byref(e)), "qlinear_saved8_bytes")
    return c.value, e.value


def _workspace_of(where: str, workspace, nbytes: int, dev: int, stream):
    """(tensor, address) of the caller's workspace, checked, or of one from the pool that torch's allocator keeps for
    the call's stream (so that it is handed on only to work behind this call's)."""
    import torch
    if workspace is None:
        with torch.cuda.stream(stream):  # None: the current one
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
    return workspace, _buffer_of(where, workspace, nbytes, dev)


@functools.lru_cache(maxsize=None)
def _current_raw_stream():
    """Device index -> address of its current stream: torch's own short way to it (a microsecond less a call than
    through a Stream object), or that object where a torch lacks it."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _run(where: str, dev: int, stream, f, *args):
    import torch
    if stream is None:
        s = _current_raw_stream()(dev)
    elif stream.device.index == dev:
        s = stream.cuda_stream
    else:
        raise QLinearError(QL_ERR_UNSUPPORTED, f"{where}: the stream belongs to another device than the tensors")
    if torch.cuda.current_device() == dev:
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status:
        raise QLinearError(status, where)


def qlinear_saved8_bytes(rows: int, cols: int):
    """Bytes of (codes, exps) of a [rows][cols] matrix in 8 bits."""
    return _saved8_sizes(rows, cols)


def alloc_saved8(rows: int, cols: int, device="cuda"):
    """Allocate (uninitialised) buffers of a [rows][cols] matrix in 8 bits: codes int8 [rows][cols rounded up to
    16] and exps uint8 [rows][that / 16].  A gated block's checkpoint has rows = 2 M, cols = F."""
    import torch
    c, e = _saved8_sizes(rows, cols)
    return (torch.empty((rows, c // rows), dtype=torch.int8, device=device),
            torch.empty((rows, e // rows), dtype=torch.uint8, device=device))


def _saved8_of(where: str, saved, rows: int, cols: int, dev: int) -> ql_saved8:
    import torch
    c, e = _saved8_sizes(rows, cols)
    return ql_saved8(_ptr_of(where, saved[0], torch.int8, c, dev), _ptr_of(where, saved[1], torch.uint8, e, dev))


def qlinear_save8(x, rows: int, cols: int, saved, stream=None):
    """bf16 [rows][cols] -> its 8-bit form in ``saved`` = (codes, exps) of alloc_saved8()."""
    import torch
    w = "qlinear_save8"
    dev = _device_of(w, x)
    s = _saved8_of(w, saved, rows, cols, dev)
    _run(w, dev, stream, lib().qlinear_save8, _ptr_of(w, x, torch.bfloat16, rows * cols, dev), rows, cols, C.byref(s))


def qlinear_restore8(saved, rows: int, cols: int, out, stream=None):
    """The 8-bit form -> bf16 [rows][cols]."""
    import torch
    w = "qlinear_restore8"
    dev = _device_of(w, out)
    s = _saved8_of(w, saved, rows, cols, dev)
    _run(w, dev, stream, lib().qlinear_restore8, C.byref(s), rows, cols,
         _ptr_of(w, out, torch.bfloat16, rows * cols, dev))


def qlinear_gated_workspace_bytes(desc: Desc, M: int) -> int:
    return _bytes_for("qlinear_gated_workspace_bytes", desc, M)


def alloc_gated_workspace(desc: Desc, M: int, device="cuda"):
    import torch
    return torch.empty(qlinear_gated_workspace_bytes(desc, M), dtype=torch.uint8, device=device)


def qlinear_gated(desc: Desc, codes, gmeta, steps, x, M: int, act: str, h, saved=None, workspace=None, stream=None):
    """h[M][F] = act(x Wg^T) * (x Wu^T) for a packed layer of F gate rows and then F up rows (desc.N = 2 F, as
    qlinear_concat_n stacks them).  ``act``: a key of ACTIVATIONS.  ``saved``: alloc_saved8(2 * M, F), where the
    8-bit checkpoint for qlinear_gated_backward goes.  ``workspace``: a uint8 CUDA tensor of at least
    qlinear_gated_workspace_bytes(desc, M) bytes; allocated here when omitted."""
    import torch
    w = "qlinear_gated"
    _, d, sizes, need = _layer_plan("qlinear_gated_workspace_bytes", desc, M)
    a, F, bf16 = _activation(w, act), desc.N // 2, torch.bfloat16
    dev = _device_of(w, x)
    xp, hp = _ptr_of(w, x, bf16, M * desc.K, dev), _ptr_of(w, h, bf16, M * F, dev)
    p = _packed_of(w, sizes, codes, gmeta, steps, dev)
    s = None if saved is None else C.byref(_saved8_of(w, saved, 2 * M, F, dev))
    workspace, wp = _workspace_of(w, workspace, need, dev, stream)
    _run(w, dev, stream, lib().qlinear_gated, d, C.byref(p), xp, M, a, hp, s, wp, need)


def qlinear_gemm_dx_workspace_bytes(desc: Desc, M: int) -> int:
    return _bytes_for("qlinear_gemm_dx_workspace_bytes", desc, M)


def alloc_gemm_dx_workspace(desc: Desc, M: int, device="cuda"):
    """Workspace of qlinear_gemm_dx and qlinear_gated_backward."""
    import torch
    return torch.empty(qlinear_gemm_dx_workspace_bytes(desc, M), dtype=torch.uint8, device=device)


def qlinear_gemm_dx(desc: Desc, codes, gmeta, steps, dy, M: int, dx, workspace=None, stream=None):
    """dx[M][K] = dy[M][N] W: the input gradient of the layer.  ``workspace``: a uint8 CUDA tensor of at least
    qlinear_gemm_dx_workspace_bytes(desc, M) bytes; allocated here when omitted."""
    import torch
    w = "qlinear_gemm_dx"
    _, d, sizes, need = _layer_plan("qlinear_gemm_dx_workspace_bytes", desc, M)
    dev, bf16 = _device_of(w, dy), torch.bfloat16
    yp, xp = _ptr_of(w, dy, bf16, M * desc.N, dev), _ptr_of(w, dx, bf16, M * desc.K, dev)
    p = _packed_of(w, sizes, codes, gmeta, steps, dev)
    workspace, wp = _workspace_of(w, workspace, need, dev, stream)
    _run(w, dev, stream, lib().qlinear_gemm_dx, d, C.byref(p), yp, M, xp, wp, need)


def qlinear_gated_backward(desc: Desc, codes, gmeta, steps, saved, dh, M: int, act: str, dx, dgu=None,
                           workspace=None, stream=None):
    """Backward pass of qlinear_gated from its checkpoint ``saved`` and the gradient dh[M][F]: dx[M][K], and
    (dg | du) in ``dgu`` [M][2 F] when given.  ``workspace``: as qlinear_gemm_dx."""
    import torch
    w = "qlinear_gated_backward"
    if desc.N % 2:
        raise QLinearError(QL_ERR_SHAPE, f"{w}: the layer has an odd number of rows")
    _, d, sizes, need = _layer_plan("qlinear_gemm_dx_workspace_bytes", desc, M)
    a, F, bf16 = _activation(w, act), desc.N // 2, torch.bfloat16
    dev = _device_of(w, dh)
    hp, xp = _ptr_of(w, dh, bf16, M * F, dev), _ptr_of(w, dx, bf16, M * desc.K, dev)
    gp = None if dgu is None else _ptr_of(w, dgu, bf16, M * desc.N, dev)
    p = _packed_of(w, sizes, codes, gmeta, steps, dev)
    s = _saved8_of(w, saved, 2 * M, F, dev)
    workspace, wp = _workspace_of(w, workspace, need, dev, stream)
    _run(w, dev, stream, lib().qlinear_gated_backward, d, C.byref(p), C.byref(s), hp, M, a, gp, xp, wp, need)


def qlinear_set_withhold_copies(on: bool) -> None:
    """Whether the current device's kernels start no copies, so that their first wait for data runs
    out (after about 1 s).  For tests of the give-up path (QL_ERR_TIMEOUT)."""
    _check(lib().qlinear_set_withhold_copies(1 if on else 0), "qlinear_set_withhold_copies")


def qlinear_sync_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status (QL_OK / QL_ERR_TIMEOUT / ...)."""
    return lib().qlinear_sync_status(_stream(stream))
