"""k3huf on GB300: lossless decode of bf16 weights whose high-byte plane is
Huffman coded (canonical, longest-first, 12-bit limit) and whose low-byte
plane is stored raw.

This module is a thin ctypes binding of the C ABI in ``include/k3huf.h``
(``_build/libk3huf.so``, built by ``_build.build()``): it only marshals
arguments.  Every step of the decode runs in the library's CUDA kernels;
there is no CPU fallback -- calls raise when the library is missing.
Device buffers and streams are plain pointers; torch tensors and streams
are accepted and converted with ``data_ptr()`` / ``cuda_stream``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import _build

OK, E_ARG, E_EMPTY, E_OVERSUB, E_BADLEN, E_FORMAT, E_CUDA, E_NOMEM, E_IO = 0, -1, -2, -3, -4, -5, -6, -7, -8
ST_BADCODE, ST_OVERRUN, ST_INDEX, ST_HEADER, ST_TIMEOUT, ST_TOKEN = 1, 2, 4, 8, 16, 32
MAXLEN = 12
STRIPE_VALUES = 1 << 25

EXPORTS = [
    "k3huf_build", "k3huf_layer_info", "k3huf_tensor_info", "k3huf_decode_layer", "k3huf_decode_layer_ws",
    "k3huf_decode_layer_ex", "k3huf_decode_tensor",
    "k3huf_decode_stripe",
    "k3huf_set_decoder_variant", "k3huf_encode_layer", "k3huf_ring_create", "k3huf_ring_run",
    "k3huf_ring_destroy", "k3huf_last_cuda_error", "k3huf_strerror", "k3huf_feed_open", "k3huf_feed_direct",
    "k3huf_feed_read", "k3huf_feed_close", "k3huf_ring_create_staged", "k3huf_ring_run_file",
    "k3huf_encode_scratch_bytes", "k3huf_encode_bound", "k3huf_encode_layer_gpu", "k3huf_gemv_layer",
    "k3huf_gemv_layer_ex", "k3huf_gemv_layer_batch", "k3huf_embed_layer", "k3huf_embed_grad_scratch_bytes",
    "k3huf_embed_grad", "k3huf_adapter_scratch_bytes", "k3huf_adapter_apply", "k3huf_adapter_grad",
    "k3huf_token_logprobs", "k3huf_token_logprobs_grad",
]
FILE_ALIGN = 4096


class K3HufError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = _lib().k3huf_strerror(code).decode() if _lib_handle is not None else str(code)
        if code == E_CUDA and _lib_handle is not None:
            msg += f" (cudaError {_lib_handle.k3huf_last_cuda_error()})"
        super().__init__(f"{what}: {msg} [{code}]" if what else f"{msg} [{code}]")


class LayerInfo(ctypes.Structure):
    _fields_ = [("chunk_syms", ctypes.c_uint32), ("n_tables", ctypes.c_uint32), ("n_tensors", ctypes.c_uint32),
                ("n_stripes", ctypes.c_uint32), ("raw_bytes", ctypes.c_uint64), ("blob_bytes", ctypes.c_uint64),
                ("out_bytes", ctypes.c_uint64), ("hdr_bytes", ctypes.c_uint32), ("stripe_values", ctypes.c_uint32),
                ("sub_syms", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class TensorInfo(ctypes.Structure):
    _fields_ = [("table", ctypes.c_uint32), ("first_stripe", ctypes.c_uint32), ("n_stripes", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("n_values", ctypes.c_uint64), ("out_offset", ctypes.c_uint64)]


class RingStats(ctypes.Structure):
    _fields_ = [("total_ms", ctypes.c_float), ("decode_ms", ctypes.c_float), ("copy_ms", ctypes.c_float),
                ("h2d_bytes", ctypes.c_uint64), ("out_bytes", ctypes.c_uint64)]


class FeedStats(ctypes.Structure):
    _fields_ = [("total_ms", ctypes.c_float), ("read_ms", ctypes.c_float), ("copy_ms", ctypes.c_float),
                ("decode_ms", ctypes.c_float), ("read_bytes", ctypes.c_uint64), ("out_bytes", ctypes.c_uint64)]


class Adapters(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("n_adapters", ctypes.c_uint32), ("rank", ctypes.c_uint32), ("cols", ctypes.c_uint64),
                ("rows", ctypes.c_uint64)]


_lib_handle = None
_lock = threading.Lock()
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t


def library_path() -> str:
    return _build.LIB


def _lib():
    """Load the library; raises if it was not built (no fallback)."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    with _lock:
        if _lib_handle is None:
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"k3huf CUDA library not built ({_build.LIB}); run "
                                   "lossless_bf16_weight_k3huf_gb300._build.build()")
            L = ctypes.CDLL(_build.LIB)
            L.k3huf_build.argtypes = [_vp, _vp]
            L.k3huf_layer_info.argtypes = [_vp, _sz, ctypes.POINTER(LayerInfo)]
            L.k3huf_tensor_info.argtypes = [_vp, _sz, ctypes.c_uint32, ctypes.POINTER(TensorInfo)]
            L.k3huf_decode_layer.argtypes = [_vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp]
            L.k3huf_decode_layer_ws.argtypes = [_vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp, _sz, _vp]
            L.k3huf_decode_layer_ex.argtypes = [_vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp, _sz, ctypes.c_uint32, _vp]
            L.k3huf_decode_tensor.argtypes = [_vp, _sz, _vp, _sz, ctypes.c_uint32, _vp, _sz, _vp, _vp, _sz,
                                              ctypes.c_uint32, _vp]
            L.k3huf_decode_stripe.argtypes = [_vp, ctypes.c_uint32, ctypes.c_uint32, _vp, _sz, ctypes.c_uint32, _vp,
                                              _vp, _vp]
            L.k3huf_set_decoder_variant.argtypes = [ctypes.c_int]
            L.k3huf_encode_layer.argtypes = [ctypes.c_uint32, ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_uint64),
                                             ctypes.c_uint32, ctypes.c_uint32, ctypes.c_int, ctypes.c_int, _vp, _sz,
                                             ctypes.POINTER(_sz)]
            L.k3huf_ring_create.argtypes = [_sz, ctypes.c_int, ctypes.POINTER(_vp)]
            L.k3huf_ring_run.argtypes = [_vp, ctypes.c_int, ctypes.POINTER(_vp), ctypes.POINTER(_sz),
                                         ctypes.POINTER(_vp), ctypes.POINTER(_sz), _vp, ctypes.POINTER(RingStats)]
            L.k3huf_ring_destroy.argtypes = [_vp]
            L.k3huf_encode_scratch_bytes.argtypes = [ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint32,
                                                     ctypes.c_uint32, ctypes.c_int, ctypes.POINTER(_sz)]
            L.k3huf_encode_bound.argtypes = [ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint32,
                                             ctypes.c_uint32, ctypes.c_int, ctypes.POINTER(_sz)]
            L.k3huf_encode_layer_gpu.argtypes = [ctypes.c_uint32, ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_uint64),
                                                 ctypes.c_uint32, ctypes.c_uint32, ctypes.c_int, _vp, _sz, _vp, _sz,
                                                 ctypes.POINTER(_sz), _vp]
            L.k3huf_gemv_layer.argtypes = [_vp, _sz, _vp, _sz, ctypes.c_uint32, ctypes.c_uint64, _vp, _vp, _vp, _vp]
            L.k3huf_gemv_layer_ex.argtypes = [_vp, _sz, _vp, _sz, ctypes.c_uint32, ctypes.c_uint64, _vp, _vp, _vp,
                                              ctypes.c_uint32, _vp]
            L.k3huf_gemv_layer_batch.argtypes = [_vp, _sz, _vp, _sz, ctypes.c_uint32, ctypes.c_uint64, _vp,
                                                 ctypes.c_uint32, _vp, _vp, ctypes.c_uint32, _vp]
            L.k3huf_feed_open.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.POINTER(_vp)]
            L.k3huf_feed_direct.argtypes = [_vp]
            L.k3huf_feed_read.argtypes = [_vp, ctypes.c_uint64, _sz, _vp, _sz]
            L.k3huf_feed_close.argtypes = [_vp]
            L.k3huf_ring_create_staged.argtypes = [_sz, ctypes.c_int, ctypes.POINTER(_vp)]
            L.k3huf_ring_run_file.argtypes = [_vp, _vp, ctypes.c_int, ctypes.POINTER(ctypes.c_uint64),
                                              ctypes.POINTER(_sz), ctypes.POINTER(_vp), ctypes.POINTER(_sz), _vp,
                                              ctypes.POINTER(FeedStats)]
            u32, u64, f32 = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float
            L.k3huf_embed_layer.argtypes = [_vp, _sz, _vp, _sz, u32, u64, _vp, u32, u64, f32, _vp, u32, u64, _vp, _vp]
            L.k3huf_embed_grad_scratch_bytes.argtypes = [u64, u64, u64, ctypes.POINTER(_sz)]
            L.k3huf_embed_grad.argtypes = [_vp, u32, u64, _vp, u32, u64, u64, u64, f32, _vp, _vp, _sz, _vp, u32, _vp]
            L.k3huf_adapter_scratch_bytes.argtypes = [u64, u32, u32, u64, u64, ctypes.c_int, ctypes.POINTER(_sz)]
            L.k3huf_adapter_apply.argtypes = [_vp, _vp, u64, _vp, u64, _vp, u64, _vp, u64, u32, _vp, _sz, _vp, _vp]
            L.k3huf_adapter_grad.argtypes = [_vp, _vp, u64, _vp, u64, _vp, u64, _vp, u64, _vp, u64, u32, _vp, _vp, _vp,
                                             _sz, _vp, u32, _vp]
            L.k3huf_token_logprobs.argtypes = [_vp, u32, u64, u64, u32, f32, _vp, u32, _vp, _vp, _vp, u32, _vp, _vp,
                                               _vp, _vp]
            L.k3huf_token_logprobs_grad.argtypes = [_vp, u32, u64, u64, u32, f32, _vp, u32, _vp, _vp, _vp, _vp, _vp,
                                                    u64, _vp, _vp]
            L.k3huf_strerror.restype = ctypes.c_char_p
            L.k3huf_strerror.argtypes = [ctypes.c_int]
            _lib_handle = L
    return _lib_handle


def _check(rc: int, what: str):
    if rc != OK:
        raise K3HufError(rc, what)


def _host(a) -> np.ndarray:
    if type(a) is np.ndarray and a.dtype == np.uint8 and a.ndim == 1 and a.flags.c_contiguous:
        return a
    if isinstance(a, (bytes, bytearray, memoryview)):
        return np.frombuffer(a, dtype=np.uint8)
    if hasattr(a, "numpy") and not isinstance(a, np.ndarray):      # torch CPU tensor
        a = a.numpy()
    return np.ascontiguousarray(a).view(np.uint8).reshape(-1)


def _dptr(x) -> int:
    """Device pointer of a CUDA tensor (or an int address)."""
    if isinstance(x, int):
        return x
    if getattr(x, "is_cuda", False):
        return int(x.data_ptr())
    raise TypeError("expected a CUDA tensor or a device address")


def _nbytes(x) -> int:
    if isinstance(x, int):
        raise TypeError("size needed for a raw address")
    return int(x.numel() * x.element_size())


_raw_stream = None      # torch's call for the current stream's address, once CUDA is initialised


def _stream(stream) -> int:
    global _raw_stream
    if isinstance(stream, int):
        return stream
    if stream is not None:
        return int(stream.cuda_stream)
    import torch
    if _raw_stream is None and torch.cuda.is_initialized():
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is not None:                          # (the address without a Stream object: 2 us less per call)
        return _raw_stream(torch._C._cuda_getDevice())
    return int(torch.cuda.current_stream().cuda_stream)


# ---------------------------------------------------------------------------

def build_table(codelen) -> np.ndarray:
    """The 4096-entry (symbol << 4) | length table of a code-length vector."""
    cl = np.zeros(256, dtype=np.uint8)
    cl[: len(codelen)] = np.asarray(codelen, dtype=np.uint8)
    out = np.zeros(4096, dtype=np.uint16)
    _check(_lib().k3huf_build(cl.ctypes.data, out.ctypes.data), "k3huf_build")
    return out


def check_table(codelen) -> int:
    """Return code of the Kraft check of a code-length vector."""
    cl = np.zeros(256, dtype=np.uint8)
    cl[: len(codelen)] = np.asarray(codelen, dtype=np.uint8)
    return int(_lib().k3huf_build(cl.ctypes.data, None))


def layer_info(hdr) -> dict:
    h = _host(hdr)
    info = LayerInfo()
    _check(_lib().k3huf_layer_info(h.ctypes.data, h.size, ctypes.byref(info)), "k3huf_layer_info")
    return {f: getattr(info, f) for f, _ in LayerInfo._fields_}


def tensor_info(hdr, t: int) -> dict:
    h = _host(hdr)
    ti = TensorInfo()
    _check(_lib().k3huf_tensor_info(h.ctypes.data, h.size, t, ctypes.byref(ti)), "k3huf_tensor_info")
    return {f: getattr(ti, f) for f, _ in TensorInfo._fields_}


def encode_layer(tensors, chunk_syms: int = 4096, shared_table: bool = False, threads: int = 0,
                 out: np.ndarray | None = None, sub_syms: int = 256) -> np.ndarray:
    """Container bytes of a layer of bf16 tensors (numpy uint16 / torch bf16
    CPU); chunk_syms values per indexed chunk, sub_syms per sub-stream."""
    arrs = []
    for t in tensors:
        if hasattr(t, "view") and hasattr(t, "dtype") and str(getattr(t, "dtype", "")) == "torch.bfloat16":
            import torch
            t = t.contiguous().view(torch.int16).numpy().view(np.uint16)
        arrs.append(np.ascontiguousarray(t).reshape(-1).view(np.uint16))
    n = len(arrs)
    ptrs = (_vp * n)(*[a.ctypes.data for a in arrs])
    nv = (ctypes.c_uint64 * n)(*[a.size for a in arrs])
    size = _sz(0)
    L = _lib()
    _check(L.k3huf_encode_layer(n, ptrs, nv, chunk_syms, sub_syms, int(shared_table), threads, None, 0,
                                ctypes.byref(size)), "k3huf_encode_layer")
    if out is None:
        out = np.empty(size.value, dtype=np.uint8)
    elif out.size < size.value:
        raise ValueError("output buffer too small")
    _check(L.k3huf_encode_layer(n, ptrs, nv, chunk_syms, sub_syms, int(shared_table), threads, out.ctypes.data,
                                out.size, ctypes.byref(size)), "k3huf_encode_layer")
    return out[: size.value]


def encode_scratch_bytes(n_values, chunk_syms: int = 4096, sub_syms: int = 256, shared_table: bool = False) -> int:
    """Device scratch bytes that encode_layer_gpu needs for tensors of these sizes."""
    n = len(n_values)
    nv = (ctypes.c_uint64 * n)(*[int(v) for v in n_values])
    out = _sz(0)
    _check(_lib().k3huf_encode_scratch_bytes(n, nv, chunk_syms, sub_syms, int(shared_table), ctypes.byref(out)),
           "k3huf_encode_scratch_bytes")
    return int(out.value)


def encode_bound(sizes, chunk_syms: int = 4096, sub_syms: int = 256, shared_table: bool = False) -> int:
    """Bytes that hold the container of tensors of these sizes whatever their
    values (k3huf_encode_bound)."""
    n = len(sizes)
    nv = (ctypes.c_uint64 * n)(*[int(x) for x in sizes])
    out = _sz(0)
    _check(_lib().k3huf_encode_bound(n, nv, chunk_syms, sub_syms, int(shared_table), ctypes.byref(out)),
           "k3huf_encode_bound")
    return int(out.value)


def encode_layer_gpu(tensors, chunk_syms: int = 4096, sub_syms: int = 256, shared_table: bool = False,
                     stream=None, scratch=None, out=None):
    """Container of a layer of bf16 CUDA tensors (16-byte aligned), built on
    the GPU; returns a CUDA uint8 tensor.  ``scratch`` (a CUDA tensor) is
    allocated here when not given.  ``out``: a CUDA uint8 tensor of at least
    encode_bound(...) bytes, 256-byte aligned; the container is encoded in
    one call into its first bytes and that prefix is returned (without
    ``out``, a first call sizes the container and a second fills a tensor
    of exactly that size)."""
    import torch
    n = len(tensors)
    sizes = [int(t.numel()) for t in tensors]
    dev = tensors[0].device
    if scratch is None:
        scratch = torch.empty(encode_scratch_bytes(sizes, chunk_syms, sub_syms, shared_table), dtype=torch.uint8,
                              device=dev)
    ptrs = (_vp * n)(*[int(t.data_ptr()) for t in tensors])
    nv = (ctypes.c_uint64 * n)(*sizes)
    size = _sz(0)
    L = _lib()
    s = _stream(stream)
    if out is not None:
        _check(L.k3huf_encode_layer_gpu(n, ptrs, nv, chunk_syms, sub_syms, int(shared_table), _dptr(scratch),
                                        _nbytes(scratch), _dptr(out), _nbytes(out), ctypes.byref(size), s),
               "k3huf_encode_layer_gpu")
        return out[: size.value]
    _check(L.k3huf_encode_layer_gpu(n, ptrs, nv, chunk_syms, sub_syms, int(shared_table), _dptr(scratch),
                                    _nbytes(scratch), None, 0, ctypes.byref(size), s), "k3huf_encode_layer_gpu")
    blob = torch.empty(size.value, dtype=torch.uint8, device=dev)
    _check(L.k3huf_encode_layer_gpu(n, ptrs, nv, chunk_syms, sub_syms, int(shared_table), _dptr(scratch),
                                    _nbytes(scratch), _dptr(blob), _nbytes(blob), ctypes.byref(size), s),
           "k3huf_encode_layer_gpu")
    return blob


WORK_BYTES = 68
DECODE_EARLY_START = 1


def decode_layer(hdr, d_layer, d_out, d_status, stream=None, layer_bytes: int | None = None,
                 out_bytes: int | None = None, work=None, early_start: bool = False) -> None:
    """Launch the decode of a layer; asynchronous on ``stream``.  ``work``: a
    zeroed device buffer of at least WORK_BYTES that no other launch uses
    meanwhile (k3huf_decode_layer_ws: the end of the launch is spread over
    all CTAs), or None.  ``early_start`` (k3huf_decode_layer_ex): the launch
    may begin while the kernel before it in the stream finishes; that kernel
    must not write ``d_layer``."""
    h = _host(hdr)
    lb = _nbytes(d_layer) if layer_bytes is None else layer_bytes
    ob = _nbytes(d_out) if out_bytes is None else out_bytes
    if early_start:
        _check(_lib().k3huf_decode_layer_ex(h.ctypes.data, h.size, _dptr(d_layer), lb, _dptr(d_out), ob,
                                            _dptr(d_status), None if work is None else _dptr(work),
                                            0 if work is None else _nbytes(work), DECODE_EARLY_START,
                                            _stream(stream)), "k3huf_decode_layer_ex")
    elif work is None:
        _check(_lib().k3huf_decode_layer(h.ctypes.data, h.size, _dptr(d_layer), lb, _dptr(d_out), ob,
                                         _dptr(d_status), _stream(stream)), "k3huf_decode_layer")
    else:
        _check(_lib().k3huf_decode_layer_ws(h.ctypes.data, h.size, _dptr(d_layer), lb, _dptr(d_out), ob,
                                            _dptr(d_status), _dptr(work), _nbytes(work), _stream(stream)),
               "k3huf_decode_layer_ws")


def decode_tensor(hdr, d_layer, tensor: int, d_out, d_status, stream=None, layer_bytes: int | None = None,
                  out_bytes: int | None = None, work=None, early_start: bool = False) -> None:
    """Launch the decode of one tensor of a layer (k3huf_decode_tensor):
    ``d_out`` receives its bf16 bytes from offset 0.  ``work`` and
    ``early_start`` as for decode_layer."""
    h = _host(hdr)
    lb = _nbytes(d_layer) if layer_bytes is None else layer_bytes
    ob = _nbytes(d_out) if out_bytes is None else out_bytes
    _check(_lib().k3huf_decode_tensor(h.ctypes.data, h.size, _dptr(d_layer), lb, int(tensor), _dptr(d_out), ob,
                                      _dptr(d_status), None if work is None else _dptr(work),
                                      0 if work is None else _nbytes(work),
                                      DECODE_EARLY_START if early_start else 0, _stream(stream)),
           "k3huf_decode_tensor")


GEMV_ZERO_Y = 2


def gemv_layer(hdr, d_layer, tensor: int, cols: int, d_x, d_y, d_status, stream=None,
               layer_bytes: int | None = None, zero_y: bool = False, early_start: bool = False) -> None:
    """y += W x with tensor ``tensor`` of the layer as a row-major matrix of
    ``cols`` columns, decoded on chip (never written out); asynchronous.
    ``zero_y``: y = W x (the call zeroes y first); ``early_start``: the
    call's kernels may begin while the kernel before them finishes, which
    must not write ``d_layer`` (k3huf_gemv_layer_ex)."""
    h = _host(hdr)
    lb = _nbytes(d_layer) if layer_bytes is None else layer_bytes
    flags = (GEMV_ZERO_Y if zero_y else 0) | (DECODE_EARLY_START if early_start else 0)
    if flags:
        _check(_lib().k3huf_gemv_layer_ex(h.ctypes.data, h.size, _dptr(d_layer), lb, tensor, cols, _dptr(d_x),
                                          _dptr(d_y), _dptr(d_status), flags, _stream(stream)), "k3huf_gemv_layer_ex")
        return
    _check(_lib().k3huf_gemv_layer(h.ctypes.data, h.size, _dptr(d_layer), lb, tensor, cols, _dptr(d_x), _dptr(d_y),
                                   _dptr(d_status), _stream(stream)), "k3huf_gemv_layer")


def gemv_layer_batch(hdr, d_layer, tensor: int, cols: int, d_x, d_y, d_status, stream=None,
                     layer_bytes: int | None = None, zero_y: bool = False, early_start: bool = False) -> None:
    """Y += W X for several vectors with one decode of W (k3huf_gemv_layer_batch):
    ``d_x`` a CUDA bf16 tensor of n_vec x cols (n_vec 1, 2, 4 or 8), ``d_y`` a
    CUDA float32 tensor of n_vec x rows; ``zero_y``: Y = W X."""
    h = _host(hdr)
    lb = _nbytes(d_layer) if layer_bytes is None else layer_bytes
    n_vec = _nbytes(d_x) // (2 * cols)
    flags = (GEMV_ZERO_Y if zero_y else 0) | (DECODE_EARLY_START if early_start else 0)
    _check(_lib().k3huf_gemv_layer_batch(h.ctypes.data, h.size, _dptr(d_layer), lb, tensor, cols, _dptr(d_x), n_vec,
                                         _dptr(d_y), _dptr(d_status), flags, _stream(stream)),
           "k3huf_gemv_layer_batch")


def decode_stripe(codelen, chunk_syms: int, sub_syms: int, d_stripe, stripe_bytes: int, n_values: int, d_out,
                  d_status, stream=None) -> None:
    cl = np.zeros(256, dtype=np.uint8)
    cl[: len(codelen)] = np.asarray(codelen, dtype=np.uint8)
    _check(_lib().k3huf_decode_stripe(cl.ctypes.data, chunk_syms, sub_syms, _dptr(d_stripe), stripe_bytes, n_values,
                                      _dptr(d_out), _dptr(d_status), _stream(stream)), "k3huf_decode_stripe")


def set_decoder_variant(variant: int) -> None:
    """Codes per lockstep table lookup: 0 = default (2), 1 or 2."""
    _check(_lib().k3huf_set_decoder_variant(variant), "k3huf_set_decoder_variant")


# --- operators next to the coded weights ---------------------------------------
# Tensors are CUDA tensors; a matrix's rows may be any stride apart, its columns
# are adjacent.  The calls are asynchronous on ``stream`` (the current one) and
# OR faults into ``d_status`` (an int32 CUDA tensor) as the decode calls do.

MAX_RANK, MAX_TOP = 128, 64
ACCUMULATE = 4
_BF16, _F32 = 0, 1


_types = None           # (element types by dtype, id sizes by dtype, fp32, int32, bf16), filled at the first call


def _dtypes():
    global _types
    if _types is None:
        import torch
        _types = ({torch.bfloat16: _BF16, torch.float32: _F32}, {torch.int32: 4, torch.int64: 8}, torch.float32, torch.int32,
                  torch.bfloat16)
    return _types


def _matrix(t, n: int, cols: int, what: str, elem: int | None = None):
    """(address, element type, row stride) of a bf16 or fp32 CUDA matrix of n rows."""
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    e = _dtypes()[0].get(t.dtype)
    if e is None or (elem is not None and e != elem):
        raise TypeError(f"{what}: wrong element type {t.dtype}")
    if t.shape != (n, cols):
        raise ValueError(f"{what}: expected shape {(n, cols)}, got {tuple(t.shape)}")
    rows, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: columns must be adjacent")
    return t.data_ptr(), e, rows if n > 1 else max(rows, cols)


def _dense(t, shape, what: str, dtype):
    """Address of a contiguous CUDA tensor of this shape and dtype."""
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _ids(t, what: str = "ids"):
    """(address, bytes per id, count) of a contiguous int32 or int64 CUDA vector."""
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    size = _dtypes()[1].get(t.dtype)
    if size is None:
        raise TypeError(f"{what}: expected int32 or int64, got {t.dtype}")
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous vector")
    return t.data_ptr(), size, t.numel()


def embed_layer(hdr, d_layer, tensor: int, cols: int, ids, out, d_status, scale: float = 1.0, stream=None,
                layer_bytes: int | None = None) -> None:
    """out[t] = scale * W[ids[t]] for tensor ``tensor`` of the layer as a table of
    ``cols`` columns (k3huf_embed_layer): only what the rows meet is decoded.
    ``ids``: int32 or int64, negative for a row of zeros; ``out``: bf16 or fp32,
    len(ids) x cols."""
    h = _host(hdr)
    lb = _nbytes(d_layer) if layer_bytes is None else layer_bytes
    ip, ib, n = _ids(ids)
    op, oe, os_ = _matrix(out, n, cols, "out")
    _check(_lib().k3huf_embed_layer(h.__array_interface__["data"][0], h.size, _dptr(d_layer), lb, int(tensor), cols, ip, ib, n, scale,
                                    op, oe, os_, _dptr(d_status), _stream(stream)), "k3huf_embed_layer")


def embed_grad_scratch_bytes(n_tokens: int, rows: int, cols: int) -> int:
    """Device scratch bytes of embed_grad."""
    out = _sz(0)
    _check(_lib().k3huf_embed_grad_scratch_bytes(n_tokens, rows, cols, ctypes.byref(out)),
           "k3huf_embed_grad_scratch_bytes")
    return int(out.value)


def embed_grad(ids, dy, grad, scratch, d_status, scale: float = 1.0, accumulate: bool = False, stream=None) -> None:
    """grad[v] = scale * (sum of dy[t] over the tokens with ids[t] = v), rows
    without a token zero (k3huf_embed_grad); ``accumulate``: added to grad.
    ``dy``: bf16 or fp32, len(ids) x cols; ``grad``: fp32, rows x cols."""
    ip, ib, n = _ids(ids)
    rows, cols = grad.shape
    gp = _dense(grad, (rows, cols), "grad", _dtypes()[2])
    dp, de, ds = _matrix(dy, n, cols, "dy")
    _check(_lib().k3huf_embed_grad(ip, ib, n, dp, de, ds, rows, cols, scale, gp, _dptr(scratch), _nbytes(scratch),
                                   _dptr(d_status), ACCUMULATE if accumulate else 0, _stream(stream)),
           "k3huf_embed_grad")


def adapter_scratch_bytes(n_tokens: int, n_adapters: int, rank: int, cols: int, rows: int, grad: bool = False) -> int:
    """Device scratch bytes of adapter_apply, or of adapter_grad."""
    out = _sz(0)
    _check(_lib().k3huf_adapter_scratch_bytes(n_tokens, n_adapters, rank, cols, rows, int(grad), ctypes.byref(out)),
           "k3huf_adapter_scratch_bytes")
    return int(out.value)


def _adapters(a, b, scales) -> Adapters:
    n, rank, cols = a.shape
    rows = b.shape[2]
    _, _, f32, _, bf16 = _dtypes()
    return Adapters(_dense(a, (n, rank, cols), "a", bf16), _dense(b, (n, rank, rows), "b", bf16), _dense(scales, (n,), "scales", f32),
                    n, rank, cols, rows)


def adapter_apply(x, a, b, ids, scales, y, scratch, d_status, base=None, stream=None) -> None:
    """y[t] = base[t] + scales[i] (x[t] a[i]^T) b[i] with i = ids[t], base alone
    where ids[t] < 0 (k3huf_adapter_apply).  ``a``: bf16, adapters x rank x cols;
    ``b``: bf16, adapters x rank x rows; ``ids``: int32; ``y``: fp32 or bf16;
    ``base``: of y's type, may be y, None for zero."""
    ad = _adapters(a, b, scales)
    n = ids.numel()
    ip = _dense(ids, (n,), "ids", _dtypes()[3])
    xp, _, xs = _matrix(x, n, ad.cols, "x", _BF16)
    yp, ye, ys = _matrix(y, n, ad.rows, "y")
    bp, _, bs = (None, ye, 0) if base is None else _matrix(base, n, ad.rows, "base", ye)
    _check(_lib().k3huf_adapter_apply(ctypes.addressof(ad), xp, xs, ip, n, bp, bs, yp, ys, ye, _dptr(scratch),
                                      _nbytes(scratch), _dptr(d_status), _stream(stream)), "k3huf_adapter_apply")


def adapter_grad(x, a, b, ids, scales, dy, da, db, scratch, d_status, dx=None, dx_base=None, accumulate: bool = False,
                 stream=None) -> None:
    """Gradients of adapter_apply for the bf16 gradient ``dy`` (k3huf_adapter_grad):
    ``da``, ``db`` fp32, shaped as a and b (``accumulate``: added to); ``dx`` (fp32
    or bf16, None if not wanted) = dx_base + the adapters' part."""
    ad = _adapters(a, b, scales)
    n = ids.numel()
    _, _, f32, i32, _ = _dtypes()
    ip = _dense(ids, (n,), "ids", i32)
    xp, _, xs = _matrix(x, n, ad.cols, "x", _BF16)
    yp, _, ys = _matrix(dy, n, ad.rows, "dy", _BF16)
    if dx is None and dx_base is not None:
        raise ValueError("dx_base without dx")
    dp, de, ds = (None, _BF16, 0) if dx is None else _matrix(dx, n, ad.cols, "dx")
    bp, _, bs = (None, de, 0) if dx_base is None else _matrix(dx_base, n, ad.cols, "dx_base", de)
    _check(_lib().k3huf_adapter_grad(ctypes.addressof(ad), xp, xs, ip, n, yp, ys, bp, bs, dp, ds, de,
                                     _dense(da, a.shape, "da", f32),
                                     _dense(db, b.shape, "db", f32), _dptr(scratch),
                                     _nbytes(scratch), _dptr(d_status), ACCUMULATE if accumulate else 0,
                                     _stream(stream)), "k3huf_adapter_grad")


def token_logprobs(logits, tokens, logprob, d_status, entropy=None, lse=None, top_ids=None, top_logprobs=None,
                   scale: float = 1.0, stream=None) -> None:
    """Log probabilities of one token per row under softmax(scale * logits), with
    entropy, log-sum-exp and the largest logits (k3huf_token_logprobs).
    ``logits``: bf16 or fp32, n x vocab; ``tokens``: int32 or int64, negative for
    an unscored row; outputs fp32 of n, ``top_ids`` int32 and ``top_logprobs`` fp32
    of n x top (both or neither)."""
    tp, tb, n = _ids(tokens, "tokens")
    vocab = logits.shape[1]
    xp, xe, xs = _matrix(logits, n, vocab, "logits")
    _, _, f32, i32, _ = _dtypes()
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    top, ti, tl = 0, None, None
    if top_ids is not None:
        top = top_ids.shape[1]
        ti, tl = _dense(top_ids, (n, top), "top_ids", i32), _dense(top_logprobs, (n, top), "top_logprobs", f32)
    _check(_lib().k3huf_token_logprobs(xp, xe, xs, n, vocab, scale, tp, tb, _dense(logprob, (n,), "logprob", f32),
                                       None if entropy is None else _dense(entropy, (n,), "entropy", f32),
                                       None if lse is None else _dense(lse, (n,), "lse", f32), top, ti, tl,
                                       _dptr(d_status), _stream(stream)), "k3huf_token_logprobs")


def token_logprobs_grad(logits, tokens, lse, g_logprob, dlogits, d_status, entropy=None, g_entropy=None,
                        scale: float = 1.0, stream=None) -> None:
    """Gradient of token_logprobs with respect to the logits
    (k3huf_token_logprobs_grad), for the gradients of the log probabilities and
    (with ``entropy`` as the forward gave it) of the entropies.  ``dlogits``: as
    logits, may be logits itself."""
    tp, tb, n = _ids(tokens, "tokens")
    vocab = logits.shape[1]
    xp, xe, xs = _matrix(logits, n, vocab, "logits")
    dp, _, ds = _matrix(dlogits, n, vocab, "dlogits", xe)
    f32 = _dtypes()[2]
    _check(_lib().k3huf_token_logprobs_grad(xp, xe, xs, n, vocab, scale, tp, tb, _dense(lse, (n,), "lse", f32),
                                            None if entropy is None else _dense(entropy, (n,), "entropy", f32),
                                            _dense(g_logprob, (n,), "g_logprob", f32),
                                            None if g_entropy is None else _dense(g_entropy, (n,), "g_entropy", f32),
                                            dp, ds, _dptr(d_status), _stream(stream)), "k3huf_token_logprobs_grad")


class Feed:
    """A container file opened for the storage feed (O_DIRECT where the
    filesystem allows it), read with parallel preads."""

    def __init__(self, path: str, threads: int = 8):
        self._h = _vp()
        _check(_lib().k3huf_feed_open(os.fsencode(path), threads, ctypes.byref(self._h)), "k3huf_feed_open")

    @property
    def direct(self) -> bool:
        return _lib().k3huf_feed_direct(self._h) == 1

    def read(self, offset: int, nbytes: int, buf, buf_bytes: int | None = None) -> None:
        """Read into host memory at ``buf`` (an address or a numpy/torch CPU
        buffer); offset and the buffer 4096-byte aligned."""
        if isinstance(buf, int):
            addr, cap = buf, buf_bytes
        elif hasattr(buf, "data_ptr"):
            addr, cap = int(buf.data_ptr()), _nbytes(buf)
        else:
            addr, cap = buf.ctypes.data, buf.nbytes
        _check(_lib().k3huf_feed_read(self._h, offset, nbytes, addr, cap), "k3huf_feed_read")

    def close(self):
        if self._h:
            _lib().k3huf_feed_close(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def aligned_host(nbytes: int, align: int = FILE_ALIGN) -> np.ndarray:
    """A uint8 host array of nbytes whose first byte is align-aligned."""
    raw = np.empty(nbytes + align, dtype=np.uint8)
    off = (-raw.ctypes.data) % align
    return raw[off: off + nbytes]


def write_layers(path: str, blobs) -> list:
    """Write containers back to back into a file, each at a 4096-aligned
    offset; returns the offsets."""
    offs, pos = [], 0
    with open(path, "wb") as f:
        for b in blobs:
            b = _host(b)
            offs.append(pos)
            f.write(b.tobytes())
            pos += b.size
            pad = (-pos) % FILE_ALIGN
            f.write(b"\0" * pad)
            pos += pad
        f.flush()
        os.fsync(f.fileno())
    return offs


class Ring:
    """Pinned-host -> HBM double-buffered feed of layers into the decoder.
    ``staged=True`` also allocates pinned host slots, for ``run_file``."""

    def __init__(self, slot_bytes: int, n_slots: int = 2, staged: bool = False):
        self._h = _vp()
        create = _lib().k3huf_ring_create_staged if staged else _lib().k3huf_ring_create
        _check(create(slot_bytes, n_slots, ctypes.byref(self._h)), "k3huf_ring_create")

    def run_file(self, feed: "Feed", offsets, sizes, d_outs, d_status) -> dict:
        """Decode the containers stored in the feed's file at ``offsets``
        (``sizes`` bytes each) into ``d_outs`` (CUDA tensors)."""
        n = len(offsets)
        op = (ctypes.c_uint64 * n)(*[int(o) for o in offsets])
        sp = (_sz * n)(*[int(x) for x in sizes])
        dp = (_vp * n)(*[_dptr(d) for d in d_outs])
        db = (_sz * n)(*[_nbytes(d) for d in d_outs])
        st = FeedStats()
        _check(_lib().k3huf_ring_run_file(self._h, feed._h, n, op, sp, dp, db, _dptr(d_status), ctypes.byref(st)),
               "k3huf_ring_run_file")
        return {f: getattr(st, f) for f, _ in FeedStats._fields_}

    def run(self, h_layers, d_outs, d_status) -> dict:
        """h_layers: pinned host uint8 tensors (containers); d_outs: CUDA tensors."""
        n = len(h_layers)
        hp = (_vp * n)(*[int(h.data_ptr()) for h in h_layers])
        hb = (_sz * n)(*[_nbytes(h) for h in h_layers])
        dp = (_vp * n)(*[_dptr(d) for d in d_outs])
        db = (_sz * n)(*[_nbytes(d) for d in d_outs])
        st = RingStats()
        _check(_lib().k3huf_ring_run(self._h, n, hp, hb, dp, db, _dptr(d_status), ctypes.byref(st)),
               "k3huf_ring_run")
        return {f: getattr(st, f) for f, _ in RingStats._fields_}

    def close(self):
        if self._h:
            _lib().k3huf_ring_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def last_cuda_error() -> int:
    return int(_lib().k3huf_last_cuda_error())


def strerror(code: int) -> str:
    return _lib().k3huf_strerror(code).decode()
