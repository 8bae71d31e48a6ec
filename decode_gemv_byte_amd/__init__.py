"""Python binding of libnwc -- lossless BF16 weight compression decoded inside
the matrix-vector kernel, for MI355X (gfx950).

Argument marshalling only: every step runs in the native library
(``libnwc.so``: C++ host codec + HIP kernels).  The functions carry the names
of the C ABI in ``include/nwc.h``.  Host buffers are numpy arrays; device
buffers are torch CUDA tensors (PyTorch provides device memory and streams).
Importing fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnwc.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libnwc.so is not built; run `python decode_gemv_byte_amd/build.py` "
                      "(or __graft_entry__.build())")

# The binding hands torch tensors' device memory and streams to the library,
# so both must run on one HIP runtime.  PyTorch ships its own copy of it;
# with torch loaded first, the library's dependency on the runtime's soname
# resolves to that copy.  Loaded the other way round, the library would map
# the ROCm install's runtime and torch would then map its own beside it: two
# runtimes (and two HSA runtimes) in one process, under which torch's
# streams and allocations are foreign handles and launches fail.
try:
    import torch  # noqa: F401
except ImportError:   # a torch-free caller of the C ABI: the ROCm install's runtime
    pass

_lib = ctypes.CDLL(LIB_PATH)

NWC_OK = 0
NWC_ERR_INVALID_ARG = -1
NWC_ERR_BUFFER_TOO_SMALL = -2
NWC_ERR_BAD_FORMAT = -3
NWC_ERR_UNSUPPORTED = -4
NWC_ERR_ALIGNMENT = -5
NWC_ERR_HIP = -6
NWC_ERR_SCRATCH_LIMIT = -7
NWC_OUT_BF16 = 0
NWC_OUT_F32 = 1
NWC_ROPE_HALF = 0
NWC_ROPE_PAIRS = 1


class nwc_params(ctypes.Structure):
    _fields_ = [("tile_rows", ctypes.c_uint32), ("tile_cols", ctypes.c_uint32),
                ("chunks_per_tile", ctypes.c_uint32), ("max_code_len", ctypes.c_uint32),
                ("pair_fit", ctypes.c_uint32), ("code_family", ctypes.c_uint32)]


class nwc_info(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64), ("blob_bytes", ctypes.c_uint64),
                ("tile_rows", ctypes.c_uint32), ("tile_cols", ctypes.c_uint32),
                ("chunks_per_tile", ctypes.c_uint32), ("max_code_len", ctypes.c_uint32),
                ("n_tiles", ctypes.c_uint64), ("n_chunks", ctypes.c_uint64), ("raw_ld", ctypes.c_uint64),
                ("stream_words", ctypes.c_uint64), ("off_code_len", ctypes.c_uint64),
                ("off_table", ctypes.c_uint64), ("off_tile_words", ctypes.c_uint64),
                ("off_chunk_bits", ctypes.c_uint64), ("off_raw", ctypes.c_uint64),
                ("off_stream", ctypes.c_uint64), ("max_tile_words", ctypes.c_uint32),
                ("n_symbols", ctypes.c_uint32), ("max_chunk_bits", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("payload_bits", ctypes.c_uint64),
                ("code_len", ctypes.c_uint8 * 256)]


class nwc_heads(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("ld_src", ctypes.c_uint64), ("ld_dst", ctypes.c_uint64), ("heads", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class nwc_rope(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("dims", ctypes.c_uint32), ("style", ctypes.c_uint32)]


class nwc_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_uint64),
                ("page_stride", ctypes.c_uint64), ("kv_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32),
                ("page_len", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class nwc_page_table(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("ld", ctypes.c_uint64), ("rows", ctypes.c_uint32), ("cols", ctypes.c_uint32)]


class nwc_groups(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p), ("len", ctypes.c_void_p), ("count", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class NwcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, nwc_status_str(status)))


_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32
_i = ctypes.c_int
_st = ctypes.c_int

_lib.nwc_status_str.argtypes = [_st]
_lib.nwc_status_str.restype = ctypes.c_char_p
_lib.nwc_encode_bound.argtypes = [_u64, _u64, ctypes.POINTER(nwc_params), ctypes.POINTER(_sz)]
_lib.nwc_encode.argtypes = [_vp, _u64, _u64, _u64, ctypes.POINTER(nwc_params), _vp, _sz, ctypes.POINTER(_sz)]
_lib.nwc_inspect.argtypes = [_vp, _sz, ctypes.POINTER(nwc_info)]
_lib.nwc_decode.argtypes = [ctypes.POINTER(nwc_info), _vp, _vp, _u64, _vp]
_lib.nwc_workspace_size.argtypes = [ctypes.POINTER(nwc_info), _i, ctypes.POINTER(_sz)]
_lib.nwc_gemv.argtypes = [ctypes.POINTER(nwc_info), _vp, _vp, _vp, _i, _vp, _sz, _vp]
_lib.nwc_gemm_skinny.argtypes = [ctypes.POINTER(nwc_info), _vp, _vp, _u64, _i, _vp, _u64, _i, _vp, _sz, _vp]
_lib.nwc_bf16_workspace_size.argtypes = [_u64, _u64, ctypes.POINTER(_sz)]
_lib.nwc_gemv_bf16.argtypes = [_vp, _u64, _u64, _u64, _vp, _vp, _i, _vp, _sz, _vp]
_lib.nwc_gemv_batched.argtypes = [_i, ctypes.POINTER(nwc_info), ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                  ctypes.POINTER(_vp), _i, _vp, _sz, _vp]
_lib.nwc_decode_batched.argtypes = [_i, ctypes.POINTER(nwc_info), ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                    ctypes.POINTER(_u64), _vp]
_lib.nwc_gather_rows.argtypes = [ctypes.POINTER(nwc_info), _vp, _vp, _u32, _vp, _u64, _vp]
_lib.nwc_blas_create.argtypes = [ctypes.POINTER(_vp)]
_lib.nwc_blas_destroy.argtypes = [_vp]
_lib.nwc_prefill_workspace_size.argtypes = [ctypes.POINTER(nwc_info), ctypes.POINTER(_sz)]
_lib.nwc_gemm_prefill.argtypes = [_vp, ctypes.POINTER(nwc_info), _vp, _vp, _u64, _i, _vp, _u64, _i, _vp, _sz, _vp]
_lib.nwc_read_probe.argtypes = [_vp, _sz, _vp, _u32, _i, _vp]
_lib.nwc_noalloc_scratch_bytes.argtypes = [ctypes.POINTER(_sz)]
_lib.nwc_gemv_noalloc.argtypes = [ctypes.POINTER(nwc_info), _vp, _vp, _vp, _i, _vp]
_lib.nwc_set_wait_limit.argtypes = [_u32]
_f32 = ctypes.c_float
_lib.nwc_qk_norm_rope.argtypes = [ctypes.POINTER(nwc_heads), ctypes.POINTER(nwc_heads), _u32, _u32, _f32,
                                  ctypes.POINTER(nwc_rope), _vp, _vp]
_lib.nwc_kv_append.argtypes = [ctypes.POINTER(nwc_cache), ctypes.POINTER(nwc_page_table), ctypes.POINTER(nwc_heads),
                               _vp, _u64, ctypes.POINTER(nwc_heads), _u32, _f32, ctypes.POINTER(nwc_rope), _vp, _vp, _vp]
_lib.nwc_attend_workspace_size.argtypes = [ctypes.POINTER(nwc_cache), _u32, _u32, _u32, ctypes.POINTER(_sz)]
_lib.nwc_attend.argtypes = [ctypes.POINTER(nwc_cache), ctypes.POINTER(nwc_page_table), ctypes.POINTER(nwc_groups), _vp,
                            _vp, _u64, _u32, _f32, _vp, _u64, _vp, _sz, _vp]
for _f in ("nwc_encode_bound", "nwc_encode", "nwc_inspect", "nwc_decode", "nwc_workspace_size", "nwc_gemv",
           "nwc_gemm_skinny", "nwc_bf16_workspace_size", "nwc_gemv_bf16", "nwc_gemv_batched", "nwc_decode_batched",
           "nwc_blas_create", "nwc_blas_destroy", "nwc_prefill_workspace_size", "nwc_gemm_prefill",
           "nwc_gather_rows", "nwc_read_probe", "nwc_noalloc_scratch_bytes", "nwc_gemv_noalloc",
           "nwc_set_wait_limit", "nwc_qk_norm_rope", "nwc_kv_append", "nwc_attend_workspace_size", "nwc_attend"):
    getattr(_lib, _f).restype = _st

# the exported C symbols, for checks against include/nwc.h
EXPORTS = ("nwc_status_str", "nwc_encode_bound", "nwc_encode", "nwc_inspect", "nwc_decode",
           "nwc_workspace_size", "nwc_gemv", "nwc_gemm_skinny", "nwc_bf16_workspace_size", "nwc_gemv_bf16",
           "nwc_gemv_batched", "nwc_decode_batched", "nwc_blas_create", "nwc_blas_destroy",
           "nwc_prefill_workspace_size", "nwc_gemm_prefill", "nwc_gather_rows", "nwc_read_probe",
           "nwc_noalloc_scratch_bytes", "nwc_gemv_noalloc", "nwc_set_wait_limit", "nwc_qk_norm_rope",
           "nwc_kv_append", "nwc_attend_workspace_size", "nwc_attend")


def _check(st: int, where: str):
    if st != NWC_OK:
        raise NwcError(st, where)


def _params(p) -> Optional[nwc_params]:
    if p is None:
        return None
    if isinstance(p, nwc_params):
        return p
    return nwc_params(*[int(p.get(k, 0)) for k in ("tile_rows", "tile_cols", "chunks_per_tile",
                                                    "max_code_len", "pair_fit", "code_family")])


def _ptr_params(p):
    return ctypes.byref(p) if p is not None else None


# the current stream's handle without building a Stream object (3 us of an 8 us
# call) and the current device; the public lookups where this torch does not
# have them
_raw_stream = getattr(getattr(globals().get("torch"), "_C", None), "_cuda_getCurrentRawStream", None)
_raw_device = getattr(getattr(globals().get("torch"), "_C", None), "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        import torch
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dptr(t, rows: bool = False) -> ctypes.c_void_p:
    """Device address of a tensor: contiguous, or with rows=True a 2-D tensor
    whose rows are contiguous and may sit any stride(0) apart."""
    if hasattr(t, "data_ptr"):
        if not t.is_cuda:
            raise ValueError("expected a device (cuda) tensor")
        if rows and t.dim() == 2 and t.stride(1) == 1:
            return ctypes.c_void_p(t.data_ptr())
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        return ctypes.c_void_p(t.data_ptr())
    return ctypes.c_void_p(int(t))


def _ytype(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return NWC_OUT_F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return NWC_OUT_BF16
    raise ValueError("y must be float32 or bfloat16")


# ------------------------------------------------------------------ host ---

def nwc_status_str(status: int) -> str:
    return _lib.nwc_status_str(int(status)).decode()


def nwc_encode_bound(rows: int, cols: int, params=None) -> int:
    p = _params(params)
    out = _sz(0)
    _check(_lib.nwc_encode_bound(rows, cols, _ptr_params(p), ctypes.byref(out)), "nwc_encode_bound")
    return out.value


def nwc_encode(w: np.ndarray, params=None) -> np.ndarray:
    """Encode a 2-D uint16 (BF16 bit pattern) matrix into a blob (uint8 array)."""
    if w.dtype != np.uint16 or w.ndim != 2:
        raise ValueError("expected a 2-D uint16 array of BF16 bit patterns")
    if w.strides[1] != 2 or w.strides[0] % 2:
        w = np.ascontiguousarray(w)
    rows, cols = w.shape
    ld = w.strides[0] // 2
    p = _params(params)
    cap = nwc_encode_bound(rows, cols, p)
    blob = np.empty(cap, np.uint8)
    used = _sz(0)
    _check(_lib.nwc_encode(w.ctypes.data, rows, cols, ld, _ptr_params(p), blob.ctypes.data, cap,
                           ctypes.byref(used)), "nwc_encode")
    return blob[: used.value]


def nwc_inspect(blob: np.ndarray) -> nwc_info:
    blob = np.ascontiguousarray(blob, np.uint8)
    info = nwc_info()
    _check(_lib.nwc_inspect(blob.ctypes.data, blob.size, ctypes.byref(info)), "nwc_inspect")
    return info


def nwc_workspace_size(info: nwc_info, batch: int = 1) -> int:
    out = _sz(0)
    _check(_lib.nwc_workspace_size(ctypes.byref(info), batch, ctypes.byref(out)), "nwc_workspace_size")
    return out.value


def nwc_bf16_workspace_size(rows: int, cols: int) -> int:
    out = _sz(0)
    _check(_lib.nwc_bf16_workspace_size(rows, cols, ctypes.byref(out)), "nwc_bf16_workspace_size")
    return out.value


# ---------------------------------------------------------------- device ---

def nwc_decode(info: nwc_info, blob_dev, w_dev, ld: Optional[int] = None, stream=None):
    """Decode into w_dev (device uint16/bfloat16, rows x ld)."""
    if ld is None:
        ld = int(w_dev.shape[-1])
    _check(_lib.nwc_decode(ctypes.byref(info), _dptr(blob_dev), _dptr(w_dev), ld, _stream(stream)), "nwc_decode")


class DecodeBatch:
    """Marshalled arguments of one nwc_decode_batched call (blobs i written to
    w_devs[i], row stride = its last dimension), built once and reusable."""

    def __init__(self, infos: Sequence[nwc_info], blobs_dev, w_devs):
        n = len(infos)
        if not (n == len(blobs_dev) == len(w_devs)) or n < 1:
            raise ValueError("need equal, non-empty lists")
        self.count = n
        self.infos = (nwc_info * n)(*infos)
        self.blobs = (_vp * n)(*[_dptr(t).value for t in blobs_dev])
        self.outs = (_vp * n)(*[_dptr(t).value for t in w_devs])
        self.ld = (_u64 * n)(*[int(t.shape[-1]) for t in w_devs])
        self._keep = (list(blobs_dev), list(w_devs))


def nwc_decode_batched(batch: DecodeBatch, stream=None):
    """Several independent decodes in one launch."""
    _check(_lib.nwc_decode_batched(batch.count, batch.infos, batch.blobs, batch.outs, batch.ld, _stream(stream)),
           "nwc_decode_batched")


def _ws(ws):
    if ws is None:
        return ctypes.c_void_p(None), 0
    return _dptr(ws), ws.numel() * ws.element_size()


def nwc_gemv(info: nwc_info, blob_dev, x_dev, y_dev, ws=None, stream=None):
    """y = W x; y_dev float32 or bfloat16 (rows); ws a device byte tensor of
    nwc_workspace_size(info, 1) bytes (zero-filled before its first use on the
    fused path), or None when that size is 0."""
    wp, wn = _ws(ws)
    _check(_lib.nwc_gemv(ctypes.byref(info), _dptr(blob_dev), _dptr(x_dev), _dptr(y_dev), _ytype(y_dev),
                         wp, wn, _stream(stream)), "nwc_gemv")


def nwc_noalloc_scratch_bytes() -> int:
    out = _sz(0)
    _check(_lib.nwc_noalloc_scratch_bytes(ctypes.byref(out)), "nwc_noalloc_scratch_bytes")
    return out.value


def nwc_set_wait_limit(polls: int = 0):
    """Polls after which the matrix-core skinny GEMM's waits give up (its outputs then NaN); 0 = default."""
    _check(_lib.nwc_set_wait_limit(int(polls)), "nwc_set_wait_limit")


def nwc_gemv_noalloc(info: nwc_info, blob_dev, x_dev, y_dev, stream=None):
    """y = W x like nwc_gemv, with no workspace: the library's static per-device scratch holds the
    exchange slots (calls that overlap on one GPU race)."""
    _check(_lib.nwc_gemv_noalloc(ctypes.byref(info), _dptr(blob_dev), _dptr(x_dev), _dptr(y_dev), _ytype(y_dev),
                                 _stream(stream)), "nwc_gemv_noalloc")


def gemv_batched_workspace_size(infos) -> int:
    """Workspace bytes of one nwc_gemv_batched call over these blobs: the sum
    of their batch-1 workspace sizes."""
    return sum(nwc_workspace_size(i, 1) for i in infos)


class GemvBatch:
    """Marshalled arguments of one nwc_gemv_batched call, built once and reusable
    (e.g. inside a captured graph).  ws is a device byte tensor of at least
    gemv_batched_workspace_size(infos) bytes, zero-filled before its first use.
    Keeps the tensors alive."""

    def __init__(self, infos, blobs_dev, xs_dev, ys_dev, ws):
        n = len(infos)
        if not (n == len(blobs_dev) == len(xs_dev) == len(ys_dev)) or n < 1:
            raise ValueError("need equal, non-empty lists")
        self.count = n
        self.infos = (nwc_info * n)(*infos)
        self.blobs = (_vp * n)(*[_dptr(t).value for t in blobs_dev])
        self.xs = (_vp * n)(*[_dptr(t).value for t in xs_dev])
        self.ys = (_vp * n)(*[_dptr(t).value for t in ys_dev])
        ytypes = {_ytype(t) for t in ys_dev}
        if len(ytypes) != 1:
            raise ValueError("all outputs must have one dtype")
        self.ytype = ytypes.pop()
        self.ws, self.ws_bytes = _ws(ws)
        self._keep = (list(blobs_dev), list(xs_dev), list(ys_dev), ws)


def nwc_gemv_batched(batch: GemvBatch, stream=None):
    """Independent GEMVs y_i = W_i x_i in one launch (see GemvBatch)."""
    _check(_lib.nwc_gemv_batched(batch.count, batch.infos, batch.blobs, batch.xs, batch.ys, batch.ytype,
                                 batch.ws, batch.ws_bytes, _stream(stream)), "nwc_gemv_batched")


def nwc_gemm_skinny(info: nwc_info, blob_dev, X_dev, Y_dev, ws=None, stream=None):
    """Y[b] = W X[b] for X_dev [batch, cols] and Y_dev [batch, rows]."""
    batch = int(X_dev.shape[0])
    wp, wn = _ws(ws)
    _check(_lib.nwc_gemm_skinny(ctypes.byref(info), _dptr(blob_dev), _dptr(X_dev, rows=True), int(X_dev.stride(0)),
                                batch, _dptr(Y_dev, rows=True), int(Y_dev.stride(0)), _ytype(Y_dev), wp, wn,
                                _stream(stream)),
           "nwc_gemm_skinny")


def nwc_gather_rows(info: nwc_info, blob_dev, ids_dev, out_dev, stream=None):
    """out_dev[i] = W[ids_dev[i]] (exact BF16 bits; ids past the matrix give zeros): ids_dev a device
    uint32 / int32 vector, out_dev a device [n, cols] int16 or bfloat16 tensor (rows may be strided)."""
    n = int(ids_dev.numel())
    _check(_lib.nwc_gather_rows(ctypes.byref(info), _dptr(blob_dev), _dptr(ids_dev), n, _dptr(out_dev, rows=True),
                                int(out_dev.stride(0)), _stream(stream)), "nwc_gather_rows")


class Blas:
    """Owns an nwc_blas context (a hipBLASLt handle and its algorithm cache)."""

    def __init__(self):
        h = _vp()
        _check(_lib.nwc_blas_create(ctypes.byref(h)), "nwc_blas_create")
        self.handle = h

    def close(self):
        if self.handle is not None and self.handle.value:
            _check(_lib.nwc_blas_destroy(self.handle), "nwc_blas_destroy")
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def nwc_prefill_workspace_size(info: nwc_info) -> int:
    out = _sz()
    _check(_lib.nwc_prefill_workspace_size(ctypes.byref(info), ctypes.byref(out)), "nwc_prefill_workspace_size")
    return out.value


def nwc_gemm_prefill(blas: Blas, info: nwc_info, blob_dev, X_dev, Y_dev, ws, stream=None):
    """Y[b] = W X[b] for any batch: W decoded into ws, then one hipBLASLt GEMM."""
    batch = int(X_dev.shape[0])
    _check(_lib.nwc_gemm_prefill(blas.handle, ctypes.byref(info), _dptr(blob_dev), _dptr(X_dev, rows=True),
                                 int(X_dev.stride(0)), batch, _dptr(Y_dev, rows=True), int(Y_dev.stride(0)),
                                 _ytype(Y_dev), _dptr(ws),
                                 int(ws.numel() * ws.element_size()), _stream(stream)), "nwc_gemm_prefill")


def nwc_gemv_bf16(w_dev, x_dev, y_dev, ws, stream=None):
    """Uncompressed comparator: y = W x with W a device BF16 matrix [rows, cols]; ws a device byte
    tensor of nwc_bf16_workspace_size(rows, cols) bytes, zero-filled before its first use."""
    rows, cols = int(w_dev.shape[0]), int(w_dev.shape[1])
    wp, wn = _ws(ws)
    _check(_lib.nwc_gemv_bf16(_dptr(w_dev), rows, cols, int(w_dev.stride(0)), _dptr(x_dev), _dptr(y_dev),
                              _ytype(y_dev), wp, wn, _stream(stream)), "nwc_gemv_bf16")


def nwc_read_probe(buf_dev, sink_dev, groups: int = 0, layout: int = 1, stream=None):
    """Stream-read every byte of the device tensor buf_dev (HBM read probe); sink_dev a device tensor
    of at least 4 bytes; layout 0 grid-stride, 1 one contiguous range per workgroup."""
    _check(_lib.nwc_read_probe(_dptr(buf_dev), int(buf_dev.numel() * buf_dev.element_size()), _dptr(sink_dev),
                               int(groups), int(layout), _stream(stream)), "nwc_read_probe")


# --------------------------------------------------------- attention side ---

# The same library once more, without declared argument types: the calls below
# hand over ctypes values made beforehand, which need no conversion (0.3 us of 4).
_direct = ctypes.CDLL(LIB_PATH)

_ROPE_STYLES = {"half": NWC_ROPE_HALF, "pairs": NWC_ROPE_PAIRS}


class _Call:
    """Marshalled arguments of one call, built once and reusable (for example
    inside a captured graph): the tensors are kept alive, must be on one
    device, and are read and written anew by every call."""

    def __init__(self):
        self.device = None
        self._keep = []

    def _tensor(self, t, name: str, dtypes, dim: Optional[int] = None):
        if not hasattr(t, "data_ptr"):
            raise ValueError("%s: expected a tensor" % name)
        if not t.is_cuda:
            raise ValueError("%s: expected a device (cuda) tensor" % name)
        if t.dtype not in dtypes:
            raise ValueError("%s: expected %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
        if dim is not None and t.dim() != dim:
            raise ValueError("%s: expected %d dimensions, got %d" % (name, dim, t.dim()))
        if self.device is None:
            self.device = t.device
        elif t.device != self.device:
            raise ValueError("%s: on %s, other tensors on %s" % (name, t.device, self.device))
        self._keep.append(t)
        return t.data_ptr()

    def _vector(self, t, name: str, n: int, dtype):
        p = self._tensor(t, name, (dtype,), 1)
        if t.numel() != n or not t.is_contiguous():
            raise ValueError("%s: expected %d contiguous entries" % (name, n))
        return p

    def _rows(self, t, name: str, tokens: Optional[int], head_dim: Optional[int]):
        """Heads [tokens, heads, head_dim], a token's heads side by side: (address, token stride)."""
        p = self._tensor(t, name, (torch.bfloat16, torch.int16), 3)
        if (tokens is not None and t.shape[0] != tokens) or (head_dim is not None and t.shape[2] != head_dim):
            raise ValueError("%s: unexpected shape %s" % (name, tuple(t.shape)))
        if (t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError("%s: the heads of a token must be contiguous" % name)
        # a single row has no stride of its own
        return p, (int(t.stride(0)) if t.shape[0] > 1 else (t.shape[1] * t.shape[2] + 7) // 8 * 8)

    def _heads(self, src, dst, weight, name: str, tokens: int, head_dim: int):
        h = nwc_heads()
        h.src, h.ld_src = self._rows(src, name, tokens, head_dim)
        h.heads = int(src.shape[1])
        if dst is not None:
            if tuple(dst.shape) != tuple(src.shape):
                raise ValueError("%s_out: expected the shape of %s" % (name, name))
            h.dst, h.ld_dst = self._rows(dst, name + "_out", tokens, head_dim)
        if weight is not None:
            h.weight = self._vector(weight, name + "_weight", head_dim, torch.bfloat16)
        return h

    def _rope(self, freqs, style):
        if style not in _ROPE_STYLES:
            raise ValueError("style must be 'half' or 'pairs'")
        r = nwc_rope()
        if freqs is not None:
            r.freqs = self._vector(freqs, "freqs", int(freqs.numel()), torch.float32)
            r.dims = 2 * int(freqs.numel())
        r.style = _ROPE_STYLES[style]
        return r

    def _table(self, table):
        t = nwc_page_table()
        t.ids = self._tensor(table, "table", (torch.int32,), 2)
        if table.shape[1] > 1 and table.stride(1) != 1:
            raise ValueError("table: rows must be contiguous")
        t.rows, t.cols = int(table.shape[0]), int(table.shape[1])
        t.ld = int(table.stride(0)) if t.rows > 1 else t.cols
        return t

    def _cache(self, cache: "PagedCache"):
        for t, name in ((cache.k_pages, "k_pages"), (cache.v_pages, "v_pages")):
            self._tensor(t, name, (torch.bfloat16, torch.int16), 4)
        return cache.struct

    def _run(self, fn, where: str, stream):
        index = self.device.index
        if index != (_raw_device or torch.cuda.current_device)():   # streams and launches belong to the tensors' device
            with torch.cuda.device(self.device):
                return _check(fn(*self.args, _stream(stream)), where)
        st = fn(*self.args, _vp(_raw_stream(index)) if stream is None and _raw_stream else _stream(stream))
        if st:
            _check(st, where)


class PagedCache:
    """Key and value pages of one layer: two device tensors [n_pages, kv_heads,
    page_len, head_dim] of BF16; pages may be any distance apart, the same in
    both (views of one allocation for all layers, for example)."""

    def __init__(self, k_pages, v_pages):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if t.dim() != 4 or tuple(t.shape) != tuple(k_pages.shape):
                raise ValueError("%s: expected [n_pages, kv_heads, page_len, head_dim], the same for keys and values" % name)
            _, h, n, d = t.shape
            # a single head has no stride of its own
            if (t.stride(3), t.stride(2)) != (1, d) or (h > 1 and t.stride(1) != n * d):
                raise ValueError("%s: the slots of a page must be contiguous" % name)
            if t.shape[0] > 1 and t.stride(0) != k_pages.stride(0):
                raise ValueError("key and value pages must be the same distance apart")
        self.k_pages, self.v_pages = k_pages, v_pages
        n_pages, heads, page_len, d = (int(x) for x in k_pages.shape)
        stride = int(k_pages.stride(0)) if n_pages > 1 else heads * page_len * d
        self.struct = nwc_cache(k_pages.data_ptr(), v_pages.data_ptr(), n_pages, stride, heads, d, page_len, 0)


class QkNormRope(_Call):
    """Arguments of nwc_qk_norm_rope: q [tokens, q_heads, head_dim] and / or k
    [tokens, kv_heads, head_dim] (views into a joint projection output are
    fine), positions int32 [tokens] (negative: padding), weights BF16
    [head_dim] or None (no norm), freqs float32 [dims / 2] radians per position
    or None (no rotation).  Outputs default to the inputs (in place)."""

    def __init__(self, q, k, positions, q_out=None, k_out=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 freqs=None, style: str = "half"):
        super().__init__()
        if q is None and k is None:
            raise ValueError("need queries or keys")
        some = q if q is not None else k
        tokens, d = int(some.shape[0]), int(some.shape[-1])
        self.q = None if q is None else self._heads(q, q if q_out is None else q_out, q_weight, "q", tokens, d)
        self.k = None if k is None else self._heads(k, k if k_out is None else k_out, k_weight, "k", tokens, d)
        self.rope = self._rope(freqs, style)
        pos = self._vector(positions, "positions", tokens, torch.int32)
        self.args = (None if q is None else ctypes.byref(self.q), None if k is None else ctypes.byref(self.k), _u32(tokens),
                     _u32(d), _f32(eps), ctypes.byref(self.rope), _vp(pos))


def nwc_qk_norm_rope(call: QkNormRope, stream=None):
    """Norm and rotation of query and key heads in one pass (see QkNormRope)."""
    call._run(_direct.nwc_qk_norm_rope, "nwc_qk_norm_rope", stream)


class KvAppend(_Call):
    """Arguments of nwc_kv_append: keys (normed and turned on the way) and values
    [tokens, kv_heads, head_dim] of the tokens to positions int32 [tokens] of
    page table rows `rows` (int32 [tokens]; None: token t is row t); queries q,
    if given, are normed and turned in the same launch, in place or to q_out."""

    def __init__(self, cache: PagedCache, table, k, v, positions, rows=None, k_weight=None, q=None, q_out=None, q_weight=None,
                 eps: float = 1e-6, freqs=None, style: str = "half"):
        super().__init__()
        c, t = self._cache(cache), self._table(table)
        tokens, d = int(k.shape[0]), int(c.head_dim)
        self.k = self._heads(k, None, k_weight, "k", tokens, d)
        if tuple(v.shape) != tuple(k.shape):
            raise ValueError("v: expected the shape of k")
        vp, ld_v = self._rows(v, "v", tokens, d)
        self.q = None if q is None else self._heads(q, q if q_out is None else q_out, q_weight, "q", tokens, d)
        self.rope = self._rope(freqs, style)
        pos = self._vector(positions, "positions", tokens, torch.int32)
        row = None if rows is None else self._vector(rows, "rows", tokens, torch.int32)
        self.table = t
        self.args = (ctypes.byref(c), ctypes.byref(t), ctypes.byref(self.k), _vp(vp), _u64(ld_v),
                     None if q is None else ctypes.byref(self.q), _u32(tokens), _f32(eps), ctypes.byref(self.rope), _vp(pos),
                     _vp(row))


def nwc_kv_append(call: KvAppend, stream=None):
    """Keys and values into the paged cache (see KvAppend)."""
    call._run(_direct.nwc_kv_append, "nwc_kv_append", stream)


def nwc_attend_workspace_size(cache: PagedCache, rows: int, q_heads: int, n_groups: int = 0) -> int:
    out = _sz(0)
    _check(_lib.nwc_attend_workspace_size(ctypes.byref(cache.struct), rows, q_heads, n_groups, ctypes.byref(out)),
           "nwc_attend_workspace_size")
    return out.value


class Attend(_Call):
    """Arguments of nwc_attend: one query token per page table row, q and out
    [rows, q_heads, head_dim], lengths int32 [rows] (0: zeros, negative: row
    left as it was), ws a device byte tensor of nwc_attend_workspace_size
    bytes.  group_start int32 [n + 1] and shared_len int32 [n]: rows
    group_start[i] .. group_start[i + 1] - 1 share their first shared_len[i]
    positions, which are then read once.  scale defaults to head_dim ** -0.5."""

    def __init__(self, cache: PagedCache, table, lengths, q, out, ws, scale: Optional[float] = None, group_start=None,
                 shared_len=None):
        super().__init__()
        c, t = self._cache(cache), self._table(table)
        rows, d = int(t.rows), int(c.head_dim)
        qp, ldq = self._rows(q, "q", rows, d)
        if tuple(out.shape) != tuple(q.shape):
            raise ValueError("out: expected the shape of q")
        op, ldo = self._rows(out, "out", rows, d)
        lp = self._vector(lengths, "lengths", rows, torch.int32)
        self.groups = nwc_groups()
        if (group_start is None) != (shared_len is None):
            raise ValueError("group_start and shared_len come together")
        if group_start is not None:
            n = int(shared_len.numel())
            self.groups.count = n
            if n:
                self.groups.start = self._vector(group_start, "group_start", n + 1, torch.int32)
                self.groups.len = self._vector(shared_len, "shared_len", n, torch.int32)
        wp = self._tensor(ws, "ws", (torch.uint8,))
        if not ws.is_contiguous():
            raise ValueError("ws: expected a contiguous tensor")
        self.table = t
        self.args = (ctypes.byref(c), ctypes.byref(t), ctypes.byref(self.groups), _vp(lp), _vp(qp), _u64(ldq),
                     _u32(q.shape[1]), _f32(d ** -0.5 if scale is None else scale), _vp(op), _u64(ldo), _vp(wp),
                     _sz(ws.numel()))


def nwc_attend(call: Attend, stream=None):
    """Attention of one query token per row over the paged cache (see Attend)."""
    call._run(_direct.nwc_attend, "nwc_attend", stream)


def info_dict(info: nwc_info) -> dict:
    d = {name: getattr(info, name) for name, _ in nwc_info._fields_ if name != "code_len"}
    d["code_len"] = bytes(info.code_len)
    return d
