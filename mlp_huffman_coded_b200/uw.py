"""Thin ctypes binding of libuw (include/uw.h).

Argument marshalling only: every step of the compressed-weight path runs in
the C++ host codec or the CUDA kernels of libuw.so.  PyTorch is used for
device memory (``tensor.data_ptr()``) and streams
(``torch.cuda.current_stream().cuda_stream``) and nothing else.

``lib()`` raises ``UwError`` when the library has not been built; there is no
fallback.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# UW_LIB_PATH selects another build of the same library (e.g. a tuning build)
LIB_PATH = os.environ.get("UW_LIB_PATH") or os.path.join(_HERE, "libuw.so")

PIPE_FULL, PIPE_EXPONENT, PIPE_TRANSCODE, PIPE_DIRECT, PIPE_BF16 = 0, 1, 2, 3, 4
PIPELINES = {"full": PIPE_FULL, "exponent": PIPE_EXPONENT, "transcode": PIPE_TRANSCODE,
             "direct": PIPE_DIRECT}
PIPE_NAMES = {v: k for k, v in PIPELINES.items()}
PIPE_NAMES[PIPE_BF16] = "bf16"

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "corrupt compressed data",
          4: "on-GPU wait timed out", 5: "CUDA error", 6: "workspace too small", 7: "no sm_100 device"}
UW_OK, UW_ERR_INVALID_ARG, UW_ERR_UNSUPPORTED_SHAPE, UW_ERR_CORRUPT = 0, 1, 2, 3
UW_ERR_TIMEOUT, UW_ERR_CUDA, UW_ERR_WORKSPACE_TOO_SMALL, UW_ERR_NO_DEVICE = 4, 5, 6, 7


class UwError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        super().__init__(f"{what}: {STATUS.get(int(status), 'status %d' % status)} ({int(status)})")


class Codebook(C.Structure):
    _fields_ = [("palette", C.c_uint8 * 16), ("code_len", C.c_uint8 * 16), ("code", C.c_uint16 * 16),
                ("freq", C.c_uint64 * 16), ("n_symbols", C.c_uint8), ("max_len", C.c_uint8),
                ("reserved", C.c_uint8 * 6)]


class Layout(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("chunk_groups", C.c_int32),
                ("words_per_row", C.c_int32), ("n_groups", C.c_int64), ("n_chunks", C.c_int64),
                ("n_verbatim", C.c_int64), ("stream_words", C.c_int64), ("total_bits", C.c_int64)]


class Matrix(C.Structure):
    _fields_ = [("L", Layout), ("cb", Codebook), ("sm", C.c_void_p), ("stream", C.c_void_p),
                ("chunk_bit_off", C.c_void_p), ("vflags", C.c_void_p), ("vprefix", C.c_void_p),
                ("verbatim", C.c_void_p), ("idx4", C.c_void_p), ("pack", C.c_void_p),
                ("pack_off", C.c_void_p)]


class Epilogue(C.Structure):
    _fields_ = [("bias", C.c_void_p), ("residual", C.c_void_p), ("activation", C.c_int32), ("out_type", C.c_int32)]


class ExpertTable(C.Structure):
    _fields_ = [("n_experts", C.c_int32), ("reserved", C.c_int32), ("rows", C.c_int64), ("cols", C.c_int64),
                ("table", C.c_void_p)]


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
OUT_BF16, OUT_FP32 = 0, 1

_P = C.c_void_p
_SIGS = {
    "uw_build_palette_codebook": (C.c_int, [_P, C.c_int64, C.c_int64, C.POINTER(Codebook)]),
    "uw_encode": (C.c_int, [_P, C.c_int64, C.c_int64, C.POINTER(Codebook), C.c_int32, C.POINTER(Layout),
                            _P, _P, _P, _P, _P, _P]),
    "uw_validate": (C.c_int, [C.POINTER(Matrix)]),
    "uw_encode_gpu_workspace_bytes": (C.c_size_t, [C.c_int64, C.c_int64]),
    "uw_build_palette_codebook_gpu": (C.c_int, [_P, C.c_int64, C.c_int64, C.POINTER(Codebook), _P, C.c_size_t, _P]),
    "uw_encode_gpu": (C.c_int, [_P, C.c_int64, C.c_int64, C.POINTER(Codebook), C.c_int32, C.POINTER(Layout),
                                _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "uw_direct_pack_offsets": (C.c_int, [C.POINTER(Layout), _P, _P, C.POINTER(C.c_uint64)]),
    "uw_selftest_bounded_wait": (C.c_int, [_P, C.c_size_t, C.c_uint32, _P]),
    "uw_pack_direct_palette": (C.c_int, [C.POINTER(Matrix), _P, _P, _P]),
    "uw_workspace_bytes": (C.c_size_t, [C.POINTER(Layout), C.c_int32, C.c_int32]),
    "uw_workspace_init": (C.c_int, [_P, C.c_size_t, _P]),
    "uw_workspace_status": (C.c_int, [_P, _P]),
    "uw_decode_full": (C.c_int, [C.POINTER(Matrix), _P, _P, C.c_size_t, _P]),
    "uw_decode_exponent_only": (C.c_int, [C.POINTER(Matrix), _P, _P, C.c_size_t, _P]),
    "uw_transcode_palette": (C.c_int, [C.POINTER(Matrix), _P, _P, C.c_size_t, _P]),
    "uw_decode_rows": (C.c_int, [C.POINTER(Matrix), _P, C.c_int32, _P, _P, C.c_size_t, _P]),
    "uw_gemm_direct_palette": (C.c_int, [C.POINTER(Matrix), _P, C.c_int32, _P, _P, C.c_size_t, _P]),
    "uw_gemm_direct_palette_general_lookup": (C.c_int, [C.POINTER(Matrix), _P, C.c_int32, _P, _P,
                                                        C.c_size_t, _P]),
    "uw_gemm_direct_palette_noalloc": (C.c_int, [C.POINTER(Matrix), _P, C.c_int32, _P, _P]),
    "uw_gemm": (C.c_int, [C.POINTER(Matrix), C.c_int32, _P, C.c_int32, _P, _P, C.c_size_t, _P]),
    "uw_gemm_bf16": (C.c_int, [_P, C.c_int64, C.c_int64, _P, C.c_int32, _P, _P, C.c_size_t, _P]),
    "uw_swiglu": (C.c_int, [_P, _P, _P, C.c_int64, _P]),
    "uw_mlp_workspace_bytes": (C.c_size_t, [C.POINTER(Matrix), C.POINTER(Matrix), C.POINTER(Matrix),
                                            C.POINTER(C.c_int32), C.c_int32]),
    "uw_mlp_block": (C.c_int, [C.POINTER(Matrix), C.POINTER(Matrix), C.POINTER(Matrix), C.POINTER(C.c_int32),
                               _P, C.c_int32, _P, _P, C.c_size_t, _P]),
    "uw_mlp_stack_workspace_bytes": (C.c_size_t, [C.POINTER(C.POINTER(Matrix)), C.POINTER(C.c_int32), C.c_int32,
                                                  C.c_int32]),
    "uw_mlp_stack": (C.c_int, [C.POINTER(C.POINTER(Matrix)), C.POINTER(C.c_int32), C.c_int32, _P, C.c_int32, _P,
                               _P, C.c_size_t, _P]),
    "uw_autotune": (C.c_int, [C.POINTER(Matrix), C.POINTER(C.c_int32), C.c_int32, C.c_int32, _P, _P, _P,
                              C.c_size_t, _P, C.c_size_t, C.POINTER(C.c_int32), C.POINTER(C.c_float), _P]),
    "uw_experts_table_bytes": (C.c_size_t, [C.c_int32]),
    "uw_experts_init": (C.c_int, [C.POINTER(C.POINTER(Matrix)), C.c_int32, _P, C.c_size_t, C.POINTER(ExpertTable),
                                  _P]),
    "uw_grouped_workspace_bytes": (C.c_size_t, [C.POINTER(ExpertTable), C.c_int32, C.c_int32]),
    "uw_gemm_grouped": (C.c_int, [C.POINTER(ExpertTable), _P, C.c_int32, _P, _P, C.c_int32, C.POINTER(Epilogue), _P,
                                  _P, C.c_size_t, _P]),
    "uw_gemm_grouped_swiglu": (C.c_int, [C.POINTER(ExpertTable), C.POINTER(ExpertTable), _P, C.c_int32, _P, _P,
                                         C.c_int32, _P, _P, C.c_size_t, _P]),
    "uw_gemm_epilogue_workspace_bytes": (C.c_size_t, [C.POINTER(Layout), C.c_int32]),
    "uw_gemm_epilogue": (C.c_int, [C.POINTER(Matrix), _P, C.c_int32, C.POINTER(Epilogue), _P, _P, C.c_size_t, _P]),
    "uw_moe_route_workspace_bytes": (C.c_size_t, [C.c_int32, C.c_int32, C.c_int32]),
    "uw_moe_route": (C.c_int, [_P, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32, _P, _P, _P, _P, _P, _P,
                               C.c_size_t, _P]),
    "uw_moe_combine": (C.c_int, [_P, C.c_int32, _P, _P, C.c_int32, C.c_int32, C.c_int64, C.c_int32, _P, _P, _P]),
    "uw_moe_workspace_bytes": (C.c_size_t, [C.POINTER(ExpertTable), C.POINTER(ExpertTable), C.POINTER(ExpertTable),
                                            C.c_int32, C.c_int32]),
    "uw_moe_block": (C.c_int, [C.POINTER(ExpertTable), C.POINTER(ExpertTable), C.POINTER(ExpertTable), _P, C.c_int32,
                               C.c_int32, C.c_int32, _P, C.c_int32, _P, _P, _P, C.c_size_t, _P]),
    "uw_status_string": (C.c_char_p, [C.c_int]),
    "uw_version": (C.c_int32, []),
    "uw_launch_count": (C.c_uint64, []),
}

_lib = None


def lib() -> C.CDLL:
    """Load libuw.so (built by ``python -m mlp_huffman_coded_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise UwError(UW_ERR_NO_DEVICE, f"libuw.so not built at {LIB_PATH}")
        h = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def _check(status: int, what: str):
    if status != UW_OK:
        raise UwError(status, what)


def _ptr(a) -> int:
    """Address of a numpy array or torch tensor (None -> NULL)."""
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# host codec
# ---------------------------------------------------------------------------

@dataclass
class HostEncoded:
    layout: Layout
    cb: Codebook
    sm: np.ndarray
    stream: np.ndarray
    chunk_bit_off: np.ndarray
    vflags: np.ndarray
    vprefix: np.ndarray
    verbatim: np.ndarray

    @property
    def rows(self):
        return int(self.layout.rows)

    @property
    def cols(self):
        return int(self.layout.cols)

    def matrix(self) -> Matrix:
        """uw_matrix whose pointers are these host arrays (for uw_validate)."""
        m = Matrix()
        m.L = self.layout
        m.cb = self.cb
        m.sm, m.stream, m.chunk_bit_off = _ptr(self.sm), _ptr(self.stream), _ptr(self.chunk_bit_off)
        m.vflags, m.vprefix = _ptr(self.vflags), _ptr(self.vprefix)
        m.verbatim = _ptr(self.verbatim) if self.verbatim.size else None
        m.idx4 = None
        m.pack = None
        m.pack_off = None
        return m

    def pack_offsets(self):
        """Direct-palette pack offsets (verbatim rows before each tile) and
        total pack bytes."""
        return _pack_offsets(self.layout, self.vflags)

    def compressed_bytes(self, form: str = "huffman") -> int:
        meta = self.vflags.nbytes + self.vprefix.nbytes + self.verbatim.nbytes
        if form == "huffman":
            return self.sm.nbytes + self.stream.nbytes + self.chunk_bit_off.nbytes + meta
        if form == "palette":
            return self.sm.nbytes + self.rows * self.cols // 2 + meta
        raise ValueError(form)


def _pack_offsets(layout: Layout, vflags: np.ndarray):
    n_tiles = -(-int(layout.rows) // 128) * (int(layout.cols) // 64)
    off = np.empty(n_tiles + 1, np.uint32)
    total = C.c_uint64()
    vflags = np.ascontiguousarray(vflags, dtype=np.uint32)
    _check(lib().uw_direct_pack_offsets(C.byref(layout), _ptr(vflags), _ptr(off), C.byref(total)),
           "uw_direct_pack_offsets")
    return off, int(total.value)


def build_codebook(w: np.ndarray) -> Codebook:
    w = np.ascontiguousarray(w, dtype=np.uint16)
    cb = Codebook()
    _check(lib().uw_build_palette_codebook(_ptr(w), w.shape[0], w.shape[1], C.byref(cb)),
           "uw_build_palette_codebook")
    return cb


def encode(w: np.ndarray, chunk_groups: int = 4, cb: Codebook | None = None) -> HostEncoded:
    w = np.ascontiguousarray(w, dtype=np.uint16)
    rows, cols = w.shape
    if cb is None:
        cb = build_codebook(w)
    L = Layout()
    f = lib().uw_encode
    _check(f(_ptr(w), rows, cols, C.byref(cb), chunk_groups, C.byref(L), None, None, None, None, None, None),
           "uw_encode (sizes)")
    sm = np.empty(rows * cols, np.uint8)
    stream = np.empty(L.stream_words, np.uint32)
    off = np.empty(L.n_chunks + 1, np.uint32)
    vflags = np.empty(rows * L.words_per_row, np.uint32)
    vprefix = np.empty(rows * L.words_per_row + 1, np.uint32)
    verbatim = np.empty(L.n_verbatim * 64, np.uint16)
    _check(f(_ptr(w), rows, cols, C.byref(cb), chunk_groups, C.byref(L), _ptr(sm), _ptr(stream), _ptr(off),
             _ptr(vflags), _ptr(vprefix), _ptr(verbatim) if verbatim.size else None), "uw_encode")
    return HostEncoded(L, cb, sm, stream, off, vflags, vprefix, verbatim)


def validate(enc: HostEncoded) -> int:
    """Host-side format check; returns the status code (0 = ok)."""
    m = enc.matrix()
    return int(lib().uw_validate(C.byref(m)))


# ---------------------------------------------------------------------------
# device side
# ---------------------------------------------------------------------------

class Workspace:
    """Caller-owned device workspace (a torch uint8 tensor), zeroed once."""

    def __init__(self, nbytes: int, device="cuda"):
        import torch
        self.nbytes = max(int(nbytes), 256)
        self.t = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        with torch.cuda.device(self.t.device):
            _check(lib().uw_workspace_init(self.ptr, self.nbytes, _stream(None)), "uw_workspace_init")

    @property
    def ptr(self) -> int:
        return self.t.data_ptr()

    def status(self, stream=None) -> int:
        return int(lib().uw_workspace_status(self.ptr, _stream(stream)))

    def check(self, what="device", stream=None):
        _check(self.status(stream), what)


class DeviceMatrix:
    """One compressed matrix uploaded to the GPU (torch tensors own memory)."""

    def __init__(self, enc: HostEncoded, device="cuda"):
        import torch

        def up(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(device)

        self.enc = enc
        self.device = device
        self.sm = up(enc.sm)
        self.stream = up(enc.stream.view(np.int32))
        self.chunk_bit_off = up(enc.chunk_bit_off.view(np.int32))
        self.vflags = up(enc.vflags.view(np.int32))
        self.vprefix = up(enc.vprefix.view(np.int32))
        self.verbatim = up(enc.verbatim.view(np.int16)) if enc.verbatim.size else None
        self.idx4 = None
        self.mat = Matrix()
        self.mat.L = enc.layout
        self.mat.cb = enc.cb
        self.mat.sm, self.mat.stream = self.sm.data_ptr(), self.stream.data_ptr()
        self.mat.chunk_bit_off = self.chunk_bit_off.data_ptr()
        self.mat.vflags, self.mat.vprefix = self.vflags.data_ptr(), self.vprefix.data_ptr()
        self.mat.verbatim = self.verbatim.data_ptr() if self.verbatim is not None else None
        self.mat.idx4 = None
        self.mat.pack = None
        self.mat.pack_off = None
        self.pack = None
        self.pack_off = None

    @property
    def rows(self):
        return int(self.mat.L.rows)

    @property
    def cols(self):
        return int(self.mat.L.cols)

    @classmethod
    def encode_on_device(cls, w, chunk_groups: int = 4, cb: Codebook | None = None, stream=None):
        """Compress a device-resident BF16 matrix on the GPU (torch int16 /
        bfloat16 tensor [rows, cols]): uw_build_palette_codebook_gpu and
        uw_encode_gpu, whose outputs equal the host encoder's byte for
        byte.  No host copy of W is made."""
        import torch
        w = w.contiguous()
        rows, cols = w.shape
        dev = w.device
        wsn = int(lib().uw_encode_gpu_workspace_bytes(rows, cols))
        if wsn == 0:
            raise UwError(UW_ERR_UNSUPPORTED_SHAPE, "uw_encode_gpu_workspace_bytes")
        ws = torch.empty(wsn, dtype=torch.uint8, device=dev)
        st = _stream(stream)
        if cb is None:
            cb = Codebook()
            _check(lib().uw_build_palette_codebook_gpu(w.data_ptr(), rows, cols, C.byref(cb), ws.data_ptr(), wsn, st),
                   "uw_build_palette_codebook_gpu")
        L = Layout()
        f = lib().uw_encode_gpu
        _check(f(w.data_ptr(), rows, cols, C.byref(cb), chunk_groups, C.byref(L), None, None, None, None, None, None,
                 ws.data_ptr(), wsn, st), "uw_encode_gpu (sizes)")
        self = cls.__new__(cls)
        self.enc = None
        self.device = dev
        self.sm = torch.empty(rows * cols, dtype=torch.uint8, device=dev)
        self.stream = torch.empty(int(L.stream_words), dtype=torch.int32, device=dev)
        self.chunk_bit_off = torch.empty(int(L.n_chunks) + 1, dtype=torch.int32, device=dev)
        self.vflags = torch.empty(rows * int(L.words_per_row), dtype=torch.int32, device=dev)
        self.vprefix = torch.empty(rows * int(L.words_per_row) + 1, dtype=torch.int32, device=dev)
        self.verbatim = torch.empty(int(L.n_verbatim) * 64, dtype=torch.int16, device=dev) if L.n_verbatim else None
        _check(f(w.data_ptr(), rows, cols, C.byref(cb), chunk_groups, C.byref(L), self.sm.data_ptr(),
                 self.stream.data_ptr(), self.chunk_bit_off.data_ptr(), self.vflags.data_ptr(),
                 self.vprefix.data_ptr(), _ptr(self.verbatim), ws.data_ptr(), wsn, st), "uw_encode_gpu")
        self.idx4 = None
        self.mat = Matrix()
        self.mat.L = L
        self.mat.cb = cb
        self.mat.sm, self.mat.stream = self.sm.data_ptr(), self.stream.data_ptr()
        self.mat.chunk_bit_off = self.chunk_bit_off.data_ptr()
        self.mat.vflags, self.mat.vprefix = self.vflags.data_ptr(), self.vprefix.data_ptr()
        self.mat.verbatim = self.verbatim.data_ptr() if self.verbatim is not None else None
        self.mat.idx4 = None
        self.mat.pack = None
        self.mat.pack_off = None
        self.pack = None
        self.pack_off = None
        return self

    def prepare_direct_palette(self, ws: Workspace, stream=None, keep_idx4: bool = True):
        """Load-time preparation of the direct-palette form: transcode to 4-bit
        palette indices, then gather sm + indices + verbatim rows into one
        record per 128x64 tile (uw_pack_direct_palette)."""
        import torch
        self.idx4 = torch.empty(self.rows * self.cols // 2, dtype=torch.uint8, device=self.device)
        transcode_palette(self, self.idx4, ws, stream)
        self.mat.idx4 = self.idx4.data_ptr()
        if self.enc is not None:
            off, nbytes = self.enc.pack_offsets()
        else:
            off, nbytes = _pack_offsets(self.mat.L, self.vflags.cpu().numpy().view(np.uint32))
        self.pack_off = torch.from_numpy(off.view(np.int32)).to(self.device)
        self.pack = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _check(lib().uw_pack_direct_palette(C.byref(self.mat), self.pack_off.data_ptr(), self.pack.data_ptr(),
                                            _stream(stream)), "uw_pack_direct_palette")
        self.mat.pack = self.pack.data_ptr()
        self.mat.pack_off = self.pack_off.data_ptr()
        if not keep_idx4:
            self.mat.idx4 = None
            self.idx4 = None
        return self

    def direct_palette_bytes(self) -> int:
        """Bytes the direct-palette GEMM reads from HBM for W: the pack
        records (sm + 4-bit indices + masks + inline verbatim rows)."""
        return int(self.pack.numel()) if self.pack is not None else 0


def workspace_bytes(dm_or_layout, pipeline: int, batch: int) -> int:
    L = dm_or_layout.mat.L if isinstance(dm_or_layout, DeviceMatrix) else dm_or_layout
    return int(lib().uw_workspace_bytes(C.byref(L), pipeline, batch))


def decode_full(dm: DeviceMatrix, out, ws: Workspace, stream=None):
    _check(lib().uw_decode_full(C.byref(dm.mat), _ptr(out), ws.ptr, ws.nbytes, _stream(stream)), "uw_decode_full")


def decode_exponent_only(dm: DeviceMatrix, out, ws: Workspace, stream=None):
    _check(lib().uw_decode_exponent_only(C.byref(dm.mat), _ptr(out), ws.ptr, ws.nbytes, _stream(stream)),
           "uw_decode_exponent_only")


def decode_rows(dm: DeviceMatrix, rows, out, ws: Workspace, stream=None):
    """out[i] = row rows[i] of W (rows: device int32 tensor)."""
    _check(lib().uw_decode_rows(C.byref(dm.mat), _ptr(rows), rows.numel(), _ptr(out), ws.ptr, ws.nbytes,
                                _stream(stream)), "uw_decode_rows")


def transcode_palette(dm: DeviceMatrix, out, ws: Workspace, stream=None):
    _check(lib().uw_transcode_palette(C.byref(dm.mat), _ptr(out), ws.ptr, ws.nbytes, _stream(stream)),
           "uw_transcode_palette")


def gemm(dm: DeviceMatrix, pipeline: int, x, y, ws: Workspace, stream=None):
    _check(lib().uw_gemm(C.byref(dm.mat), pipeline, _ptr(x), x.shape[0], _ptr(y), ws.ptr, ws.nbytes,
                         _stream(stream)), "uw_gemm")


def gemm_direct_palette(dm: DeviceMatrix, x, y, ws: Workspace, stream=None, general_lookup=False):
    f = lib().uw_gemm_direct_palette_general_lookup if general_lookup else lib().uw_gemm_direct_palette
    _check(f(C.byref(dm.mat), _ptr(x), x.shape[0], _ptr(y), ws.ptr, ws.nbytes, _stream(stream)),
           "uw_gemm_direct_palette")


def gemm_direct_palette_noalloc(dm: DeviceMatrix, x, y, stream=None):
    """Direct-palette GEMM for callers that cannot allocate: the scratch is
    the library's own fixed device array (see uw.h)."""
    _check(lib().uw_gemm_direct_palette_noalloc(C.byref(dm.mat), _ptr(x), x.shape[0], _ptr(y), _stream(stream)),
           "uw_gemm_direct_palette_noalloc")


def gemm_bf16(w, x, y, ws: Workspace, stream=None):
    _check(lib().uw_gemm_bf16(_ptr(w), w.shape[0], w.shape[1], _ptr(x), x.shape[0], _ptr(y), ws.ptr, ws.nbytes,
                              _stream(stream)), "uw_gemm_bf16")


def swiglu(g, u, h, stream=None):
    _check(lib().uw_swiglu(_ptr(g), _ptr(u), _ptr(h), g.numel(), _stream(stream)), "uw_swiglu")


def _pipes(pipelines):
    arr = (C.c_int32 * 3)(*[int(p) for p in pipelines])
    return arr


def mlp_workspace_bytes(gate: DeviceMatrix, up: DeviceMatrix, down: DeviceMatrix, pipelines, batch: int) -> int:
    return int(lib().uw_mlp_workspace_bytes(C.byref(gate.mat), C.byref(up.mat), C.byref(down.mat),
                                            _pipes(pipelines), batch))


def mlp_block(gate: DeviceMatrix, up: DeviceMatrix, down: DeviceMatrix, pipelines, x, y, ws: Workspace,
              stream=None):
    _check(lib().uw_mlp_block(C.byref(gate.mat), C.byref(up.mat), C.byref(down.mat), _pipes(pipelines),
                              _ptr(x), x.shape[0], _ptr(y), ws.ptr, ws.nbytes, _stream(stream)), "uw_mlp_block")


def _stack_args(layers, pipelines):
    """layers: [(gate, up, down), ...] DeviceMatrix triples; pipelines: one
    triple per layer (or one triple for every layer)."""
    mats = [m for triple in layers for m in triple]
    if len(pipelines) == 3 and not hasattr(pipelines[0], "__len__"):
        pipelines = [pipelines] * len(layers)
    pipes = [int(p) for triple in pipelines for p in triple]
    if len(mats) != 3 * len(layers) or len(pipes) != len(mats):
        raise ValueError("one (gate, up, down) triple and one pipeline triple per layer")
    arr = (C.POINTER(Matrix) * len(mats))(*[C.pointer(m.mat) for m in mats])
    return arr, (C.c_int32 * len(pipes))(*pipes), len(layers)


def mlp_stack_workspace_bytes(layers, pipelines, batch: int) -> int:
    arr, pipes, n = _stack_args(layers, pipelines)
    return int(lib().uw_mlp_stack_workspace_bytes(arr, pipes, n, batch))


def mlp_stack(layers, pipelines, x, y, ws: Workspace, stream=None):
    """One decode step's MLP work through the stack: y = MLP_{L-1}(...
    MLP_0(x)) (uw_mlp_stack)."""
    arr, pipes, n = _stack_args(layers, pipelines)
    _check(lib().uw_mlp_stack(arr, pipes, n, _ptr(x), x.shape[0], _ptr(y), ws.ptr, ws.nbytes, _stream(stream)),
           "uw_mlp_stack")


# ---------------------------------------------------------------------------
# products grouped by expert, fused epilogues, mixture of experts
# ---------------------------------------------------------------------------
# These calls check their tensors (shape, type, contiguity, device) and run on
# the tensors' device; a mismatch raises UwError(UW_ERR_INVALID_ARG) before
# anything is launched.  BF16 tensors may be torch.bfloat16 or, as elsewhere
# in this module, int16 views of it.

_torch = None  # torch, imported with the first of these calls
_BF16 = _FP32 = _INT32 = ()  # the element types a tensor argument may have


def _need_torch():
    global _torch, _BF16, _FP32, _INT32
    if _torch is None:
        import torch
        _BF16, _FP32, _INT32 = (torch.bfloat16, torch.int16), (torch.float32,), (torch.int32,)
        _torch = torch


def _tensor(t, what, types, shape, device):
    """Address of a tensor argument after its checks (`device`: CUDA ordinal);
    None stays None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype not in types or t.get_device() != device or not t.is_contiguous():
        raise UwError(UW_ERR_INVALID_ARG, f"{what}: a contiguous {' or '.join(map(str, types))} tensor of shape "
                                          f"{tuple(shape)} on cuda:{device} is wanted, got {t.dtype} {tuple(t.shape)} "
                                          f"on {t.device}")
    return t.data_ptr()


_INT32_MAX = 2**31 - 1


def _count(n, what):
    """A count that the library takes in 32 bits (ctypes would wrap it)."""
    if not 0 <= n <= _INT32_MAX:
        raise UwError(UW_ERR_INVALID_ARG, f"{what}: {n} is not a count of at most 2^31 - 1")
    return n


def _size_arg(n):
    """The same for the workspace sizes, which are 0 for what is too large."""
    return max(-1, min(n, _INT32_MAX))


def _matrix_of(t, what):
    """[rows, cols] of a 2-D tensor argument."""
    if t is None or t.dim() != 2 or t.shape[0] > _INT32_MAX:
        raise UwError(UW_ERR_INVALID_ARG, f"{what}: a 2-D tensor of fewer than 2^31 rows is wanted")
    return t.shape


def _out_type(t, what):
    """(uw_out_type, element types) of a BF16 or FP32 tensor."""
    if _torch is None:
        _need_torch()
    if t is None:
        raise UwError(UW_ERR_INVALID_ARG, f"{what}: a tensor is wanted")
    if t.dtype in _BF16:
        return OUT_BF16, _BF16
    if t.dtype in _FP32:
        return OUT_FP32, _FP32
    raise UwError(UW_ERR_INVALID_ARG, f"{what}: BF16 or FP32 is wanted, got {t.dtype}")


def _space(ws, device):
    """Address and size of a workspace on `device`."""
    if ws.t.get_device() != device:
        raise UwError(UW_ERR_INVALID_ARG, f"workspace: one on cuda:{device} is wanted, got {ws.t.device}")
    return ws.ptr, ws.nbytes


def _call(name, device, stream, *args):
    """One library call on `device` (a CUDA ordinal), whichever is current.
    The current stream is asked for by its raw handle: building the Stream
    object of _stream() takes 3 us, as long as the launch."""
    if device < 0:
        raise UwError(UW_ERR_INVALID_ARG, f"{name}: tensors on a CUDA device are wanted")
    fn = getattr(_lib or lib(), name)
    st = _torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if _torch.cuda.current_device() != device:
        with _torch.cuda.device(device):
            return _check(fn(*args, st), name)
    _check(fn(*args, st), name)


class Experts:
    """One compressed matrix per expert (same shape, direct-palette form), as
    the grouped products take them (uw_experts_init).  The device table holds
    addresses, so the tensors of that form are kept: a matrix may be prepared
    again or dropped, and the products go on with the form it had here."""

    def __init__(self, matrices, stream=None):
        _need_torch()
        self.matrices = list(matrices)
        if not self.matrices:
            raise UwError(UW_ERR_INVALID_ARG, "Experts: no matrices")
        self.device = self.matrices[0].sm.get_device()
        if any(m.sm.get_device() != self.device for m in self.matrices):
            raise UwError(UW_ERR_INVALID_ARG, "Experts: matrices on different devices")
        n = len(self.matrices)
        self._packs = [(m.pack, m.pack_off) for m in self.matrices]
        nbytes = int(lib().uw_experts_table_bytes(n))
        self.table = _torch.empty(max(nbytes, 16), dtype=_torch.uint8, device=f"cuda:{self.device}")
        self.c = ExpertTable()
        arr = (C.POINTER(Matrix) * n)(*[C.pointer(m.mat) for m in self.matrices])
        _call("uw_experts_init", self.device, stream, arr, n, self.table.data_ptr(), nbytes, C.byref(self.c))
        self.rows, self.cols = int(self.c.rows), int(self.c.cols)

    def __len__(self):
        return len(self.matrices)


def grouped_workspace_bytes(experts: Experts, n_rows: int, swiglu: bool = False) -> int:
    return int(lib().uw_grouped_workspace_bytes(C.byref(experts.c), _size_arg(n_rows), int(swiglu)))


def epilogue_workspace_bytes(dm_or_layout, batch: int) -> int:
    L = dm_or_layout.mat.L if isinstance(dm_or_layout, DeviceMatrix) else dm_or_layout
    return int(lib().uw_gemm_epilogue_workspace_bytes(C.byref(L), _size_arg(batch)))


def _epilogue(device, bias_shape, n_rows, rows, y, bias, activation, residual):
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise UwError(UW_ERR_INVALID_ARG, f"activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    out, types = _out_type(y, "y")
    yp = _tensor(y, "y", types, (n_rows, rows), device)
    if bias is None and residual is None and act == 0 and out == OUT_BF16:
        return None, yp
    return C.byref(Epilogue(_tensor(bias, "bias", _BF16, bias_shape, device),
                            _tensor(residual, "residual", _BF16, (n_rows, rows), device), act, out)), yp


def gemm_epilogue(dm: DeviceMatrix, x, y, ws: Workspace, bias=None, activation: str = "none", residual=None,
                  stream=None):
    """y = act(x W^T + bias) + residual (uw_gemm_epilogue): x BF16 [batch,
    cols], y BF16 or FP32 [batch, rows], bias BF16 [rows], residual BF16
    [batch, rows]."""
    batch, _ = _matrix_of(x, "x")
    dev = dm.sm.get_device()
    rows = dm.rows
    e, yp = _epilogue(dev, (rows,), batch, rows, y, bias, activation, residual)
    _call("uw_gemm_epilogue", dev, stream, C.byref(dm.mat),
          _tensor(x, "x", _BF16, (batch, dm.cols), dev), batch, e, yp, *_space(ws, dev))


def _groups(experts, x, offsets, n_rows, rows):
    dev = experts.device
    x_rows, _ = _matrix_of(x, "x")
    return (_tensor(x, "x", _BF16, (x_rows, experts.cols), dev), x_rows, _tensor(rows, "rows", _INT32, (n_rows,), dev),
            _tensor(offsets, "offsets", _INT32, (len(experts) + 1,), dev), n_rows)


def gemm_grouped(experts: Experts, x, offsets, y, ws: Workspace, rows=None, bias=None, activation: str = "none",
                 residual=None, stream=None):
    """y[s] = act(x[rows[s]] W_e^T + bias[e]) + residual[s] for the slots s in
    [offsets[e], offsets[e+1]) of each expert e (uw_gemm_grouped): y BF16 or
    FP32 [n_rows, rows of W], bias BF16 [n_experts, rows of W]."""
    n_rows, _ = _matrix_of(y, "y")
    e, yp = _epilogue(experts.device, (len(experts), experts.rows), n_rows, experts.rows, y, bias, activation, residual)
    _call("uw_gemm_grouped", experts.device, stream, C.byref(experts.c),
          *_groups(experts, x, offsets, n_rows, rows), e, yp,
          *_space(ws, experts.device))


def gemm_grouped_swiglu(gate: Experts, up: Experts, x, offsets, h, ws: Workspace, rows=None, stream=None):
    """h[s] = SiLU(x[rows[s]] G_e^T) * (x[rows[s]] U_e^T) (uw_gemm_grouped_swiglu):
    h BF16 [n_rows, rows of G]."""
    n_rows, _ = _matrix_of(h, "h")
    if up.device != gate.device:
        raise UwError(UW_ERR_INVALID_ARG, "gate and up on different devices")
    _call("uw_gemm_grouped_swiglu", gate.device, stream, C.byref(gate.c), C.byref(up.c),
          *_groups(gate, x, offsets, n_rows, rows), _tensor(h, "h", _BF16, (n_rows, gate.rows), gate.device),
          *_space(ws, gate.device))


class Route:
    """Where uw_moe_route leaves its results (torch tensors own memory).  The
    tensors stay the same for the object's life: their addresses are taken
    once."""

    def __init__(self, n_tokens: int, n_experts: int, top_k: int, device="cuda"):
        import torch
        self.n_tokens, self.n_experts, self.top_k = (_count(n, "Route") for n in (n_tokens, n_experts, top_k))
        self._tensors = (torch.empty(n_tokens, top_k, dtype=torch.float32, device=device),
                         torch.empty(n_tokens, top_k, dtype=torch.int32, device=device),
                         torch.empty(n_tokens, top_k, dtype=torch.int32, device=device),
                         torch.empty(n_tokens * top_k, dtype=torch.int32, device=device),
                         torch.empty(n_experts + 1, dtype=torch.int32, device=device))
        self.device = self.weights.get_device()
        self.addresses = tuple(t.data_ptr() for t in self._tensors)

    weights = property(lambda self: self._tensors[0])
    experts = property(lambda self: self._tensors[1])
    slots = property(lambda self: self._tensors[2])
    rows = property(lambda self: self._tensors[3])
    offsets = property(lambda self: self._tensors[4])


def route_workspace_bytes(n_tokens: int, n_experts: int, top_k: int) -> int:
    return int(lib().uw_moe_route_workspace_bytes(_size_arg(n_tokens), _size_arg(n_experts), _size_arg(top_k)))


def moe_route(logits, route: Route, ws: Workspace, renormalize: bool = True, stream=None):
    """Top-k routing of logits [n_tokens, n_experts] (BF16 or FP32) into
    `route` (uw_moe_route)."""
    typ, types = _out_type(logits, "logits")
    lp = _tensor(logits, "logits", types, (route.n_tokens, route.n_experts), route.device)
    _call("uw_moe_route", route.device, stream, lp, typ, route.n_tokens, route.n_experts,
          route.top_k, int(renormalize), *route.addresses, *_space(ws, route.device))


def moe_combine(parts, slots, weights, y, residual=None, stream=None):
    """y[t] = residual[t] + sum_j weights[t, j] parts[slots[t, j]]
    (uw_moe_combine): parts FP32 or BF16 [n_rows, cols]."""
    n_rows, cols = _matrix_of(parts, "parts")
    n_tokens, top_k = _matrix_of(slots, "slots")
    _count(top_k, "top_k")
    dev = parts.get_device()
    typ, types = _out_type(parts, "parts")
    _call("uw_moe_combine", dev, stream,
          _tensor(parts, "parts", types, (n_rows, cols), dev), typ,
          _tensor(slots, "slots", _INT32, (n_tokens, top_k), dev),
          _tensor(weights, "weights", _FP32, (n_tokens, top_k), dev), n_tokens, top_k, cols, n_rows,
          _tensor(residual, "residual", _BF16, (n_tokens, cols), dev), _tensor(y, "y", _BF16, (n_tokens, cols), dev))


def moe_workspace_bytes(gate: Experts, up: Experts, down: Experts, n_tokens: int, top_k: int) -> int:
    return int(lib().uw_moe_workspace_bytes(C.byref(gate.c), C.byref(up.c), C.byref(down.c), _size_arg(n_tokens),
                                            _size_arg(top_k)))


def moe_block(gate: Experts, up: Experts, down: Experts, x, logits, top_k: int, y, ws: Workspace, residual=None,
              renormalize: bool = True, stream=None):
    """Sparse SwiGLU MLP block (uw_moe_block): y[t] = residual[t] + sum over
    token t's top_k experts of weight * W_down (SiLU(W_gate x) * (W_up x))."""
    n_tokens, _ = _matrix_of(x, "x")
    dev = gate.device
    typ, types = _out_type(logits, "logits")
    if up.device != dev or down.device != dev:
        raise UwError(UW_ERR_INVALID_ARG, "gate, up and down on different devices")
    shape = (n_tokens, gate.cols)
    _call("uw_moe_block", dev, stream, C.byref(gate.c), C.byref(up.c), C.byref(down.c),
          _tensor(logits, "logits", types, (n_tokens, len(gate)), dev), typ, _count(top_k, "top_k"),
          int(renormalize), _tensor(x, "x", _BF16, shape, dev), n_tokens,
          _tensor(residual, "residual", _BF16, shape, dev), _tensor(y, "y", _BF16, shape, dev),
          *_space(ws, dev))


def autotune(dm: DeviceMatrix, batches, reps: int, x, y, ws: Workspace, flush=None, stream=None):
    """Returns (choice[n_batches], us[n_batches, 4])."""
    n = len(batches)
    b = (C.c_int32 * n)(*batches)
    choice = (C.c_int32 * n)()
    us = (C.c_float * (4 * n))()
    _check(lib().uw_autotune(C.byref(dm.mat), b, n, reps, _ptr(x), _ptr(y), _ptr(flush),
                             0 if flush is None else flush.numel() * flush.element_size(), ws.ptr, ws.nbytes,
                             choice, us, _stream(stream)), "uw_autotune")
    return list(choice), np.array(list(us), dtype=np.float64).reshape(n, 4)


def selftest_bounded_wait(ws: Workspace, limit_us: int, stream=None):
    """Launch the bounded-wait self-test (see uw.h); the status it leaves is
    read with ws.status()."""
    _check(lib().uw_selftest_bounded_wait(ws.ptr, ws.nbytes, int(limit_us), _stream(stream)),
           "uw_selftest_bounded_wait")


def launch_count() -> int:
    return int(lib().uw_launch_count())


def version() -> int:
    return int(lib().uw_version())
