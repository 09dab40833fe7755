"""bit_packing_amd -- Python binding of the MI355X Invariant Bit Packing codec.

Argument marshalling only: every step of the codec runs in the HIP kernels of
``libibp.so`` (built from ``csrc/`` for gfx950, C ABI in ``include/ibp.h``).
torch supplies device memory, pinned host memory and streams.  The functions
have the names of the C entry points:

* ``ibp_build_metadata`` -- Mask/Bitval from a sample batch (IBP page,
  "Algoritmo Core", step 1);
* ``ibp_compress`` -- fused size / look-back / pack compression (step 2);
* ``ibp_decompress`` -- device-resident decompression (step 3);
* ``ibp_decompress_gather`` -- rows decoded straight from pinned host memory
  over PCIe ("Integrazione del Sistema", PCIe transfer compression);
* ``ibp_compress_slots`` / ``ibp_decompress_gather_slots`` -- the fixed-slot
  (in-place) layout of the PCIe transfer mode: each row keeps a slot of its raw
  size, only the used part is read, a bit vector marks compressed rows;
* ``ibp_gather_raw`` -- the uncompressed zero-copy gather the codec is
  measured against;
* ``ibp_embedding_lookup`` / ``ibp_embedding_grad`` -- embedding rows with scaling, and
  their gradient by sorted tokens;
* ``ibp_mx_pack`` / ``ibp_mx_unpack`` -- microscaled tensors (e4m3 or e2m1 elements, a
  power-of-two scale per 32);
* ``ibp_mx_swiglu`` / ``ibp_mx_swiglu_backward`` / ``ibp_mx_linear_wgrad`` -- 8-bit
  activation checkpoints and the backward pass from them;
* ``ibp_mx_matmul`` -- product of packed activations with packed 4-bit weights.

The operators take part in no autograd graph: a tensor that requires a gradient gets none
from them, and the backward ones are called by name.

There is no fallback: if ``libibp.so`` is missing or no GPU is present the calls
raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

import torch  # imported first so that libibp.so binds to the HIP runtime torch loaded

_HERE = os.path.dirname(os.path.abspath(__file__))
# IBP_SANITIZE_LIB=1 loads the build whose host code carries AddressSanitizer and
# UndefinedBehaviorSanitizer checks (build_library(sanitize=True); the process must
# preload the clang ASan runtime, see tests/sanitize.sh)
LIB_PATH = os.path.join(_HERE, "libibp_san.so" if os.environ.get("IBP_SANITIZE_LIB") == "1" else "libibp.so")

IBP_OK, IBP_ERR_INVALID_ARG, IBP_ERR_SIZE, IBP_ERR_CAPACITY, IBP_ERR_DEVICE = 0, 1, 2, 3, 4
IBP_DEVERR_CORRUPT, IBP_DEVERR_BAD_ID, IBP_DEVERR_TIMEOUT = 1, 2, 4
IBP_MAX_S = 1024
IBP_NOALLOC_SCRATCH_BYTES = 8 << 20  # device array behind ibp_compress_noalloc, per GPU
IBP_F32, IBP_F16, IBP_BF16 = 0, 1, 2
IBP_MAX_COLS, IBP_MAX_TOKENS = 1 << 30, 1 << 31
IBP_MX_E4M3, IBP_MX_E2M1 = 0, 1

EXPORTS = (
    "ibp_status_str", "ibp_num_segments", "ibp_max_stream_bytes", "ibp_stream_bytes",
    "ibp_metadata_workspace_bytes", "ibp_compress_workspace_bytes", "ibp_build_metadata",
    "ibp_compress", "ibp_decompress", "ibp_decompress_gather", "ibp_gather_raw",
    "ibp_slot_flag_words", "ibp_compress_slots", "ibp_decompress_gather_slots",
    "ibp_metadata_pos_workspace_bytes", "ibp_build_metadata_pos", "ibp_compress_pos", "ibp_decompress_pos",
    "ibp_zip_table_from_sigma", "ibp_zip_blocks", "ibp_zip_codes_bytes", "ibp_zip_workspace_bytes",
    "ibp_zip_compress", "ibp_zip_decompress", "ibp_set_wait_limit", "ibp_set_halves_min_chunks",
    "ibp_compress_noalloc",
    "ibp_embedding_lookup", "ibp_embedding_grad", "ibp_embedding_grad_workspace_bytes",
    "ibp_mx_codes_pitch", "ibp_mx_scales_pitch", "ibp_mx_pack", "ibp_mx_unpack", "ibp_mx_swiglu",
    "ibp_mx_swiglu_backward", "ibp_mx_matmul", "ibp_mx_matmul_workspace_bytes", "ibp_mx_linear_wgrad",
    "ibp_mx_linear_wgrad_workspace_bytes",
)


class ibp_meta_t(ctypes.Structure):
    """Mask and Bitval of a dataset; only the low W bits are used."""
    _fields_ = [("W", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("mask", ctypes.c_uint64), ("bitval", ctypes.c_uint64)]

    def __repr__(self):
        return f"ibp_meta_t(W={self.W}, mask={self.mask:#x}, bitval={self.bitval:#x})"


class ibp_pos_meta_t(ctypes.Structure):
    """Position-dependent metadata: Mask_i / Bitval_i (device arrays of S words) for
    chunk position i of every segment."""
    _fields_ = [("W", ctypes.c_uint32), ("S", ctypes.c_uint32),
                ("mask", ctypes.c_void_p), ("bitval", ctypes.c_void_p)]


class ibp_mx_t(ctypes.Structure):
    """A packed microscaled tensor: element format, shape, device pointers."""
    _fields_ = [("format", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("rows", ctypes.c_uint64),
                ("cols", ctypes.c_uint64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class MxTensor:
    """A microscaled tensor of rows x cols elements: uint8 codes [rows, ibp_mx_codes_pitch]
    and scale bytes [rows, ibp_mx_scales_pitch] on the device."""
    __slots__ = ("rows", "cols", "format", "_codes", "_scales", "_both")

    def __init__(self, codes: torch.Tensor | None, scales: torch.Tensor | None, rows: int, cols: int, format: int,
                 both: torch.Tensor | None = None):
        self.rows, self.cols, self.format = rows, cols, format
        # tensors made here share one allocation, scales behind the codes; views of it are
        # made when asked for (the calls need the addresses alone)
        self._codes, self._scales, self._both = codes, scales, both

    def __repr__(self):
        return f"MxTensor({self.rows} x {self.cols}, {'e4m3' if self.format == IBP_MX_E4M3 else 'e2m1'})"

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            pitch = _mx_pitches(self.cols, self.format)[0]
            self._codes = self._both[: self.rows * pitch].view(self.rows, pitch)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            codes, scales = _mx_pitches(self.cols, self.format)
            self._scales = self._both[self.rows * codes:].view(self.rows, scales)
        return self._scales

    @property
    def device(self) -> torch.device:
        return _device(self._both if self._both is not None else self._codes)

    def struct(self) -> ibp_mx_t:
        rows, cols = self.rows, self.cols
        codes, scales = _mx_pitches(cols, self.format)
        if self._both is not None:
            at = self._both.data_ptr()
            return ibp_mx_t(self.format, 0, rows, cols, at, at + rows * codes)
        # the C side sees pointers only: the tensors must hold what the shape says
        if _nbytes(self._codes) < rows * codes or _nbytes(self._scales) < rows * scales:
            raise ValueError("codes or scales are smaller than their shape needs")
        return ibp_mx_t(self.format, 0, rows, cols, _ptr(self._codes), _ptr(self._scales))


def _mx_pitches(cols: int, format: int) -> tuple[int, int]:
    """Bytes from one row of codes, and of scales, to the next."""
    blocks = (cols + 31) // 32
    return blocks * (32 if format == IBP_MX_E4M3 else 16), (blocks + 3) // 4 * 4


@dataclass
class PosMeta:
    """ibp_pos_meta_t plus the device tensors that hold its tables (kept alive here)."""
    W: int
    S: int
    mask: torch.Tensor    # int64[S], device
    bitval: torch.Tensor  # int64[S], device

    def struct(self) -> ibp_pos_meta_t:
        return ibp_pos_meta_t(self.W, self.S, _ptr(self.mask), _ptr(self.bitval))


def make_meta(W: int, mask: int, bitval: int) -> ibp_meta_t:
    return ibp_meta_t(W, 0, mask, bitval)


class IBPError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what} failed: {status_name(status)}")


_lib = None
_u64, _u32, _vp, _dbl, _int = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_double, ctypes.c_int
_metap = ctypes.POINTER(ibp_meta_t)


def load_library() -> ctypes.CDLL:
    """Load libibp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(bit_packing_amd.build.build_library())")
        lib = ctypes.CDLL(LIB_PATH)
        lib.ibp_status_str.argtypes = [_int]
        lib.ibp_status_str.restype = ctypes.c_char_p
        lib.ibp_num_segments.argtypes = [_u64, _u32]
        lib.ibp_max_stream_bytes.argtypes = [_u64, _u32]
        lib.ibp_stream_bytes.argtypes = [_u64]
        lib.ibp_metadata_workspace_bytes.argtypes = [_u64, _u32]
        lib.ibp_compress_workspace_bytes.argtypes = [_u64, _u32]
        for f in ("ibp_num_segments", "ibp_max_stream_bytes", "ibp_stream_bytes",
                  "ibp_metadata_workspace_bytes", "ibp_compress_workspace_bytes"):
            getattr(lib, f).restype = _u64
        lib.ibp_build_metadata.argtypes = [_vp, _u64, _u32, _dbl, _metap, _vp, _vp, _u64, _vp]
        lib.ibp_compress.argtypes = [_metap, _vp, _u64, _u32, _vp, _u64, _vp, _vp, _u64, _vp, _vp]
        lib.ibp_decompress.argtypes = [_metap, _vp, _u64, _vp, _u64, _u32, _vp, _vp, _vp]
        lib.ibp_decompress_gather.argtypes = [_metap, _vp, _u64, _vp, _u64, _u32, _vp, _u64, _vp, _vp, _vp]
        lib.ibp_gather_raw.argtypes = [_vp, _u64, _u64, _vp, _u64, _vp, _vp, _vp]
        lib.ibp_slot_flag_words.argtypes = [_u64]
        lib.ibp_slot_flag_words.restype = _u64
        lib.ibp_compress_slots.argtypes = [_metap, _vp, _u64, _u32, _vp, _u64, _vp, _vp, _vp]
        lib.ibp_decompress_gather_slots.argtypes = [_metap, _vp, _u64, _u64, _u32, _vp, _vp, _u64, _vp, _vp, _vp]
        _posp = ctypes.POINTER(ibp_pos_meta_t)
        lib.ibp_metadata_pos_workspace_bytes.argtypes = [_u32, _u32]
        lib.ibp_metadata_pos_workspace_bytes.restype = _u64
        lib.ibp_build_metadata_pos.argtypes = [_vp, _u64, _u32, _u32, _dbl, _vp, _vp, _vp, _vp, _u64, _vp]
        lib.ibp_compress_pos.argtypes = [_posp, _vp, _u64, _vp, _u64, _vp, _vp, _u64, _vp, _vp]
        lib.ibp_decompress_pos.argtypes = [_posp, _vp, _u64, _vp, _u64, _vp, _vp, _vp]
        lib.ibp_zip_table_from_sigma.argtypes = [_dbl, _vp]
        for f in ("ibp_zip_blocks", "ibp_zip_codes_bytes", "ibp_zip_workspace_bytes"):
            getattr(lib, f).argtypes = [_u64]
            getattr(lib, f).restype = _u64
        lib.ibp_zip_compress.argtypes = [_vp, _vp, _u64, _vp, _vp, _vp, _u64, _vp, _vp, _u64, _vp, _vp]
        lib.ibp_zip_decompress.argtypes = [_vp, _vp, _vp, _vp, _u64, _vp, _u64, _vp, _vp, _vp]
        lib.ibp_compress_noalloc.argtypes = [_metap, _vp, _u64, _u32, _vp, _u64, _vp, _vp, _vp]
        lib.ibp_compress_noalloc.restype = _int
        lib.ibp_set_wait_limit.argtypes = [_u32]
        lib.ibp_set_wait_limit.restype = _u32
        lib.ibp_set_halves_min_chunks.argtypes = [_u64]
        lib.ibp_set_halves_min_chunks.restype = _u64
        _flt, _mxp = ctypes.c_float, ctypes.POINTER(ibp_mx_t)
        lib.ibp_embedding_lookup.argtypes = [_vp, _int, _u64, _u32, _vp, _u64, _flt, _vp, _int, _vp, _vp]
        lib.ibp_embedding_grad.argtypes = [_vp, _int, _vp, _u64, _u64, _u32, _flt, ctypes.c_int64, _vp, _int, _vp,
                                           _u64, _vp, _vp]
        lib.ibp_embedding_grad_workspace_bytes.argtypes = [_u64, _u64, _u32]
        lib.ibp_mx_codes_pitch.argtypes = [_u64, _u32]
        lib.ibp_mx_scales_pitch.argtypes = [_u64]
        lib.ibp_mx_pack.argtypes = [_vp, _int, _mxp, _vp]
        lib.ibp_mx_unpack.argtypes = [_mxp, _vp, _int, _vp]
        lib.ibp_mx_swiglu.argtypes = [_vp, _vp, _int, _vp, _mxp, _mxp, _vp]
        lib.ibp_mx_swiglu_backward.argtypes = [_vp, _int, _mxp, _mxp, _vp, _vp, _vp]
        lib.ibp_mx_matmul.argtypes = [_mxp, _mxp, _vp, _int, _vp, _u64, _vp]
        lib.ibp_mx_matmul_workspace_bytes.argtypes = [_u64, _u64, _u64, _u32]
        lib.ibp_mx_linear_wgrad.argtypes = [_vp, _int, _u64, _mxp, _vp, _int, _vp, _u64, _vp]
        lib.ibp_mx_linear_wgrad_workspace_bytes.argtypes = [_u64, _u64, _u64, _int]
        for f in ("ibp_embedding_grad_workspace_bytes", "ibp_mx_codes_pitch", "ibp_mx_scales_pitch",
                  "ibp_mx_matmul_workspace_bytes", "ibp_mx_linear_wgrad_workspace_bytes"):
            getattr(lib, f).restype = _u64
        for f in ("ibp_embedding_lookup", "ibp_embedding_grad", "ibp_mx_pack", "ibp_mx_unpack", "ibp_mx_swiglu",
                  "ibp_mx_swiglu_backward", "ibp_mx_matmul", "ibp_mx_linear_wgrad",
                  "ibp_build_metadata", "ibp_compress", "ibp_decompress", "ibp_decompress_gather",
                  "ibp_gather_raw", "ibp_compress_slots", "ibp_decompress_gather_slots",
                  "ibp_build_metadata_pos", "ibp_compress_pos", "ibp_decompress_pos", "ibp_zip_table_from_sigma",
                  "ibp_zip_compress", "ibp_zip_decompress"):
            getattr(lib, f).restype = _int
        _lib = lib
    return _lib


def status_name(status: int) -> str:
    return load_library().ibp_status_str(status).decode()


def _check(rc: int, what: str) -> None:
    if rc != IBP_OK:
        raise IBPError(rc, what)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the codec must be contiguous")
    return t.data_ptr()


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# the current stream's handle without a Stream object around it (2.7 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _device(*tensors) -> torch.device:
    for t in tensors:
        if t is not None and t.is_cuda:
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


# ------------------------------------------------------------------ size queries

def ibp_num_segments(n_chunks: int, S: int) -> int:
    return int(load_library().ibp_num_segments(n_chunks, S))


def ibp_max_stream_bytes(n_chunks: int, W: int) -> int:
    return int(load_library().ibp_max_stream_bytes(n_chunks, W))


def ibp_stream_bytes(total_bits: int) -> int:
    return int(load_library().ibp_stream_bytes(total_bits))


def ibp_metadata_workspace_bytes(n_sample_chunks: int, W: int) -> int:
    return int(load_library().ibp_metadata_workspace_bytes(n_sample_chunks, W))


def ibp_compress_workspace_bytes(n_chunks: int, S: int) -> int:
    return int(load_library().ibp_compress_workspace_bytes(n_chunks, S))


def ibp_set_wait_limit(polls: int) -> int:
    """Tests of the compressors' give-up path only: look-back polls of one
    unpublished predecessor before a tile gives up (0xFFFFFFFF = the default).
    Returns the former value."""
    return int(load_library().ibp_set_wait_limit(polls))


def ibp_set_halves_min_chunks(n_chunks: int) -> int:
    """Compression inputs of at least n_chunks chunks (one Mask, W = 32 or 64, S a
    power of two) take the two-half tiles, smaller ones 8192-chunk tiles; the output
    is the same.  0xFFFFFFFFFFFFFFFF = the default (2^23).  Returns the former value."""
    return int(load_library().ibp_set_halves_min_chunks(n_chunks))


# ------------------------------------------------------------------ codec

def ibp_build_metadata(samples: torch.Tensor, W: int, T: float, stream=None,
                       workspace: torch.Tensor | None = None) -> tuple[ibp_meta_t, list[int]]:
    """(meta, per-position one-counts) of a device sample batch of W-bit chunks."""
    n = _nbytes(samples) // (W // 8) if W in (16, 32, 64) else 0
    if workspace is None:
        workspace = torch.empty(max(ibp_metadata_workspace_bytes(n, W), 8), dtype=torch.uint8,
                                device=_device(samples))
    meta = ibp_meta_t()
    counts = (ctypes.c_uint64 * 64)()
    rc = load_library().ibp_build_metadata(_ptr(samples), n, W, T, ctypes.byref(meta), counts,
                                           _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "ibp_build_metadata")
    return meta, [int(c) for c in counts[:W]]


@dataclass
class Compressed:
    """A compressed tensor: stream bytes, nseg + 1 bit offsets and the format parameters."""
    stream: torch.Tensor    # uint8, capacity >= used bytes
    offsets: torch.Tensor   # int64 bit offsets, nseg + 1 entries
    n_chunks: int
    S: int
    meta: ibp_meta_t


def ibp_compress(meta: ibp_meta_t, x: torch.Tensor, S: int, stream=None, err: torch.Tensor | None = None,
                 out_stream: torch.Tensor | None = None, out_offsets: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> Compressed:
    """Compress the bytes of x (read as W-bit little-endian chunks) with segments of S chunks."""
    W = meta.W
    n_bytes = _nbytes(x)
    n = n_bytes // (W // 8) if W in (16, 32, 64) else 0
    dev = _device(x)
    if out_stream is None:
        out_stream = torch.empty(max(ibp_max_stream_bytes(n, W), 16), dtype=torch.uint8, device=dev)
    if out_offsets is None:
        out_offsets = torch.empty(ibp_num_segments(n, S) + 1, dtype=torch.int64, device=dev)
    if workspace is None:
        workspace = torch.empty(max(ibp_compress_workspace_bytes(n, S), 8), dtype=torch.uint8, device=dev)
    rc = load_library().ibp_compress(ctypes.byref(meta), _ptr(x), n_bytes, S, _ptr(out_stream),
                                     _nbytes(out_stream), _ptr(out_offsets), _ptr(workspace),
                                     _nbytes(workspace), _ptr(err), _stream(stream))
    _check(rc, "ibp_compress")
    return Compressed(out_stream, out_offsets, n, S, meta)


def ibp_decompress(meta: ibp_meta_t, stream_buf: torch.Tensor, offsets: torch.Tensor, n_chunks: int, S: int,
                   out: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decompress n_chunks chunks; returns out (uint8 unless an output tensor is given)."""
    if out is None:
        out = torch.empty(n_chunks * (meta.W // 8), dtype=torch.uint8, device=_device(offsets, stream_buf))
    rc = load_library().ibp_decompress(ctypes.byref(meta), _ptr(stream_buf), _nbytes(stream_buf), _ptr(offsets),
                                       n_chunks, S, _ptr(out), _ptr(err), _stream(stream))
    _check(rc, "ibp_decompress")
    return out


def ibp_decompress_gather(meta: ibp_meta_t, stream_buf: torch.Tensor, offsets: torch.Tensor, S: int,
                          ids: torch.Tensor, out: torch.Tensor | None = None, err: torch.Tensor | None = None,
                          stream=None, n_segments: int | None = None) -> torch.Tensor:
    """Row j of out (S chunks) = segment ids[j]; stream_buf may be pinned host memory."""
    if n_segments is None:
        n_segments = offsets.numel() - 1
    if out is None:
        out = torch.empty(ids.numel() * S * (meta.W // 8), dtype=torch.uint8, device=_device(ids, offsets))
    rc = load_library().ibp_decompress_gather(ctypes.byref(meta), _ptr(stream_buf), _nbytes(stream_buf),
                                              _ptr(offsets), n_segments, S, _ptr(ids), ids.numel(), _ptr(out),
                                              _ptr(err), _stream(stream))
    _check(rc, "ibp_decompress_gather")
    return out


def ibp_gather_raw(src: torch.Tensor, row_bytes: int, ids: torch.Tensor, out: torch.Tensor | None = None,
                   err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Uncompressed zero-copy gather: row j of out = row ids[j] of src (rows of row_bytes bytes)."""
    n_rows = _nbytes(src) // row_bytes
    if out is None:
        out = torch.empty(ids.numel() * row_bytes, dtype=torch.uint8, device=_device(ids))
    rc = load_library().ibp_gather_raw(_ptr(src), row_bytes, n_rows, _ptr(ids), ids.numel(), _ptr(out),
                                       _ptr(err), _stream(stream))
    _check(rc, "ibp_gather_raw")
    return out


# ------------------------------------------------------------------ fixed-slot layout

def ibp_slot_flag_words(n_rows: int) -> int:
    return int(load_library().ibp_slot_flag_words(n_rows))


def ibp_compress_slots(meta: ibp_meta_t, x: torch.Tensor, S: int, slots: torch.Tensor | None = None,
                       flags: torch.Tensor | None = None, err: torch.Tensor | None = None,
                       stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Compress the rows of x (S chunks each) into fixed slots of their raw size.
    ``slots`` may be pinned host memory (compression in place in CPU memory).
    Returns (slots, flags): flags is one bit per row in int64 words (1 = compressed)."""
    row_bytes = S * meta.W // 8
    n_rows = _nbytes(x) // row_bytes if row_bytes else 0
    dev = _device(x)
    if slots is None:
        slots = torch.empty(max(n_rows * row_bytes, 16), dtype=torch.uint8, device=dev)
    if flags is None:
        flags = torch.empty(max(ibp_slot_flag_words(n_rows), 1), dtype=torch.int64, device=dev)
    rc = load_library().ibp_compress_slots(ctypes.byref(meta), _ptr(x), n_rows, S, _ptr(slots), _nbytes(slots),
                                           _ptr(flags), _ptr(err), _stream(stream))
    _check(rc, "ibp_compress_slots")
    return slots, flags


def ibp_decompress_gather_slots(meta: ibp_meta_t, slots: torch.Tensor, flags: torch.Tensor, S: int,
                                ids: torch.Tensor, n_rows: int | None = None, out: torch.Tensor | None = None,
                                err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Row j of out = row ids[j] of a slot table; slots may be pinned host memory."""
    row_bytes = S * meta.W // 8
    if n_rows is None:
        n_rows = _nbytes(slots) // row_bytes
    if out is None:
        out = torch.empty(ids.numel() * row_bytes, dtype=torch.uint8, device=_device(ids, flags))
    rc = load_library().ibp_decompress_gather_slots(ctypes.byref(meta), _ptr(slots), _nbytes(slots), n_rows, S,
                                                    _ptr(flags), _ptr(ids), ids.numel(), _ptr(out), _ptr(err),
                                                    _stream(stream))
    _check(rc, "ibp_decompress_gather_slots")
    return out


# ------------------------------------------------------------------ position-dependent metadata

def ibp_build_metadata_pos(samples: torch.Tensor, W: int, S: int, T: float, stream=None,
                           workspace: torch.Tensor | None = None, counts: bool = True) -> tuple[PosMeta, list | None]:
    """Mask_i / Bitval_i for the S chunk positions of a row, from device sample rows of S
    W-bit chunks.  Returns (PosMeta with device tables, counts[S][W] or None)."""
    n_rows = _nbytes(samples) // (S * W // 8) if W in (16, 32, 64) and S else 0
    dev = _device(samples)
    mask = torch.empty(max(S, 1), dtype=torch.int64, device=dev)
    bitval = torch.empty_like(mask)
    if workspace is None:
        workspace = torch.empty(max(int(load_library().ibp_metadata_pos_workspace_bytes(S, W)), 8),
                                dtype=torch.uint8, device=dev)
    host = (ctypes.c_uint64 * (S * W))() if counts else None
    rc = load_library().ibp_build_metadata_pos(_ptr(samples), n_rows, S, W, T, _ptr(mask), _ptr(bitval), host,
                                               _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "ibp_build_metadata_pos")
    cl = [[host[i * W + b] for b in range(W)] for i in range(S)] if counts else None
    return PosMeta(W, S, mask, bitval), cl


def ibp_compress_pos(meta: PosMeta, x: torch.Tensor, stream=None, err: torch.Tensor | None = None,
                     out_stream: torch.Tensor | None = None, out_offsets: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> Compressed:
    """Compress the bytes of x with position-dependent metadata (segments of meta.S chunks)."""
    W, S = meta.W, meta.S
    n_bytes = _nbytes(x)
    n = n_bytes // (W // 8)
    dev = _device(x)
    if out_stream is None:
        out_stream = torch.empty(max(ibp_max_stream_bytes(n, W), 16), dtype=torch.uint8, device=dev)
    if out_offsets is None:
        out_offsets = torch.empty(ibp_num_segments(n, S) + 1, dtype=torch.int64, device=dev)
    if workspace is None:
        workspace = torch.empty(max(ibp_compress_workspace_bytes(n, S), 8), dtype=torch.uint8, device=dev)
    st = meta.struct()
    rc = load_library().ibp_compress_pos(ctypes.byref(st), _ptr(x), n_bytes, _ptr(out_stream), _nbytes(out_stream),
                                         _ptr(out_offsets), _ptr(workspace), _nbytes(workspace), _ptr(err),
                                         _stream(stream))
    _check(rc, "ibp_compress_pos")
    return Compressed(out_stream, out_offsets, n, S, None)


def ibp_decompress_pos(meta: PosMeta, stream_buf: torch.Tensor, offsets: torch.Tensor, n_chunks: int,
                       out: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decompress n_chunks chunks encoded with position-dependent metadata."""
    if out is None:
        out = torch.empty(n_chunks * (meta.W // 8), dtype=torch.uint8, device=_device(offsets, stream_buf))
    st = meta.struct()
    rc = load_library().ibp_decompress_pos(ctypes.byref(st), _ptr(stream_buf), _nbytes(stream_buf), _ptr(offsets),
                                           n_chunks, _ptr(out), _ptr(err), _stream(stream))
    _check(rc, "ibp_decompress_pos")
    return out


# ------------------------------------------------------------------ comparison codec: BF16 exponent coding

@dataclass
class ZipCompressed:
    """BF16 exponent coding of n words: sign-mantissa bytes, code planes, escape
    exponents (capacity n; the first eoff[-1] are used) and per-block escape offsets."""
    sm: torch.Tensor
    codes: torch.Tensor
    esc: torch.Tensor
    eoff: torch.Tensor
    n: int
    table: bytes


def ibp_zip_table_from_sigma(sigma: float) -> bytes:
    t = (ctypes.c_uint8 * 7)()
    _check(load_library().ibp_zip_table_from_sigma(sigma, t), "ibp_zip_table_from_sigma")
    return bytes(t)


def _table_buf(table) -> ctypes.Array:
    t = bytes(table)
    if len(t) != 7:
        raise ValueError("a table is 7 exponents")
    return (ctypes.c_uint8 * 7)(*t)


def ibp_zip_compress(table, x: torch.Tensor, err: torch.Tensor | None = None, stream=None,
                     out: ZipCompressed | None = None, workspace: torch.Tensor | None = None) -> ZipCompressed:
    """Compress the BF16 words of x (any 2-byte dtype)."""
    lib = load_library()
    n = _nbytes(x) // 2
    dev = _device(x)
    if out is None:
        out = ZipCompressed(torch.empty(max(n, 16), dtype=torch.uint8, device=dev),
                            torch.empty(max(int(lib.ibp_zip_codes_bytes(n)), 16), dtype=torch.uint8, device=dev),
                            torch.empty(max(n, 16), dtype=torch.uint8, device=dev),
                            torch.empty(int(lib.ibp_zip_blocks(n)) + 1, dtype=torch.int64, device=dev), n, bytes(table))
    if workspace is None:
        workspace = torch.empty(max(int(lib.ibp_zip_workspace_bytes(n)), 8), dtype=torch.uint8, device=dev)
    rc = lib.ibp_zip_compress(_table_buf(table), _ptr(x), n, _ptr(out.sm), _ptr(out.codes), _ptr(out.esc),
                              _nbytes(out.esc), _ptr(out.eoff), _ptr(workspace), _nbytes(workspace), _ptr(err),
                              _stream(stream))
    _check(rc, "ibp_zip_compress")
    return out


def ibp_zip_decompress(z: ZipCompressed, out: torch.Tensor | None = None, err: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """BF16 words (as int16) of a ZipCompressed."""
    if out is None:
        out = torch.empty(max(z.n, 8), dtype=torch.int16, device=_device(z.sm))[: z.n]
    rc = load_library().ibp_zip_decompress(_table_buf(z.table), _ptr(z.sm), _ptr(z.codes), _ptr(z.esc),
                                           _nbytes(z.esc), _ptr(z.eoff), z.n, _ptr(out), _ptr(err), _stream(stream))
    _check(rc, "ibp_zip_decompress")
    return out


# ------------------------------------------------------------------ language-model operators
#
# With a stream given, a call runs as under ``torch.cuda.stream(stream)``: what it allocates
# belongs to that stream, so its memory is not handed out again before the work there is
# done.  Ordering that stream after the one that made the inputs is the caller's.


def _stream_context(stream):
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    return torch.cuda.stream(stream)


_DTYPES = {torch.float32: IBP_F32, torch.float16: IBP_F16, torch.bfloat16: IBP_BF16}


def _dtype(dtype) -> int:
    if dtype not in _DTYPES:
        raise ValueError(f"{dtype} is not one of float32, float16, bfloat16")
    return _DTYPES[dtype]


def _ids(ids: torch.Tensor) -> torch.Tensor:
    if ids.dtype != torch.int64:
        raise ValueError("ids are int64")
    return ids


def _matrix(x: torch.Tensor) -> tuple[int, int]:
    """(rows, cols) of a tensor read as rows of its last dimension."""
    if x.dim() == 0:
        raise ValueError("a tensor of rows is needed")
    return math.prod(x.shape[:-1]), x.shape[-1]


def _out(out: torch.Tensor | None, shape, dtype, device) -> torch.Tensor:
    """A new tensor, or the caller's after a check of its shape and dtype."""
    if out is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"the output is {tuple(out.shape)} {out.dtype}, not {tuple(shape)} {dtype}")
    return out


def ibp_embedding_lookup(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out_dtype=None,
                         out: torch.Tensor | None = None, err: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """scale * table[ids], of out_dtype (the table's by default); table [rows, dim] may be
    pinned host memory.  Ids out of range give zero rows and set IBP_DEVERR_BAD_ID."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_embedding_lookup(table, ids, scale, out_dtype, out, err)
    if table.dim() != 2:
        raise ValueError("a table is [rows, dim]")
    rows, dim = table.shape
    out = _out(out, (*_ids(ids).shape, dim), out_dtype or (table.dtype if out is None else out.dtype),
               _device(ids, table))
    rc = load_library().ibp_embedding_lookup(_ptr(table), _dtype(table.dtype), rows, dim, _ptr(ids), ids.numel(),
                                             scale, _ptr(out), _dtype(out.dtype), _ptr(err), _stream(None))
    _check(rc, "ibp_embedding_lookup")
    return out


def ibp_embedding_grad(dout: torch.Tensor, ids: torch.Tensor, n_rows: int, scale: float = 1.0, padding_id: int = -1,
                       grad_dtype=None, grad: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient [n_rows, dim] of ibp_embedding_lookup's table: scale times the sum of dout's
    rows of each id, in 32 bits, of grad_dtype (dout's by default).  Tokens with padding_id
    take no part."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_embedding_grad(dout, ids, n_rows, scale, padding_id, grad_dtype, grad, workspace, err)
    n, dim = _matrix(dout)
    if _ids(ids).numel() * dim != dout.numel() or tuple(dout.shape[:-1]) != tuple(ids.shape):
        raise ValueError("dout is [*ids.shape, dim]")
    n = ids.numel()
    dev = _device(dout, ids)
    grad = _out(grad, (n_rows, dim), grad_dtype or (dout.dtype if grad is None else grad.dtype), dev)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(max(int(lib.ibp_embedding_grad_workspace_bytes(n_rows, n, dim)), 16),
                                dtype=torch.uint8, device=dev)
    rc = lib.ibp_embedding_grad(_ptr(dout), _dtype(dout.dtype), _ptr(ids), n, n_rows, dim, scale, padding_id,
                                _ptr(grad), _dtype(grad.dtype), _ptr(workspace), _nbytes(workspace), _ptr(err),
                                _stream(None))
    _check(rc, "ibp_embedding_grad")
    return grad


def ibp_mx_codes_pitch(cols: int, format: int) -> int:
    return int(load_library().ibp_mx_codes_pitch(cols, format))


def ibp_mx_scales_pitch(cols: int) -> int:
    return int(load_library().ibp_mx_scales_pitch(cols))


def ibp_mx_matmul_workspace_bytes(m: int, n: int, k: int, a_format: int) -> int:
    return int(load_library().ibp_mx_matmul_workspace_bytes(m, n, k, a_format))


def ibp_mx_linear_wgrad_workspace_bytes(tokens: int, outs: int, ins: int, dy_dtype=torch.bfloat16) -> int:
    return int(load_library().ibp_mx_linear_wgrad_workspace_bytes(tokens, outs, ins, _dtype(dy_dtype)))


def ibp_embedding_grad_workspace_bytes(n_rows: int, n_ids: int, dim: int) -> int:
    return int(load_library().ibp_embedding_grad_workspace_bytes(n_rows, n_ids, dim))


def make_mx(rows: int, cols: int, format: int, device) -> MxTensor:
    """An MxTensor of unwritten codes and scales."""
    codes, scales = _mx_pitches(cols, format)
    return MxTensor(None, None, rows, cols, format,
                    torch.empty(rows * (codes + scales), dtype=torch.uint8, device=device))


def _mx(m: MxTensor | None, rows: int, cols: int, format: int, device) -> MxTensor:
    if m is None:
        return make_mx(rows, cols, format, device)
    if (m.rows, m.cols, m.format) != (rows, cols, format):
        raise ValueError("the packed output has another shape or format")
    return m


def ibp_mx_pack(x: torch.Tensor, format: int, out: MxTensor | None = None, stream=None) -> MxTensor:
    """Pack the rows (last dimension) of x into IBP_MX_E4M3 or IBP_MX_E2M1 blocks of 32."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_mx_pack(x, format, out)
    if format not in (IBP_MX_E4M3, IBP_MX_E2M1):
        raise ValueError("a format is IBP_MX_E4M3 or IBP_MX_E2M1")
    rows, cols = _matrix(x)
    out = _mx(out, rows, cols, format, _device(x))
    _check(load_library().ibp_mx_pack(_ptr(x), _dtype(x.dtype), ctypes.byref(out.struct()), _stream(None)),
           "ibp_mx_pack")
    return out


def ibp_mx_unpack(m: MxTensor, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values [rows, cols] of a packed tensor."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_mx_unpack(m, dtype, out)
    out = _out(out, (m.rows, m.cols), dtype, m.device)
    _check(load_library().ibp_mx_unpack(ctypes.byref(m.struct()), _ptr(out), _dtype(out.dtype), _stream(None)),
           "ibp_mx_unpack")
    return out


def ibp_mx_swiglu(gate: torch.Tensor, up: torch.Tensor, h: torch.Tensor | None = None,
                  gate8: MxTensor | None = None, up8: MxTensor | None = None,
                  stream=None) -> tuple[torch.Tensor, MxTensor, MxTensor]:
    """(silu(gate) * up, and the e4m3 checkpoints of gate and up), in one pass."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_mx_swiglu(gate, up, h, gate8, up8)
    if gate.shape != up.shape or gate.dtype != up.dtype:
        raise ValueError("gate and up differ in shape or dtype")
    rows, cols = _matrix(gate)
    dev = _device(gate)
    h = torch.empty_like(gate) if h is None else _out(h, gate.shape, gate.dtype, dev)
    gate8, up8 = _mx(gate8, rows, cols, IBP_MX_E4M3, dev), _mx(up8, rows, cols, IBP_MX_E4M3, dev)
    rc = load_library().ibp_mx_swiglu(_ptr(gate), _ptr(up), _dtype(gate.dtype), _ptr(h),
                                      ctypes.byref(gate8.struct()), ctypes.byref(up8.struct()), _stream(None))
    _check(rc, "ibp_mx_swiglu")
    return h, gate8, up8


def ibp_mx_swiglu_backward(dh: torch.Tensor, gate8: MxTensor, up8: MxTensor, dgate: torch.Tensor | None = None,
                           dup: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dgate, dup) of ibp_mx_swiglu from its checkpoints."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_mx_swiglu_backward(dh, gate8, up8, dgate, dup)
    if _matrix(dh) != (gate8.rows, gate8.cols):
        raise ValueError("dh and the checkpoints differ in shape")
    dev = _device(dh)
    dgate = torch.empty_like(dh) if dgate is None else _out(dgate, dh.shape, dh.dtype, dev)
    dup = torch.empty_like(dh) if dup is None else _out(dup, dh.shape, dh.dtype, dev)
    rc = load_library().ibp_mx_swiglu_backward(_ptr(dh), _dtype(dh.dtype), ctypes.byref(gate8.struct()),
                                               ctypes.byref(up8.struct()), _ptr(dgate), _ptr(dup), _stream(None))
    _check(rc, "ibp_mx_swiglu_backward")
    return dgate, dup


def _workspace(workspace: torch.Tensor | None, need: int, device) -> torch.Tensor | None:
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace


def ibp_mx_matmul(a: MxTensor, b: MxTensor, dtype=torch.bfloat16, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[a.rows, b.rows] product of packed a with packed 4-bit b, both along their columns."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_mx_matmul(a, b, dtype, out, workspace)
    lib, dev = load_library(), a.device
    out = _out(out, (a.rows, b.rows), dtype, dev)
    workspace = _workspace(workspace, int(lib.ibp_mx_matmul_workspace_bytes(a.rows, b.rows, a.cols, a.format)), dev)
    rc = lib.ibp_mx_matmul(ctypes.byref(a.struct()), ctypes.byref(b.struct()), _ptr(out), _dtype(out.dtype),
                           _ptr(workspace), 0 if workspace is None else _nbytes(workspace), _stream(None))
    _check(rc, "ibp_mx_matmul")
    return out


def ibp_mx_linear_wgrad(dy: torch.Tensor, x8: MxTensor, dw_dtype=None, dw: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[outs, x8.cols] weight gradient: the sum over tokens of dy's row times x8's row; dy
    [x8.rows, outs] (in bfloat16 fastest), x8 in e4m3.  dw is of dw_dtype, dy's by default."""
    if stream is not None:
        with _stream_context(stream):
            return ibp_mx_linear_wgrad(dy, x8, dw_dtype, dw, workspace)
    if dy.dim() != 2 or dy.shape[0] != x8.rows:
        raise ValueError("dy is [x8.rows, outs]")
    lib, dev = load_library(), _device(dy)
    outs = dy.shape[1]
    dw = _out(dw, (outs, x8.cols), dw_dtype or (dy.dtype if dw is None else dw.dtype), dev)
    workspace = _workspace(workspace, int(lib.ibp_mx_linear_wgrad_workspace_bytes(x8.rows, outs, x8.cols, _dtype(dy.dtype))),
                           dev)
    rc = lib.ibp_mx_linear_wgrad(_ptr(dy), _dtype(dy.dtype), outs, ctypes.byref(x8.struct()), _ptr(dw),
                                 _dtype(dw.dtype), _ptr(workspace), 0 if workspace is None else _nbytes(workspace),
                                 _stream(None))
    _check(rc, "ibp_mx_linear_wgrad")
    return dw
