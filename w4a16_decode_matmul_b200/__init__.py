"""Python binding of ``libwq.so`` (the C ABI in ``include/wq.h``).

Argument marshalling only: every step of quantize, dequantize and matmul
runs in the library's CUDA kernels.  PyTorch provides device memory and the
current stream.  The library must have been built (``python
w4a16_decode_matmul_b200/build.py``); importing this package without it raises.

Functions keep the C names without the ``wq_`` prefix:

    codes, scales, zeros = quantize(W, bits=4, group=128, symmetric=False)
    Y = matmul(X, codes, scales, zeros, N, K, bits=4, group=128)
    W_hat = dequantize(codes, scales, zeros, N, K, bits=4, group=128)

``QuantizedWeight`` bundles the three tensors with their format.

Key/value cache in 4 bits (``KV4Cache``, made by ``kv4_cache``), over the
packed rows of a batch of sequences:

    kv4_write(k, v, cache, seq_lens, page_table)
    O = kv4_attention(q, cache, seq_lens, page_table)
    k, v = kv4_read(cache, seq_lens, page_table, rows=n)

Around that attention, in a step of speculative decoding: queries and keys at
their positions (``Rotary``), the pages of a long cache that each query attends
to (``KV4Bounds``, made by ``kv4_bounds``), and the drafts that stand:

    q = kv4_write_rotary(q, k, v, cache, rot, seq_lens, page_table)
    O, lists, lens = kv4_sparse_attention(q, cache, bounds, seq_lens, page_table, max_pages=64)
    tokens, accepted, seq_lens = verify_drafts(target, tokens, uniform, draft, seqs=n,
                                               seq_lens=seq_lens)
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libwq.so")

WQ_OK = 0
WQ_OUT_F32 = 0
WQ_OUT_BF16 = 1
WQ_MATMUL_STATIC_WEIGHTS = 1
WQ_ROTARY_TRANSPOSE = 1
WQ_VERIFY_LOGITS = 1
ROTARY_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}

STATUS_NAMES = {0: "WQ_OK", 1: "WQ_ERR_INVALID_ARG", 2: "WQ_ERR_UNSUPPORTED",
                3: "WQ_ERR_ALIGNMENT", 4: "WQ_ERR_CUDA", 5: "WQ_ERR_TIMEOUT"}


class WQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = status_string(status)
        if status == 4:
            detail += ": " + lib.wq_internal_last_cuda_error().decode()
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({detail})")


class _KV4CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_meta", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_meta", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group", ctypes.c_int32)]


class _KV4BatchStruct(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("row_starts", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int32),
                ("table_stride", ctypes.c_int64), ("max_rows", ctypes.c_int32)]


class _KV4BoundsStruct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("grid", ctypes.c_void_p)]


class _KV4SelectionStruct(ctypes.Structure):
    _fields_ = [("max_pages", ctypes.c_int32), ("first", ctypes.c_int32),
                ("last", ctypes.c_int32), ("lists", ctypes.c_void_p), ("lens", ctypes.c_void_p)]


class _RotarySpecStruct(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float)]


class _VerificationStruct(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("seqs", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("row_starts", ctypes.c_void_p), ("target", ctypes.c_void_p),
                ("target_stride", ctypes.c_int64), ("draft", ctypes.c_void_p),
                ("draft_stride", ctypes.c_int64), ("tokens", ctypes.c_void_p),
                ("uniform", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p),
                ("accepted", ctypes.c_void_p), ("out_lens", ctypes.c_void_p)]


# The same structs as bytes (native alignment, trailing padding included):
# packing is a few times cheaper than filling a ctypes structure.
_BF16, _I32 = torch.bfloat16, torch.int32
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_pack_kv4_cache = struct.Struct("@PPPPqiiii").pack
_pack_kv4_batch = struct.Struct("@iiPPPiqi0q").pack
_pack_kv4_bounds = struct.Struct("@PP").pack
_pack_kv4_selection = struct.Struct("@iiiPP").pack
_pack_rotary_spec = struct.Struct("@Piif0q").pack
_pack_verification = struct.Struct("@iiiiIPPqPqPPPPPPP").pack


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIBRARY_PATH):
        raise ImportError(
            f"{LIBRARY_PATH} is missing: build it with `python w4a16_decode_matmul_b200/build.py`")
    lib = ctypes.CDLL(LIBRARY_PATH)
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    lib.wq_codes_bytes.argtypes = [i64, i64, i32]
    lib.wq_codes_bytes.restype = sz
    lib.wq_meta_elems.argtypes = [i64, i64, i32]
    lib.wq_meta_elems.restype = sz
    lib.wq_quantize.argtypes = [vp, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    lib.wq_quantize.restype = i32
    lib.wq_dequantize.argtypes = [vp, vp, vp, i64, i64, i32, i32, i32, vp, vp]
    lib.wq_dequantize.restype = i32
    lib.wq_matmul_workspace_bytes.argtypes = []
    lib.wq_matmul_workspace_bytes.restype = sz
    lib.wq_matmul.argtypes = [vp, i64, vp, vp, vp, i64, i64, i32, i32, i32, vp, i32, vp, sz,
                              ctypes.c_uint, vp]
    lib.wq_matmul.restype = i32
    lib.wq_matmul_noalloc.argtypes = [vp, i64, vp, vp, vp, i64, i64, i32, i32, i32, vp, i32,
                                      ctypes.c_uint, vp]
    lib.wq_matmul_noalloc.restype = i32
    lib.wq_matmul_noalloc_scratch_bytes.argtypes = []
    lib.wq_matmul_noalloc_scratch_bytes.restype = sz
    lib.wq_q4k_bytes.argtypes = [i64, i64]
    lib.wq_q4k_bytes.restype = sz
    lib.wq_q4k_quantize.argtypes = [vp, i64, i64, vp, vp]
    lib.wq_q4k_quantize.restype = i32
    lib.wq_q4k_matmul.argtypes = [vp, i64, vp, i64, i64, vp, i32, vp]
    lib.wq_q4k_matmul.restype = i32
    lib.wq_q4k_matmul_ex.argtypes = [vp, i64, vp, i64, i64, vp, i32, ctypes.c_uint, vp]
    lib.wq_q4k_matmul_ex.restype = i32
    lib.wq_kv4_write.argtypes = [vp, i64, vp, i64, vp, vp, vp]
    lib.wq_kv4_write.restype = i32
    lib.wq_kv4_read.argtypes = [vp, vp, vp, vp, vp]
    lib.wq_kv4_read.restype = i32
    lib.wq_kv4_attention_workspace_bytes.argtypes = []
    lib.wq_kv4_attention_workspace_bytes.restype = sz
    lib.wq_kv4_attention.argtypes = [vp, i64, i32, vp, vp, ctypes.c_float, vp, i64, vp, sz, vp]
    lib.wq_kv4_attention.restype = i32
    f64 = ctypes.c_double
    lib.wq_kv4_update_bounds.argtypes = [vp, vp, vp, vp]
    lib.wq_kv4_update_bounds.restype = i32
    lib.wq_kv4_select.argtypes = [vp, i64, i32, vp, vp, vp, vp, vp]
    lib.wq_kv4_select.restype = i32
    lib.wq_kv4_attention_pages.argtypes = [vp, i64, i32, vp, i32, vp, ctypes.c_float, vp, i64, vp,
                                           sz, vp]
    lib.wq_kv4_attention_pages.restype = i32
    lib.wq_kv4_sparse_attention.argtypes = [vp, i64, i32, vp, vp, vp, vp, ctypes.c_float, vp, i64,
                                            vp, sz, vp]
    lib.wq_kv4_sparse_attention.restype = i32
    lib.wq_rotary_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    lib.wq_rotary_frequencies.restype = i32
    lib.wq_rotary.argtypes = [vp, i64, i32, i32, i32, vp, vp, ctypes.c_uint, vp, i64, vp]
    lib.wq_rotary.restype = i32
    lib.wq_kv4_write_rotary.argtypes = [vp, i64, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp,
                                        vp]
    lib.wq_kv4_write_rotary.restype = i32
    lib.wq_verify_workspace_bytes.argtypes = [i64]
    lib.wq_verify_workspace_bytes.restype = sz
    lib.wq_verify_drafts.argtypes = [vp, vp, sz, vp]
    lib.wq_verify_drafts.restype = i32
    lib.wq_get_device_error.argtypes = [vp]
    lib.wq_get_device_error.restype = i32
    lib.wq_status_string.argtypes = [i32]
    lib.wq_status_string.restype = ctypes.c_char_p
    lib.wq_version.argtypes = []
    lib.wq_version.restype = ctypes.c_char_p
    lib.wq_internal_last_cuda_error.argtypes = []
    lib.wq_internal_last_cuda_error.restype = ctypes.c_char_p
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.wq_status_string(status).decode()


def version() -> str:
    return lib.wq_version().decode()


def _check(status: int, what: str):
    if status != WQ_OK:
        raise WQError(status, what)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require_cuda(*tensors):
    """Every tensor given is a contiguous CUDA tensor, all on one device; the
    library runs on the current device, so calls are made with that device
    current (``torch.cuda.device``)."""
    device = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"tensors on different devices: {device} and {t.device}")
    return device


def codes_bytes(N: int, K: int, bits: int) -> int:
    return lib.wq_codes_bytes(N, K, bits)


def meta_elems(N: int, K: int, group: int) -> int:
    return lib.wq_meta_elems(N, K, group)


@dataclasses.dataclass
class QuantizedWeight:
    """Packed codes [N, K*bits/8] u8, scales [N, K/group] f16, zeros [N, K/group]
    f16 (None when symmetric), and the format."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None
    N: int
    K: int
    bits: int = 4
    group: int = 128
    symmetric: bool = False

    @property
    def nbytes(self) -> int:
        return (self.codes.nbytes + self.scales.nbytes
                + (0 if self.zeros is None else self.zeros.nbytes))


def quantize(W: torch.Tensor, bits: int = 4, group: int = 128, symmetric: bool = False,
             out: QuantizedWeight | None = None) -> QuantizedWeight:
    """``wq_quantize``: W [N, K] float16 on the GPU -> QuantizedWeight."""
    if W.dtype != torch.float16 or W.dim() != 2:
        raise ValueError("W must be a 2-D float16 tensor")
    _require_cuda(W)
    N, K = W.shape
    if out is None:
        dev = W.device
        nb = codes_bytes(N, K, bits)
        ne = meta_elems(N, K, group)
        if nb == 0 or ne == 0:
            raise WQError(1, "wq_quantize")
        out = QuantizedWeight(
            codes=torch.empty((N, nb // N), dtype=torch.uint8, device=dev),
            scales=torch.empty((N, ne // N), dtype=torch.float16, device=dev),
            zeros=None if symmetric else torch.empty((N, ne // N), dtype=torch.float16, device=dev),
            N=N, K=K, bits=bits, group=group, symmetric=symmetric)
    dev = _require_cuda(W, out.codes, out.scales, out.zeros)
    with torch.cuda.device(dev):
        _check(lib.wq_quantize(_ptr(W), N, K, bits, group, int(symmetric), _ptr(out.codes),
                               _ptr(out.scales), _ptr(out.zeros), _stream(dev)), "wq_quantize")
    return out


def dequantize(qw: QuantizedWeight, out: torch.Tensor | None = None) -> torch.Tensor:
    """``wq_dequantize``: materialise What [N, K] bfloat16 (unfused baseline)."""
    _require_cuda(qw.codes, qw.scales, qw.zeros)
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=torch.bfloat16, device=qw.codes.device)
    dev = _require_cuda(qw.codes, qw.scales, qw.zeros, out)
    with torch.cuda.device(dev):
        _check(lib.wq_dequantize(_ptr(qw.codes), _ptr(qw.scales), _ptr(qw.zeros), qw.N, qw.K,
                                 qw.bits, qw.group, int(qw.symmetric), _ptr(out),
                                 _stream(dev)), "wq_dequantize")
    return out


_workspaces: dict = {}


def workspace(device: torch.device, stream: int) -> torch.Tensor:
    """The zero-filled ``wq_matmul`` workspace used for calls on ``stream``
    (one per device and stream, so that calls on different streams never
    share one)."""
    key = (device.index, stream)
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.zeros(lib.wq_matmul_workspace_bytes(), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def matmul(X: torch.Tensor, qw: QuantizedWeight, out_dtype: torch.dtype = torch.float32,
           out: torch.Tensor | None = None, static_weights: bool = False,
           use_workspace: bool = True) -> torch.Tensor:
    """``wq_matmul``: Y [M, N] = X [M, K] (bfloat16) times What^T.

    X may live on the host: it is then copied to the weights' device, the
    product is computed there and Y is copied back to the host (the
    end-to-end path; pinned host memory makes the copies asynchronous).
    ``static_weights`` passes WQ_MATMUL_STATIC_WEIGHTS: the weights are not
    written by the kernel that precedes the call on the stream.
    ``use_workspace=False`` passes no workspace (whole row tiles per SM)."""
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != qw.K:
        raise ValueError("X must be a 2-D bfloat16 tensor [M, K]")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be float32 or bfloat16")
    dev = qw.codes.device
    host = not X.is_cuda
    Xd = X.to(dev, non_blocking=True) if host else X
    _require_cuda(Xd, qw.codes, qw.scales, qw.zeros)
    M = Xd.shape[0]
    Yd = out if (out is not None and out.is_cuda) else torch.empty(
        (M, qw.N), dtype=out_dtype, device=dev)
    _require_cuda(Xd, qw.codes, qw.scales, qw.zeros, Yd)
    stream = torch.cuda.current_stream(dev).cuda_stream
    ws = workspace(dev, stream) if use_workspace else None
    with torch.cuda.device(dev):
        _check(lib.wq_matmul(_ptr(Xd), M, _ptr(qw.codes), _ptr(qw.scales), _ptr(qw.zeros), qw.N,
                             qw.K, qw.bits, qw.group, int(qw.symmetric), _ptr(Yd),
                             WQ_OUT_BF16 if Yd.dtype == torch.bfloat16 else WQ_OUT_F32,
                             _ptr(ws), 0 if ws is None else ws.numel(),
                             WQ_MATMUL_STATIC_WEIGHTS if static_weights else 0,
                             ctypes.c_void_p(stream)), "wq_matmul")
    if not host:
        return Yd
    if out is not None and not out.is_cuda:
        out.copy_(Yd, non_blocking=True)
        return out
    return Yd.cpu()


def q4k_bytes(N: int, K: int) -> int:
    """``wq_q4k_bytes``: bytes of the superblocks of an [N, K] matrix."""
    return int(lib.wq_q4k_bytes(N, K))


def q4k_quantize(W: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """``wq_q4k_quantize``: W [N, K] float16 on the GPU -> uint8 blocks
    [N, K/256 * 144] (nested superblocks, 4.5 bits per weight)."""
    if W.dtype != torch.float16 or W.dim() != 2:
        raise ValueError("W must be a 2-D float16 tensor")
    N, K = W.shape
    nb = q4k_bytes(N, K)
    if nb == 0:
        raise WQError(1, "wq_q4k_quantize")
    if out is None:
        out = torch.empty((N, nb // N), dtype=torch.uint8, device=W.device)
    dev = _require_cuda(W, out)
    with torch.cuda.device(dev):
        _check(lib.wq_q4k_quantize(_ptr(W), N, K, _ptr(out), _stream(dev)), "wq_q4k_quantize")
    return out


def q4k_matmul(X: torch.Tensor, blocks: torch.Tensor, N: int, K: int,
               out_dtype: torch.dtype = torch.float32,
               out: torch.Tensor | None = None, static_weights: bool = False) -> torch.Tensor:
    """``wq_q4k_matmul_ex``: Y [M, N] = X [M, K] (bfloat16, M <= 8) times What^T
    for superblock weights; X, blocks and Y on the GPU.  ``static_weights``
    passes WQ_MATMUL_STATIC_WEIGHTS (nothing enqueued before writes the
    blocks)."""
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != K:
        raise ValueError("X must be a 2-D bfloat16 tensor [M, K]")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be float32 or bfloat16")
    M = X.shape[0]
    Y = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=X.device)
    dev = _require_cuda(X, blocks, Y)
    with torch.cuda.device(dev):
        _check(lib.wq_q4k_matmul_ex(_ptr(X), M, _ptr(blocks), N, K, _ptr(Y),
                                    WQ_OUT_BF16 if Y.dtype == torch.bfloat16 else WQ_OUT_F32,
                                    WQ_MATMUL_STATIC_WEIGHTS if static_weights else 0,
                                    _stream(dev)), "wq_q4k_matmul_ex")
    return Y


@dataclasses.dataclass(frozen=True)
class KV4Cache:
    """A pool of pages of keys and values in 4 bits (see ``include/wq.h``):
    codes uint8 [pages, kv_heads, page_size, head_dim/2] and (scale, zero)
    pairs float16 [pages, kv_heads, page_size, head_dim/group, 2], for keys and
    for values."""
    k_codes: torch.Tensor
    k_meta: torch.Tensor
    v_codes: torch.Tensor
    v_meta: torch.Tensor
    group: int

    def __post_init__(self):
        _require_cuda(self.k_codes, self.k_meta, self.v_codes, self.v_meta)
        if self.k_codes.dim() != 4 or self.k_codes.dtype != torch.uint8:
            raise ValueError("k_codes must be uint8 [pages, kv_heads, page_size, head_dim/2]")
        if self.group < 1 or self.head_dim % self.group:
            raise ValueError("group must divide the head dimension")
        meta = (*self.k_codes.shape[:3], self.head_dim // self.group, 2)
        if self.v_codes.shape != self.k_codes.shape or self.v_codes.dtype != torch.uint8:
            raise ValueError("v_codes must have the shape and type of k_codes")
        for m in (self.k_meta, self.v_meta):
            if m.dtype != torch.float16 or tuple(m.shape) != meta:
                raise ValueError(f"metadata must be float16 {list(meta)}")
        # the sizes in the order of the C struct, the addresses being taken at each call
        sizes = (self.pages, self.page_size, self.kv_heads, self.head_dim, self.group)
        object.__setattr__(self, "_sizes", sizes)

    @property
    def pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k_codes.shape[3] * 2

    @property
    def nbytes(self) -> int:
        return (self.k_codes.nbytes + self.k_meta.nbytes + self.v_codes.nbytes
                + self.v_meta.nbytes)

    def _struct(self) -> bytes:
        return _pack_kv4_cache(self.k_codes.data_ptr(), self.k_meta.data_ptr(),
                               self.v_codes.data_ptr(), self.v_meta.data_ptr(), *self._sizes)


def kv4_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, group: int = 64,
              device: torch.device | str = "cuda") -> KV4Cache:
    """An empty cache (slots never written hold whatever the memory held)."""
    if min(pages, kv_heads, head_dim, page_size, group) < 1 or head_dim % group or head_dim % 2:
        raise ValueError("sizes must be positive and group must divide head_dim")

    def codes():
        return torch.empty((pages, kv_heads, page_size, head_dim // 2), dtype=torch.uint8,
                           device=device)

    def meta():
        return torch.empty((pages, kv_heads, page_size, head_dim // group, 2),
                           dtype=torch.float16, device=device)
    return KV4Cache(codes(), meta(), codes(), meta(), group)


def _kv4_batch(index: int, rows: int, seq_lens, page_table, row_starts, max_rows) -> bytes:
    """The batch struct after the checks the C ABI cannot make (types, shapes
    and devices of the int32 arrays)."""
    if seq_lens.dtype is not _I32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous 1-D int32 tensor")
    if page_table.dtype is not _I32 or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 tensor [sequences, pages]")
    seqs, width = page_table.shape
    if seq_lens.shape[0] != seqs:
        raise ValueError("page_table must have a row for each sequence")
    stride = width
    if not page_table.is_contiguous():
        stride, step = page_table.stride()
        if width > 1 and step != 1:
            raise ValueError("rows of page_table must be contiguous")
        if seqs <= 1:
            stride = width
    if seq_lens.get_device() != index or page_table.get_device() != index:
        raise ValueError("seq_lens and page_table must be on the cache's device")
    starts = 0
    if row_starts is not None:
        if (row_starts.dtype is not _I32 or row_starts.shape != (seqs + 1,)
                or not row_starts.is_contiguous()):
            raise ValueError("row_starts must be a contiguous int32 tensor [sequences + 1]")
        if row_starts.get_device() != index:
            raise ValueError("row_starts must be on the cache's device")
        starts = row_starts.data_ptr()
    return _pack_kv4_batch(seqs, rows, starts, seq_lens.data_ptr(), page_table.data_ptr(), width,
                           stride, max_rows or 0)


def _kv4_rows(x: torch.Tensor, heads: int | None, d: int, index: int, what: str):
    """(rows, heads, row stride in elements) of a bfloat16 tensor [rows, heads,
    d] whose heads are contiguous (a slice of a fused projection's rows, say)."""
    if x.dtype is not _BF16 or x.dim() != 3:
        raise ValueError(f"{what} must be bfloat16 [rows, {heads or 'heads'}, {d}]")
    rows, h, size = x.shape
    if size != d or (heads is not None and h != heads):
        raise ValueError(f"{what} must be bfloat16 [rows, {heads or 'heads'}, {d}]")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on the cache's device")
    if x.is_contiguous():
        return rows, h, h * d
    row, head, step = x.stride()
    if step != 1 or (h > 1 and head != d):
        raise ValueError(f"the heads of a row of {what} must be contiguous")
    return rows, h, row if rows > 1 else h * d


def _on(index: int, call, what: str, *args) -> None:
    """call(*args, the current stream of device `index`) with that device
    current; raises for a status other than WQ_OK."""
    if _current_device() == index:
        status = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _raw_stream(index))
    if status:
        raise WQError(status, what)


def kv4_write(k: torch.Tensor, v: torch.Tensor, cache: KV4Cache, seq_lens: torch.Tensor,
              page_table: torch.Tensor, row_starts: torch.Tensor | None = None) -> None:
    """``wq_kv4_write``: quantize the rows' keys and values, bfloat16 [rows,
    kv_heads, head_dim], into the cache as the last tokens of their sequences.

    seq_lens int32 [seqs] counts the tokens with the new rows included;
    page_table int32 [seqs, width]; row_starts int32 [seqs + 1] gives the rows
    of each sequence (None: rows/seqs each).  All on the GPU."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    rows, _, ks = _kv4_rows(k, heads, d, index, "k")
    v_rows, _, vs = _kv4_rows(v, heads, d, index, "v")
    if rows != v_rows:
        raise ValueError("k and v must have the same rows")
    _on(index, lib.wq_kv4_write, "wq_kv4_write", k.data_ptr(), ks, v.data_ptr(), vs,
        cache._struct(), _kv4_batch(index, rows, seq_lens, page_table, row_starts, None))


def kv4_read(cache: KV4Cache, seq_lens: torch.Tensor, page_table: torch.Tensor,
             row_starts: torch.Tensor | None = None, rows: int | None = None,
             out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """``wq_kv4_read``: the values (k, v) that the last tokens of the sequences
    stand for, bfloat16 [rows, kv_heads, head_dim]; the arguments as for
    ``kv4_write``.  ``rows`` or ``out`` gives the number of rows; rows behind
    the last sequence are left as they were in ``out`` (zeros without it)."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    if out is None:
        if rows is None:
            raise ValueError("rows or out is required")
        make = torch.empty if row_starts is None else torch.zeros
        out = tuple(make((rows, heads, d), dtype=torch.bfloat16, device=cache.k_codes.device)
                    for _ in range(2))
    k, v = out
    n, _, _ = _kv4_rows(k, heads, d, index, "out[0]")
    v_rows, _, _ = _kv4_rows(v, heads, d, index, "out[1]")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("the outputs must be contiguous")
    if n != v_rows or (rows is not None and rows != n):
        raise ValueError("the outputs must have the same rows")
    _on(index, lib.wq_kv4_read, "wq_kv4_read", cache._struct(),
        _kv4_batch(index, n, seq_lens, page_table, row_starts, None), k.data_ptr(), v.data_ptr())
    return k, v


def kv4_workspace(device: torch.device | str = "cuda") -> torch.Tensor:
    """A zero-filled ``wq_kv4_attention`` workspace.  One serves all calls of a
    stream; calls that may run at the same time need one each."""
    return torch.zeros(lib.wq_kv4_attention_workspace_bytes(), dtype=torch.uint8, device=device)


def kv4_attention(q: torch.Tensor, cache: KV4Cache, seq_lens: torch.Tensor,
                  page_table: torch.Tensor, row_starts: torch.Tensor | None = None,
                  max_rows: int | None = None, scale: float | None = None,
                  out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """``wq_kv4_attention``: causal attention of the rows' queries, bfloat16
    [rows, q_heads, head_dim], over their sequences' cached tokens (the rows'
    own included: write them first).

    ``max_rows`` bounds the rows of one sequence where ``row_starts`` is given.
    It takes part in the choice of the kernel, so results may differ with it
    within the roundings that ``include/wq.h`` states.  ``scale`` is
    1/sqrt(head_dim) by default.  ``workspace`` is a ``kv4_workspace`` that the
    caller keeps, for instance in a captured graph; without it each call makes
    and zero-fills its own.  ``out`` may not overlap ``q``; rows behind the last
    sequence are left as they were in it (zeros without it)."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    rows, q_heads, qs = _kv4_rows(q, None, d, index, "q")
    if q_heads == 0 or q_heads % heads:
        raise ValueError("q_heads must be a multiple of kv_heads")
    if out is None:
        make = torch.empty if row_starts is None else torch.zeros
        out = make(q.shape, dtype=_BF16, device=q.device)
    out_rows, _, os_ = _kv4_rows(out, q_heads, d, index, "out")
    if out_rows != rows:
        raise ValueError("out must have the rows of q")
    if workspace is None:
        workspace = kv4_workspace(q.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the cache's device")
    _on(index, lib.wq_kv4_attention, "wq_kv4_attention", q.data_ptr(), qs, q_heads,
        cache._struct(), _kv4_batch(index, rows, seq_lens, page_table, row_starts, max_rows),
        d ** -0.5 if scale is None else float(scale), out.data_ptr(), os_, workspace.data_ptr(),
        workspace.nbytes)
    return out


@dataclasses.dataclass(frozen=True)
class KV4Bounds:
    """Bounds of the keys of every page of a ``KV4Cache`` (see
    ``include/wq.h``): codes int8 [pages, kv_heads, 2, head_dim], the smallest and
    the largest value of each dimension on the page's grid float32 [pages,
    kv_heads]."""
    codes: torch.Tensor
    grid: torch.Tensor

    def __post_init__(self):
        _require_cuda(self.codes, self.grid)
        if self.codes.dim() != 4 or self.codes.dtype != torch.int8 or self.codes.shape[2] != 2:
            raise ValueError("codes must be int8 [pages, kv_heads, 2, head_dim]")
        if self.grid.dtype != torch.float32 or self.grid.shape != self.codes.shape[:2]:
            raise ValueError("grid must be float32 [pages, kv_heads]")

    def _struct(self, cache: KV4Cache) -> bytes:
        c, k = self.codes, cache.k_codes
        pages, _, heads, d, _ = cache._sizes
        if c.shape != (pages, heads, 2, d):
            raise ValueError("the bounds are another cache's")
        if c.get_device() != k.get_device():
            raise ValueError("the bounds must be on the cache's device")
        return _pack_kv4_bounds(c.data_ptr(), self.grid.data_ptr())


def kv4_bounds(cache: KV4Cache) -> KV4Bounds:
    """Bounds for a cache (those of pages never updated hold whatever the memory
    held)."""
    pages, _, heads, d, _ = cache._sizes
    device = cache.k_codes.device
    return KV4Bounds(torch.empty((pages, heads, 2, d), dtype=torch.int8, device=device),
                     torch.empty((pages, heads), dtype=torch.float32, device=device))


def kv4_update_bounds(cache: KV4Cache, bounds: KV4Bounds, seq_lens: torch.Tensor,
                      page_table: torch.Tensor, row_starts: torch.Tensor | None = None,
                      rows: int | None = None) -> None:
    """``wq_kv4_update_bounds``: the bounds of the pages that the rows are in, from
    the cache; the arguments as for ``kv4_write``, which comes before.  ``rows`` is
    the number of rows (None: one a sequence)."""
    index = cache.k_codes.get_device()
    if rows is None:
        if row_starts is not None:
            raise ValueError("rows is required with row_starts")
        rows = seq_lens.shape[0]
    _on(index, lib.wq_kv4_update_bounds, "wq_kv4_update_bounds", cache._struct(),
        bounds._struct(cache), _kv4_batch(index, rows, seq_lens, page_table, row_starts, None))


def _kv4_lists(index: int, rows: int, heads: int, max_pages, lists, lens, first: int, last: int,
               device):
    """(lists, lens, their struct), made where they are not given."""
    if lists is None:
        if max_pages is None:
            raise ValueError("max_pages or lists is required")
        lists = torch.empty((rows, heads, max_pages), dtype=torch.int32, device=device)
    if lens is None:
        lens = torch.empty((rows,), dtype=torch.int32, device=device)
    if (lists.dtype is not _I32 or lists.dim() != 3 or lists.shape[0] != rows
            or lists.shape[1] != heads or not lists.is_contiguous()):
        raise ValueError("lists must be a contiguous int32 tensor [rows, kv_heads, max_pages]")
    if max_pages is None:
        max_pages = lists.shape[2]
    elif lists.shape[2] != max_pages:
        raise ValueError("lists must hold max_pages pages")
    if lens.dtype is not _I32 or lens.shape != (rows,) or not lens.is_contiguous():
        raise ValueError("lens must be a contiguous int32 tensor [rows]")
    if lists.get_device() != index or lens.get_device() != index:
        raise ValueError("lists and lens must be on the cache's device")
    return lists, lens, _pack_kv4_selection(max_pages, first, last, lists.data_ptr(),
                                            lens.data_ptr())


def kv4_select(q: torch.Tensor, cache: KV4Cache, bounds: KV4Bounds, seq_lens: torch.Tensor,
               page_table: torch.Tensor, row_starts: torch.Tensor | None = None,
               max_pages: int | None = None, first: int = 1, last: int = 2,
               lists: torch.Tensor | None = None, lens: torch.Tensor | None = None):
    """``wq_kv4_select``: the pages that each row and kv head attends to -- the
    first ``first``, the last ``last`` and those of the largest scores, ``max_pages``
    in all -- as (lists int32 [rows, kv_heads, max_pages], lens int32 [rows])."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    rows, q_heads, qs = _kv4_rows(q, None, d, index, "q")
    if q_heads == 0 or q_heads % heads:
        raise ValueError("q_heads must be a multiple of kv_heads")
    lists, lens, selection = _kv4_lists(index, rows, heads, max_pages, lists, lens, first, last,
                                        q.device)
    _on(index, lib.wq_kv4_select, "wq_kv4_select", q.data_ptr(), qs, q_heads, cache._struct(),
        bounds._struct(cache), _kv4_batch(index, rows, seq_lens, page_table, row_starts, None),
        selection)
    return lists, lens


def _kv4_output(q, out, workspace, rows: int, q_heads: int, d: int, index: int, make):
    """(out, its row stride, workspace) of an attention call."""
    if out is None:
        out = make(q.shape, dtype=_BF16, device=q.device)
    out_rows, _, os_ = _kv4_rows(out, q_heads, d, index, "out")
    if out_rows != rows:
        raise ValueError("out must have the rows of q")
    if workspace is None:
        workspace = kv4_workspace(q.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the cache's device")
    return out, os_, workspace


def kv4_attention_pages(q: torch.Tensor, cache: KV4Cache, lists: torch.Tensor,
                        lens: torch.Tensor, scale: float | None = None,
                        out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None) -> torch.Tensor:
    """``wq_kv4_attention_pages``: attention of the rows' queries over the tokens of
    their lists (``kv4_select``'s).  ``scale``, ``out`` and ``workspace`` as for
    ``kv4_attention``; a row of negative length is left as it was in ``out`` (zeros
    without it)."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    rows, q_heads, qs = _kv4_rows(q, None, d, index, "q")
    if q_heads == 0 or q_heads % heads:
        raise ValueError("q_heads must be a multiple of kv_heads")
    _, _, selection = _kv4_lists(index, rows, heads, None, lists, lens, 0, 1, q.device)
    out, os_, workspace = _kv4_output(q, out, workspace, rows, q_heads, d, index, torch.zeros)
    _on(index, lib.wq_kv4_attention_pages, "wq_kv4_attention_pages", q.data_ptr(), qs, q_heads,
        cache._struct(), rows, selection, d ** -0.5 if scale is None else float(scale),
        out.data_ptr(), os_, workspace.data_ptr(), workspace.nbytes)
    return out


def kv4_sparse_attention(q: torch.Tensor, cache: KV4Cache, bounds: KV4Bounds,
                         seq_lens: torch.Tensor, page_table: torch.Tensor,
                         row_starts: torch.Tensor | None = None, max_pages: int | None = None,
                         first: int = 1, last: int = 2, scale: float | None = None,
                         out: torch.Tensor | None = None, lists: torch.Tensor | None = None,
                         lens: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None):
    """``wq_kv4_sparse_attention``: ``kv4_update_bounds``, ``kv4_select`` and
    ``kv4_attention_pages`` in one call, for rows that ``kv4_write`` has written.
    Returns (out, lists, lens)."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    rows, q_heads, qs = _kv4_rows(q, None, d, index, "q")
    if q_heads == 0 or q_heads % heads:
        raise ValueError("q_heads must be a multiple of kv_heads")
    lists, lens, selection = _kv4_lists(index, rows, heads, max_pages, lists, lens, first, last,
                                        q.device)
    out, os_, workspace = _kv4_output(q, out, workspace, rows, q_heads, d, index,
                                      torch.empty if row_starts is None else torch.zeros)
    _on(index, lib.wq_kv4_sparse_attention, "wq_kv4_sparse_attention", q.data_ptr(), qs, q_heads,
        cache._struct(), bounds._struct(cache),
        _kv4_batch(index, rows, seq_lens, page_table, row_starts, None), selection,
        d ** -0.5 if scale is None else float(scale), out.data_ptr(), os_, workspace.data_ptr(),
        workspace.nbytes)
    return out, lists, lens


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None,
                       factor: float = 1.0, context: float = 0.0, low: float = 1.0,
                       high: float = 32.0) -> torch.Tensor:
    """``wq_rotary_frequencies``: float32 [dim/2] on the host, radians a position.
    ``scaling`` None, "linear", "base" or "parts" (see ``include/wq.h``)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROTARY_SCALINGS)}")
    out = torch.empty(max(0, dim // 2), dtype=torch.float32)
    _check(lib.wq_rotary_frequencies(dim, base, ROTARY_SCALINGS[scaling], factor, context, low,
                                     high, _ptr(out)), "wq_rotary_frequencies")
    return out


@dataclasses.dataclass(frozen=True)
class Rotary:
    """Rotary positions of a model: frequencies float32 [dim/2] on the GPU, the layout
    of the pairs, and the factor of cosines and sines."""
    freqs: torch.Tensor
    interleaved: bool = False
    amplitude: float = 1.0

    def __post_init__(self):
        _require_cuda(self.freqs)
        if self.freqs.dim() != 1 or self.freqs.dtype != torch.float32 or not self.freqs.numel():
            raise ValueError("freqs must be a 1-D float32 tensor")

    def _struct(self, index: int) -> bytes:
        if self.freqs.get_device() != index:
            raise ValueError("freqs must be on the rows' device")
        return _pack_rotary_spec(self.freqs.data_ptr(), 2 * self.freqs.shape[0],
                                 bool(self.interleaved), self.amplitude)


def _positions(positions, rows: int, index: int) -> int:
    if positions is None:
        return 0
    if positions.dtype is not _I32 or positions.shape != (rows,) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 tensor [rows]")
    if positions.get_device() != index:
        raise ValueError("positions must be on the rows' device")
    return positions.data_ptr()


def rotary(x: torch.Tensor, positions: torch.Tensor, rot: Rotary, inverse: bool = False,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """``wq_rotary``: x bfloat16 [rows, heads, head_dim] (heads contiguous, rows any
    stride that is a multiple of 8) turned by its positions, int32 [rows].
    ``inverse`` turns by the transpose: the gradient with respect to x of a rotation
    of x.  ``out`` may be ``x`` itself."""
    if x.dim() != 3 or not x.is_cuda:
        raise ValueError("x must be a bfloat16 tensor [rows, heads, head_dim] on a CUDA device")
    index = x.get_device()
    rows, heads, xs = _kv4_rows(x, None, x.shape[2], index, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=_BF16, device=x.device)
    out_rows, _, os_ = _kv4_rows(out, heads, x.shape[2], index, "out")
    if out_rows != rows:
        raise ValueError("out must have the rows of x")
    if positions is None:
        raise ValueError("positions is required")
    _on(index, lib.wq_rotary, "wq_rotary", x.data_ptr(), xs, rows, heads, x.shape[2],
        _positions(positions, rows, index), rot._struct(index),
        WQ_ROTARY_TRANSPOSE if inverse else 0, out.data_ptr(), os_)
    return out


def kv4_write_rotary(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: KV4Cache,
                     rot: Rotary, seq_lens: torch.Tensor, page_table: torch.Tensor,
                     row_starts: torch.Tensor | None = None,
                     positions: torch.Tensor | None = None,
                     out: torch.Tensor | None = None) -> torch.Tensor | None:
    """``wq_kv4_write_rotary``: ``kv4_write`` of the keys turned by their positions
    (those of the rows' tokens, or ``positions`` int32 [rows]) and of the values;
    returns the turned queries in ``out`` (which may be ``q``).  ``q`` None: keys and
    values alone."""
    _, _, heads, d, _ = cache._sizes
    index = cache.k_codes.get_device()
    rows, _, ks = _kv4_rows(k, heads, d, index, "k")
    v_rows, _, vs = _kv4_rows(v, heads, d, index, "v")
    if rows != v_rows:
        raise ValueError("k and v must have the same rows")
    q_ptr, out_ptr, q_heads, qs, os_ = 0, 0, 0, 0, 0
    if q is not None:
        q_rows, q_heads, qs = _kv4_rows(q, None, d, index, "q")
        if out is None:
            make = torch.empty if row_starts is None else torch.zeros
            out = make(q.shape, dtype=_BF16, device=q.device)
        out_rows, _, os_ = _kv4_rows(out, q_heads, d, index, "out")
        if q_rows != rows or out_rows != rows:
            raise ValueError("q, k and out must have the same rows")
        q_ptr, out_ptr = q.data_ptr(), out.data_ptr()
    _on(index, lib.wq_kv4_write_rotary, "wq_kv4_write_rotary", q_ptr, qs, q_heads, out_ptr, os_,
        k.data_ptr(), ks, v.data_ptr(), vs, rot._struct(index),
        _positions(positions, rows, index), cache._struct(),
        _kv4_batch(index, rows, seq_lens, page_table, row_starts, None))
    return out if q is not None else None


def verify_workspace(rows: int, device: torch.device | str = "cuda") -> torch.Tensor:
    """A workspace of ``verify_drafts`` for up to ``rows`` rows.  One serves
    all calls of a stream; calls that may run at the same time need one each."""
    return torch.empty(lib.wq_verify_workspace_bytes(rows), dtype=torch.uint8, device=device)


def _verify_rows(x: torch.Tensor, rows: int, vocab: int, dtype, index: int, what: str) -> int:
    """Row stride of [rows, vocab], the vocabulary contiguous."""
    if x.dim() != 2 or x.shape != (rows, vocab) or x.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype} [{rows}, {vocab}]")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on target's device")
    row, step = x.stride()
    if step != 1 and vocab > 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    return row if rows > 1 else vocab


def _words(x, dtype, shape, index: int, what: str) -> int:
    if x is None:
        return 0
    if x.dtype is not dtype or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)}")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on target's device")
    return x.data_ptr()


def verify_drafts(target: torch.Tensor, tokens: torch.Tensor, uniform: torch.Tensor,
                  draft: torch.Tensor | None = None, seqs: int | None = None,
                  row_starts: torch.Tensor | None = None, logits: bool = False,
                  temperature: torch.Tensor | None = None, seq_lens: torch.Tensor | None = None,
                  out=None, workspace: torch.Tensor | None = None):
    """``wq_verify_drafts``: which drafts stand, and the token behind them.

    target [rows, vocab], float32 or bfloat16, holds the target's probabilities behind
    every row (``logits``: its logits, divided by temperature float32 [seqs], 0 for the
    largest); draft, of the same shape and type, the distribution that each row's token
    int32 [rows] was drawn from (None: it had all of the mass); uniform float32 [rows]
    in [0, 1).  The rows of a sequence are one that stands and its drafts; ``seqs``
    sequences of rows/seqs rows each, or row_starts int32 [seqs + 1].

    Returns (tokens int32 [rows]: the accepted drafts, the sampled token, -1s; accepted
    int32 [seqs]; ``seq_lens`` without the rejected rows, or None).  ``out`` is those
    three tensors; rows behind the last sequence are left as they were (-1 without
    it).  ``workspace`` is a ``verify_workspace`` that the caller keeps; without it each call
    makes its own."""
    if target.dtype is not torch.float32 and target.dtype is not _BF16 or target.dim() != 2:
        raise ValueError("target must be float32 or bfloat16 [rows, vocab]")
    if not target.is_cuda:
        raise ValueError("target must be on a CUDA device")
    index = target.get_device()
    rows, vocab = target.shape
    if row_starts is not None:
        n = row_starts.shape[0] - 1
        if seqs is not None and seqs != n:
            raise ValueError("row_starts must have seqs + 1 elements")
        seqs = n
    elif seqs is None:
        raise ValueError("seqs or row_starts is required")
    ts = _verify_rows(target, rows, vocab, target.dtype, index, "target")
    ds = 0 if draft is None else _verify_rows(draft, rows, vocab, target.dtype, index, "draft")
    if out is None:
        make = torch.empty if rows else torch.zeros       # without rows nothing is launched
        out = (torch.full((rows,), -1, dtype=_I32, device=target.device),
               make((seqs,), dtype=_I32, device=target.device),
               None if seq_lens is None else seq_lens.clone())
    if workspace is None:
        workspace = verify_workspace(max(rows, 1), target.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on target's device")
    if (out[2] is None) != (seq_lens is None):
        raise ValueError("seq_lens and out[2] go together")
    n_shape, b_shape = (rows,), (seqs,)
    v = _pack_verification(
        rows, seqs, vocab, WQ_OUT_BF16 if target.dtype is _BF16 else WQ_OUT_F32,
        WQ_VERIFY_LOGITS if logits else 0,
        _words(row_starts, _I32, (seqs + 1,), index, "row_starts"), target.data_ptr(), ts,
        0 if draft is None else draft.data_ptr(), ds,
        _words(tokens, _I32, n_shape, index, "tokens"),
        _words(uniform, torch.float32, n_shape, index, "uniform"),
        _words(temperature, torch.float32, b_shape, index, "temperature"),
        _words(seq_lens, _I32, b_shape, index, "seq_lens"),
        _words(out[0], _I32, n_shape, index, "out[0]"),
        _words(out[1], _I32, b_shape, index, "out[1]"),
        _words(out[2], _I32, b_shape, index, "out[2]"))
    _on(index, lib.wq_verify_drafts, "wq_verify_drafts", v, workspace.data_ptr(),
        workspace.nbytes)
    return out


def matmul_noalloc(X: torch.Tensor, qw: QuantizedWeight, out_dtype: torch.dtype = torch.float32,
                   out: torch.Tensor | None = None, static_weights: bool = False) -> torch.Tensor:
    """``wq_matmul_noalloc``: as ``matmul`` with device tensors, the workspace
    being the library's own fixed block (see ``include/wq.h``)."""
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != qw.K:
        raise ValueError("X must be a 2-D bfloat16 tensor [M, K]")
    _require_cuda(X, qw.codes, qw.scales, qw.zeros)
    dev = qw.codes.device
    M = X.shape[0]
    Y = out if out is not None else torch.empty((M, qw.N), dtype=out_dtype, device=dev)
    _require_cuda(X, qw.codes, qw.scales, qw.zeros, Y)
    # the library's scratch block is looked up on the current device
    with torch.cuda.device(dev):
        _check(lib.wq_matmul_noalloc(_ptr(X), M, _ptr(qw.codes), _ptr(qw.scales),
                                     _ptr(qw.zeros), qw.N, qw.K, qw.bits, qw.group,
                                     int(qw.symmetric), _ptr(Y),
                                     WQ_OUT_BF16 if Y.dtype == torch.bfloat16 else WQ_OUT_F32,
                                     WQ_MATMUL_STATIC_WEIGHTS if static_weights else 0,
                                     _stream(dev)), "wq_matmul_noalloc")
    return Y


def get_device_error(device: torch.device | None = None) -> int:
    """``wq_get_device_error``: read and clear the device status word."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        return lib.wq_get_device_error(_stream(device))
