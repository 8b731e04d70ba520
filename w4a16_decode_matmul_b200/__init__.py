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


# The same two structs as bytes (native alignment, trailing padding included):
# packing is a few times cheaper than filling a ctypes structure.
_BF16, _I32 = torch.bfloat16, torch.int32
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_pack_kv4_cache = struct.Struct("@PPPPqiiii").pack
_pack_kv4_batch = struct.Struct("@iiPPPiqi0q").pack


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
