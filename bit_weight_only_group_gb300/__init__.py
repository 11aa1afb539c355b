"""Python binding of libqgemm: fused-dequantization linear layers over
weight-only, group-wise, asymmetric low-bit weights on GB300 (sm_103a).

This module only marshals arguments: PyTorch supplies device memory and the
current CUDA stream, and every step of the computation runs in the library's
own CUDA kernels, reached through the C ABI declared in ``include/qgemm.h``.
If ``libqgemm.so`` is missing the functions raise; there is no fallback.

Entry points (same names as the C ABI):

* ``qpack_query_sizes(N, K, bits, group, outlier_frac)`` -> dict of bytes
* ``qpack_quantize(W, bits, group, outlier_frac)`` -> :class:`QWeight`
* ``qgemm_forward(x, qw)`` -> y = x . (dequant(W) + outliers)^T
* ``qgemm_moe_grouped(x, topk_ids, experts)`` -> y [T, k, N]
* ``qgemm_moe_grouped_multi(x, topk_ids, [experts_0, experts_1])`` -> [y_0, y_1]
  (products sharing one routing, e.g. an MoE layer's gate and up)
* ``qkv_append(cache, batch, k, v, q=, rope=, q_norm=, k_norm=)`` -> q (normed
  and) turned; k (normed and turned) and v written to the pages of a
  :class:`KVCache`, or quantised to those of a :class:`KVCache8` (8 bits)
* ``qkv_read(cache, batch)`` -> k, v: the values an 8-bit cache holds
* ``qattn_forward(q, cache, batch)`` -> attention over a shared prefix and each
  sequence's own cached tokens (:class:`KVBatch`)

``stream`` (every call that launches kernels): a torch stream or a raw
cudaStream_t, the current stream by default.  What a call allocates itself, its
results and its scratch memory, is allocated on that stream, as under
``torch.cuda.stream(stream)``.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemm.so")

QG_OK = 0
STATUS_NAMES = {0: "QG_OK", -1: "QG_ERR_INVALID_ARG", -2: "QG_ERR_UNSUPPORTED", -3: "QG_ERR_ALIGNMENT",
                -4: "QG_ERR_WORKSPACE", -5: "QG_ERR_CUDA", -6: "QG_ERR_TIMEOUT", -7: "QG_ERR_DEVICE_STATUS"}
Y_F32, Y_BF16 = 0, 1

QUANT_MODES = {"asymmetric": 0, "symmetric": 1, "linear2": 2}

ABI_FUNCTIONS = ("qpack_query_sizes", "qpack_workspace_size", "qpack_quantize", "qpack_quantize_mode",
                 "qpack_quantize_noalloc",
                 "qgemm_workspace_size",
                 "qgemm_forward", "qgemm_forward_multi", "qgemm_moe_workspace_size", "qgemm_moe_grouped",
                 "qgemm_moe_grouped_multi",
                 "qgemm_device_status", "qgemm_selftest_bounded_wait", "qdiag_workspace_size", "qdiag_layer",
                 "qgemm_w8a8_workspace_size", "qgemm_forward_w8a8",
                 "qrepack_tiles_size", "qrepack_tiles", "qgemm_tiles_workspace_size", "qgemm_forward_tiles",
                 "qgemm_set_dependent_launch", "qkv_append", "qkv_append_norm", "qkv8_append", "qkv8_read",
                 "qattn_workspace_size", "qattn_forward", "qattn8_workspace_size", "qattn8_forward",
                 "qgemm_last_error")


class QgError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class QgQWeight(ctypes.Structure):
    """Mirror of ``qg_qweight`` in include/qgemm.h."""
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("group", ctypes.c_int32), ("packed", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("zp", ctypes.c_void_p), ("codebook", ctypes.c_void_p), ("nnz", ctypes.c_int32),
                ("out_row_ptr", ctypes.c_void_p), ("out_col", ctypes.c_void_p),
                ("out_val", ctypes.c_void_p), ("scale8", ctypes.c_void_p), ("scale8_exp", ctypes.c_void_p),
                ("fb_row_ptr", ctypes.c_void_p), ("fb_col", ctypes.c_void_p), ("fb_val", ctypes.c_void_p),
                ("fb_cap", ctypes.c_int32)]


class QgKvCache(ctypes.Structure):
    """Mirror of ``qg_kv_cache`` in include/qgemm.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class QgKv8Cache(ctypes.Structure):
    """Mirror of ``qg_kv8_cache`` in include/qgemm.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("scale_block_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64)]


class QgKvBatch(ctypes.Structure):
    """Mirror of ``qg_kv_batch`` in include/qgemm.h."""
    _fields_ = [("sequences", ctypes.c_int32), ("tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_kv", ctypes.c_int32), ("table_ld", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("prefix_table", ctypes.c_void_p)]


class QgRope(ctypes.Structure):
    """Mirror of ``qg_rope`` in include/qgemm.h."""
    _fields_ = [("table", ctypes.c_void_p), ("at", ctypes.c_void_p), ("positions", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class QgHeadNorm(ctypes.Structure):
    """Mirror of ``qg_head_norm`` in include/qgemm.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_weight_only_group_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        i32, f32, vp, sz = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
        psz, pi32 = ctypes.POINTER(sz), ctypes.POINTER(i32)
        pq = ctypes.POINTER(QgQWeight)
        L.qpack_query_sizes.argtypes = [i32, i32, i32, i32, f32, psz, psz, psz, psz, pi32]
        L.qpack_workspace_size.argtypes = [i32, i32, psz]
        L.qpack_quantize.argtypes = [vp, f32, pq, vp, sz, vp]
        L.qpack_quantize_mode.argtypes = [vp, f32, ctypes.c_int, pq, vp, sz, vp]
        L.qgemm_workspace_size.argtypes = [i32, pq, psz]
        L.qgemm_forward.argtypes = [vp, i32, i32, pq, vp, i32, ctypes.c_int, vp, sz, vp]
        L.qgemm_moe_workspace_size.argtypes = [i32, i32, i32, pq, psz]
        L.qgemm_moe_grouped.argtypes = [vp, i32, vp, i32, pq, i32, vp, ctypes.c_int, vp, sz, vp]
        L.qgemm_moe_grouped_multi.argtypes = [vp, i32, vp, i32, pq, i32, i32, ctypes.POINTER(vp), ctypes.c_int, vp,
                                              sz, vp]
        L.qgemm_device_status.argtypes = [pi32, i32]
        L.qgemm_selftest_bounded_wait.argtypes = [i32, vp]
        L.qdiag_workspace_size.argtypes = [i32, i32, i32, psz]
        L.qgemm_w8a8_workspace_size.argtypes = [i32, pq, psz]
        L.qrepack_tiles_size.argtypes = [pq, psz]
        L.qrepack_tiles.argtypes = [pq, vp, sz, vp]
        L.qgemm_tiles_workspace_size.argtypes = [i32, pq, psz]
        L.qgemm_forward_tiles.argtypes = [vp, i32, i32, pq, vp, vp, i32, ctypes.c_int, vp, sz, vp]
        L.qgemm_forward_w8a8.argtypes = [vp, i32, i32, pq, vp, i32, ctypes.c_int, vp, sz, vp]
        L.qdiag_layer.argtypes = [vp, pq, f32, vp, vp, vp, sz, vp]
        L.qgemm_forward_multi.argtypes = [vp, i32, i32, pq, i32, ctypes.POINTER(vp), pi32, ctypes.c_int, vp, sz, vp]
        i64, pc, pb = ctypes.c_int64, ctypes.POINTER(QgKvCache), ctypes.POINTER(QgKvBatch)
        L.qkv_append.argtypes = [pc, pb, ctypes.POINTER(QgRope), vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, vp, i64,
                                 vp]
        pc8, pn = ctypes.POINTER(QgKv8Cache), ctypes.POINTER(QgHeadNorm)
        L.qkv_append_norm.argtypes = [pc, pb, pn, ctypes.POINTER(QgRope), vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, vp,
                                      i64, vp]
        L.qkv8_append.argtypes = [pc8, pb, pn, ctypes.POINTER(QgRope), vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, vp,
                                  i64, ctypes.c_int, vp]
        L.qkv8_read.argtypes = [pc8, pb, vp, i64, vp, i64, ctypes.c_int, vp]
        L.qattn_workspace_size.argtypes = [pc, pb, i32, psz]
        L.qattn_forward.argtypes = [pc, pb, vp, i64, i32, f32, vp, i64, ctypes.c_int, vp, vp, sz, vp]
        L.qattn8_workspace_size.argtypes = [pc8, pb, i32, psz]
        L.qattn8_forward.argtypes = [pc8, pb, vp, i64, i32, ctypes.c_int, f32, vp, i64, ctypes.c_int, vp, vp, sz, vp]
        for name in ABI_FUNCTIONS[:-1]:
            getattr(L, name).restype = ctypes.c_int
        L.qgemm_last_error.argtypes = []
        L.qgemm_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def last_error() -> str:
    return lib().qgemm_last_error().decode()


def _check(st: int, where: str):
    if st != QG_OK:
        raise QgError(st, where, last_error())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _as_stream(stream) -> torch.cuda.Stream:
    """torch's view of a stream argument that is not None."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle in (0, 1):   # the legacy default stream, by either of its handles
        return torch.cuda.default_stream()
    return torch.cuda.ExternalStream(handle)


def _on_stream(f):
    """Runs f with its ``stream`` argument as the current stream: a block of
    the caching allocator is reused in the order of the stream it was allocated
    on, so what f allocates for kernels of another stream must come from there."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(_as_stream(stream)):
            return f(*args, **kw)
    return call


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() else None


# --------------------------------------------------------------------- sizes
def qpack_query_sizes(N: int, K: int, bits: int, group: int, outlier_frac: float = 0.0) -> dict:
    p, s, z, c = (ctypes.c_size_t() for _ in range(4))
    n = ctypes.c_int32()
    _check(lib().qpack_query_sizes(N, K, bits, group, outlier_frac, ctypes.byref(p), ctypes.byref(s),
                                   ctypes.byref(z), ctypes.byref(c), ctypes.byref(n)), "qpack_query_sizes")
    return dict(packed=p.value, scale=s.value, zp=z.value, codebook=c.value, nnz=n.value)


def qpack_workspace_size(N: int, K: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().qpack_workspace_size(N, K, ctypes.byref(b)), "qpack_workspace_size")
    return b.value


# --------------------------------------------------------------------- weights
@dataclass
class QWeight:
    """A quantized matrix in device memory (canonical planar layout)."""
    N: int
    K: int
    bits: int
    group: int
    packed: torch.Tensor                 # uint8 [N, K*bits/8]
    scale: torch.Tensor | None           # int16 (fp16 bits) [N, K/group]
    zp: torch.Tensor | None              # uint8 [N, K/group]
    codebook: torch.Tensor | None        # int16 (fp16 bits) [N, K/group, 4]
    row_ptr: torch.Tensor | None         # int32 [N+1]
    col: torch.Tensor | None             # int32 [nnz]
    val: torch.Tensor | None             # int16 (fp16 bits) [nnz]
    nnz: int = 0
    # 8-bit (E4M3) scales in place of ``scale``, with the fp16 fallback list
    scale8: torch.Tensor | None = None       # uint8 [N, K/group], 0x7F = fallback
    scale8_exp: torch.Tensor | None = None   # int32 [1]: the matrix exponent E
    fb_row_ptr: torch.Tensor | None = None   # int32 [N+1]
    fb_col: torch.Tensor | None = None       # int32 [fb_cap]
    fb_val: torch.Tensor | None = None       # int16 (fp16 bits) [fb_cap]

    @staticmethod
    def empty(N: int, K: int, bits: int, group: int, outlier_frac: float = 0.0, device="cuda",
              scale_fmt: str = "fp16", fb_cap: int | None = None) -> "QWeight":
        """Buffers for a quantized matrix.  scale_fmt 'fp8': 8-bit scales
        with a fallback list of fb_cap entries (default: 1 % of the groups,
        at least 64)."""
        sz = qpack_query_sizes(N, K, bits, group, outlier_frac)
        ng = K // group
        u8, i16, i32 = torch.uint8, torch.int16, torch.int32
        nnz = sz["nnz"]
        f8 = scale_fmt == "fp8"
        if f8 and fb_cap is None:
            fb_cap = max(64, N * ng // 100)
        return QWeight(
            N, K, bits, group,
            packed=torch.empty((N, K * bits // 8), dtype=u8, device=device),
            scale=torch.empty((N, ng), dtype=i16, device=device) if bits != 2 and not f8 else None,
            zp=torch.empty((N, ng), dtype=u8, device=device) if bits != 2 else None,
            codebook=torch.empty((N, ng, 4), dtype=i16, device=device) if bits == 2 else None,
            row_ptr=torch.empty(N + 1, dtype=i32, device=device),
            col=torch.empty(max(nnz, 1), dtype=i32, device=device)[:nnz],
            val=torch.empty(max(nnz, 1), dtype=i16, device=device)[:nnz],
            nnz=nnz,
            scale8=torch.empty((N, ng), dtype=u8, device=device) if f8 else None,
            scale8_exp=torch.zeros(1, dtype=i32, device=device) if f8 else None,
            fb_row_ptr=torch.zeros(N + 1, dtype=i32, device=device) if f8 else None,
            fb_col=torch.empty(max(fb_cap, 1), dtype=i32, device=device)[:fb_cap] if f8 else None,
            fb_val=torch.empty(max(fb_cap, 1), dtype=i16, device=device)[:fb_cap] if f8 else None)

    @property
    def fb_cap(self) -> int:
        return 0 if self.fb_col is None else int(self.fb_col.numel())

    def desc(self) -> QgQWeight:
        return QgQWeight(self.N, self.K, self.bits, self.group, _ptr(self.packed), _ptr(self.scale),
                         _ptr(self.zp), _ptr(self.codebook), self.nnz, _ptr(self.row_ptr),
                         _ptr(self.col), _ptr(self.val), _ptr(self.scale8), _ptr(self.scale8_exp),
                         _ptr(self.fb_row_ptr), _ptr(self.fb_col), _ptr(self.fb_val), self.fb_cap)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.packed, self.scale, self.zp, self.codebook, self.row_ptr, self.col, self.val,
                    self.scale8, self.scale8_exp, self.fb_row_ptr, self.fb_col, self.fb_val)
                   if t is not None)


@_on_stream
def qpack_quantize(W: torch.Tensor, bits: int, group: int, outlier_frac: float = 0.0,
                   out: QWeight | None = None, workspace: torch.Tensor | None = None, stream=None,
                   mode: str = "asymmetric", scale_fmt: str = "fp16", fb_cap: int | None = None) -> QWeight:
    """Quantize and pack W [N, K] (fp16, CUDA) on the device.  mode:
    'asymmetric' (qpack_quantize), 'symmetric' or 'linear2'
    (qpack_quantize_mode); scale_fmt 'fp8': 8-bit scales (bits 3..8)."""
    if W.dtype != torch.float16 or not W.is_cuda or W.dim() != 2:
        raise ValueError("W must be a 2-D float16 CUDA tensor")
    W = W.contiguous()
    N, K = W.shape
    qw = out if out is not None else QWeight.empty(N, K, bits, group, outlier_frac, W.device, scale_fmt, fb_cap)
    ws_bytes = qpack_workspace_size(N, K)
    ws = workspace if workspace is not None else torch.empty(ws_bytes, dtype=torch.uint8, device=W.device)
    d = qw.desc()
    if mode == "asymmetric":
        _check(lib().qpack_quantize(_ptr(W), outlier_frac, ctypes.byref(d), _ptr(ws), ws.numel(), _stream(stream)),
               "qpack_quantize")
    else:
        _check(lib().qpack_quantize_mode(_ptr(W), outlier_frac, QUANT_MODES[mode], ctypes.byref(d), _ptr(ws),
                                         ws.numel(), _stream(stream)), "qpack_quantize_mode")
    return qw


@_on_stream
def qpack_quantize_noalloc(W: torch.Tensor, bits: int, group: int, outlier_frac: float = 0.0,
                           out: QWeight | None = None, stream=None, scale_fmt: str = "fp16") -> QWeight:
    """qpack_quantize for callers that cannot allocate device memory: the
    library uses its own fixed scratch array (see include/qgemm.h).  Pass
    ``out`` (allocated beforehand) to keep this call allocation-free."""
    if W.dtype != torch.float16 or not W.is_cuda or W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D float16 CUDA tensor")
    N, K = W.shape
    qw = out if out is not None else QWeight.empty(N, K, bits, group, outlier_frac, W.device, scale_fmt)
    f = lib().qpack_quantize_noalloc
    f.argtypes = [ctypes.c_void_p, ctypes.c_float, ctypes.POINTER(QgQWeight), ctypes.c_void_p]
    f.restype = ctypes.c_int
    d = qw.desc()
    _check(f(_ptr(W), outlier_frac, ctypes.byref(d), _stream(stream)), "qpack_quantize_noalloc")
    return qw


def qgemm_workspace_size(M: int, qw: QWeight) -> int:
    b = ctypes.c_size_t()
    d = qw.desc()
    _check(lib().qgemm_workspace_size(M, ctypes.byref(d), ctypes.byref(b)), "qgemm_workspace_size")
    return b.value


@_on_stream
def qgemm_forward(x: torch.Tensor, qw: QWeight, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] (bf16, CUDA) times (dequant(W) + outliers)^T."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with unit inner stride")
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=x.device)
    yt = Y_BF16 if out.dtype == torch.bfloat16 else Y_F32
    if out.dtype not in (torch.float32, torch.bfloat16) or out.stride(1) != 1:
        raise ValueError("out must be float32 or bfloat16 with unit inner stride")
    need = qgemm_workspace_size(M, qw)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    d = qw.desc()
    _check(lib().qgemm_forward(_ptr(x), M, x.stride(0), ctypes.byref(d), _ptr(out), out.stride(0), yt,
                               _ptr(workspace) if need else None, workspace.numel() if need else 0,
                               _stream(stream)), "qgemm_forward")
    return out


@_on_stream
def qgemm_forward_multi(x: torch.Tensor, qws, outs=None, out_dtype: torch.dtype = torch.float32,
                        workspace: torch.Tensor | None = None, stream=None):
    """[y_q [M, N_q] for each weight]: the products of x with up to four
    weights that share K, bits and group, in one call."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with unit inner stride")
    M = x.shape[0]
    if outs is None:
        outs = [torch.empty((M, q.N), dtype=out_dtype, device=x.device) for q in qws]
    if len(outs) != len(qws):
        raise ValueError("one output per weight")
    yt = Y_BF16 if outs[0].dtype == torch.bfloat16 else Y_F32
    for o in outs:
        if o.dtype != outs[0].dtype or o.dtype not in (torch.float32, torch.bfloat16) or o.stride(1) != 1:
            raise ValueError("outputs must share one dtype (float32 or bfloat16) with unit inner stride")
    need = max(qgemm_workspace_size(M, q) for q in qws)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    descs = _desc_array(qws)
    ys = (ctypes.c_void_p * len(outs))(*[o.data_ptr() for o in outs])
    ld = (ctypes.c_int32 * len(outs))(*[o.stride(0) for o in outs])
    _check(lib().qgemm_forward_multi(_ptr(x), M, x.stride(0), descs, len(qws), ys, ld, yt,
                                     _ptr(workspace) if need else None, workspace.numel() if need else 0,
                                     _stream(stream)), "qgemm_forward_multi")
    return outs


def _desc_array(experts):
    arr = (QgQWeight * len(experts))()
    for i, q in enumerate(experts):
        arr[i] = q.desc()
    return arr


def qgemm_moe_workspace_size(T: int, k: int, experts) -> int:
    b = ctypes.c_size_t()
    arr = _desc_array(experts)
    _check(lib().qgemm_moe_workspace_size(T, k, len(experts), arr, ctypes.byref(b)), "qgemm_moe_workspace_size")
    return b.value


@_on_stream
def qgemm_moe_grouped(x: torch.Tensor, topk_ids: torch.Tensor, experts, out: torch.Tensor | None = None,
                      out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """y [T, k, N]: y[t, j] = x[t] . (dequant(W_e) + outliers_e)^T with e = topk_ids[t, j]."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor [T, K]")
    if topk_ids.dtype != torch.int32 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 tensor [T, k]")
    T, k = topk_ids.shape
    N = experts[0].N
    if out is None:
        out = torch.empty((T, k, N), dtype=out_dtype, device=x.device)
    yt = Y_BF16 if out.dtype == torch.bfloat16 else Y_F32
    arr = _desc_array(experts)
    need = qgemm_moe_workspace_size(T, k, experts)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_moe_grouped(_ptr(x), T, _ptr(topk_ids), k, arr, len(experts), _ptr(out), yt,
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "qgemm_moe_grouped")
    return out


@_on_stream
def qgemm_moe_grouped_multi(x: torch.Tensor, topk_ids: torch.Tensor, experts_per_product, outs=None,
                            out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                            stream=None) -> list:
    """[y_p]: the grouped product of each expert list in experts_per_product
    (at most 2 lists of equal length, all matrices of one shape, width and
    group) over one routing of topk_ids."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor [T, K]")
    if topk_ids.dtype != torch.int32 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 tensor [T, k]")
    n = len(experts_per_product)
    E = len(experts_per_product[0])
    if any(len(ex) != E for ex in experts_per_product):
        raise ValueError("every product needs the same number of experts")
    T, k = topk_ids.shape
    N = experts_per_product[0][0].N
    if outs is None:
        outs = [torch.empty((T, k, N), dtype=out_dtype, device=x.device) for _ in range(n)]
    if len(outs) != n:
        raise ValueError("one output per product")
    yt = Y_BF16 if outs[0].dtype == torch.bfloat16 else Y_F32
    if any(o.dtype != outs[0].dtype for o in outs):
        raise ValueError("outputs must share one dtype")
    arr = _desc_array([w for ex in experts_per_product for w in ex])
    ys = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    need = qgemm_moe_workspace_size(T, k, experts_per_product[0])
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_moe_grouped_multi(_ptr(x), T, _ptr(topk_ids), k, arr, E, n, ys, yt, _ptr(workspace),
                                         workspace.numel(), _stream(stream)), "qgemm_moe_grouped_multi")
    return outs


def qgemm_set_dependent_launch(enable: bool) -> None:
    """Programmatic dependent launch of the dense products (decode and tensor-core kernels) and of the paged-cache
    kernels, process-wide."""
    lib().qgemm_set_dependent_launch.argtypes = [ctypes.c_int32]
    _check(lib().qgemm_set_dependent_launch(1 if enable else 0), "qgemm_set_dependent_launch")


def qgemm_device_status(reset: bool = False) -> int:
    """Status word of the library's kernels on the current device: 0 (QG_OK),
    QG_ERR_TIMEOUT (-6) after a bounded wait gave up, QG_ERR_DEVICE_STATUS (-7)
    after a length, offset, page or position outside its bounds,
    QG_ERR_WORKSPACE (-4) after a fallback list over capacity.  Synchronizes the
    device."""
    v = ctypes.c_int32(0)
    _check(lib().qgemm_device_status(ctypes.byref(v), 1 if reset else 0), "qgemm_device_status")
    return v.value


@_on_stream
def qgemm_selftest_bounded_wait(poll_limit: int = 2, stream=None) -> None:
    """Launch the kernel whose bounded mbarrier wait must give up; afterwards
    qgemm_device_status() reads QG_ERR_TIMEOUT (-6)."""
    _check(lib().qgemm_selftest_bounded_wait(poll_limit, _stream(stream)), "qgemm_selftest_bounded_wait")


class QgDiag(ctypes.Structure):
    """Mirror of ``qg_diag`` in include/qgemm.h."""
    _fields_ = [("max_abs_err", ctypes.c_double), ("rmse", ctypes.c_double), ("cosine", ctypes.c_double),
                ("max_range_ratio", ctypes.c_double), ("groups_over", ctypes.c_int64)]


@_on_stream
def qdiag_layer(W: torch.Tensor, qw: QWeight, threshold: float = 8.0, ratio: bool = False, stream=None):
    """Diagnostics of qw against the original fp16 W [N, K] (CUDA), computed
    on the device: dict of max_abs_err, rmse, cosine, max_range_ratio,
    groups_over (and the per-group ratio tensor [N, K/group] if asked).
    Reading the result synchronizes the stream."""
    if W.dtype != torch.float16 or not W.is_cuda or tuple(W.shape) != (qw.N, qw.K) or not W.is_contiguous():
        raise ValueError("W must be the contiguous fp16 CUDA [N, K] matrix of qw")
    b = ctypes.c_size_t()
    _check(lib().qdiag_workspace_size(qw.N, qw.K, qw.group, ctypes.byref(b)), "qdiag_workspace_size")
    ws = torch.empty(max(b.value, 1), dtype=torch.uint8, device=W.device)
    out = torch.zeros(5, dtype=torch.float64, device=W.device)   # one qg_diag (40 bytes)
    r = torch.empty((qw.N, qw.K // qw.group), dtype=torch.float32, device=W.device) if ratio else None
    d = qw.desc()
    _check(lib().qdiag_layer(_ptr(W), ctypes.byref(d), threshold, _ptr(r), _ptr(out), _ptr(ws), ws.numel(),
                             _stream(stream)), "qdiag_layer")
    raw = out.cpu().numpy().tobytes()
    res = QgDiag.from_buffer_copy(raw)
    o = dict(max_abs_err=res.max_abs_err, rmse=res.rmse, cosine=res.cosine, max_range_ratio=res.max_range_ratio,
             groups_over=int(res.groups_over))
    if ratio:
        o["ratio"] = r
    return o


@_on_stream
def qgemm_forward_w8a8(x: torch.Tensor, qw: QWeight, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """W8A8 decode product (M <= 16): x [M, K] bf16 quantized to int8 per token
    inside the call, times the 8-bit weight qw."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with unit inner stride")
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=x.device)
    yt = Y_BF16 if out.dtype == torch.bfloat16 else Y_F32
    b = ctypes.c_size_t()
    d = qw.desc()
    _check(lib().qgemm_w8a8_workspace_size(M, ctypes.byref(d), ctypes.byref(b)), "qgemm_w8a8_workspace_size")
    if b.value and (workspace is None or workspace.numel() < b.value):
        workspace = torch.empty(b.value, dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_forward_w8a8(_ptr(x), M, x.stride(0), ctypes.byref(d), _ptr(out), out.stride(0), yt,
                                    _ptr(workspace) if b.value else None, workspace.numel() if b.value else 0,
                                    _stream(stream)), "qgemm_forward_w8a8")
    return out


@_on_stream
def qrepack_tiles(qw: QWeight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The tile-ordered copy of qw (uint8 CUDA tensor) for qgemm_forward_tiles."""
    b = ctypes.c_size_t()
    d = qw.desc()
    _check(lib().qrepack_tiles_size(ctypes.byref(d), ctypes.byref(b)), "qrepack_tiles_size")
    if out is None:
        out = torch.empty(b.value, dtype=torch.uint8, device=qw.packed.device)
    _check(lib().qrepack_tiles(ctypes.byref(d), _ptr(out), out.numel(), _stream(stream)), "qrepack_tiles")
    return out


@_on_stream
def qgemm_forward_tiles(x: torch.Tensor, qw: QWeight, tiles: torch.Tensor, out: torch.Tensor | None = None,
                        out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """y = x . (dequant(W) + outliers)^T on the tensor cores from the tile-ordered copy."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with unit inner stride")
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=x.device)
    yt = Y_BF16 if out.dtype == torch.bfloat16 else Y_F32
    d = qw.desc()
    b = ctypes.c_size_t()
    _check(lib().qgemm_tiles_workspace_size(M, ctypes.byref(d), ctypes.byref(b)), "qgemm_tiles_workspace_size")
    if b.value and (workspace is None or workspace.numel() < b.value):
        workspace = torch.empty(b.value, dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_forward_tiles(_ptr(x), M, x.stride(0), ctypes.byref(d), _ptr(tiles), _ptr(out), out.stride(0),
                                     yt, _ptr(workspace) if b.value else None, workspace.numel() if b.value else 0,
                                     _stream(stream)), "qgemm_forward_tiles")
    return out


# --------------------------------------------------------------------- paged cache
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}   # qg_dtype


class KVCache:
    """Pages of cached keys and values: k and v [num_pages, page_size, heads_kv,
    head_dim] (bf16 or fp16, CUDA) with one set of strides, in any order with
    the head's values contiguous."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-D with the same shape, strides and dtype")
        if k.dtype not in (torch.bfloat16, torch.float16) or not k.is_cuda or not v.is_cuda or k.stride(3) != 1:
            raise ValueError("k and v must be bfloat16 or float16 CUDA tensors with unit inner stride")
        if k.device != v.device:
            raise ValueError("k and v must lie on one device")
        self.k, self.v, self.dtype, self.device = k, v, k.dtype, k.device
        self.index = k.get_device()
        self.num_pages, self.page_size, self.heads_kv, self.head_dim = k.shape
        self._desc = QgKvCache(k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], *k.shape, *k.stride()[:3])
        self._ref = ctypes.byref(self._desc)

    @staticmethod
    def empty(num_pages: int, page_size: int, heads_kv: int, head_dim: int, dtype: torch.dtype = torch.bfloat16,
              device="cuda") -> "KVCache":
        """Pages with heads first: a head's rows of a page are one contiguous run."""
        k, v = (torch.empty((num_pages, heads_kv, page_size, head_dim), dtype=dtype, device=device).transpose(1, 2)
                for _ in range(2))
        return KVCache(k, v)


KV8_BLOCK = 16   # places of a page that share a scale


class KVCache8:
    """Pages of keys and values in 8 bits: codes k and v [num_pages, page_size,
    heads_kv, head_dim] (torch.float8_e4m3fn, CUDA) with one set of strides, in
    any order with the head's codes contiguous, and for each block of 16 places
    and head the byte of a power of two, k_scale and v_scale [num_pages,
    page_size / 16, heads_kv] (uint8) with one set of strides in any order.  A
    value is code * 2^(byte - 127)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-D with the same shape, strides and dtype")
        if k.dtype != torch.float8_e4m3fn or not k.is_cuda or k.stride(3) != 1:
            raise ValueError("k and v must be float8_e4m3fn CUDA tensors with unit inner stride")
        blocks = (k.shape[0], k.shape[1] // KV8_BLOCK, k.shape[2])
        if tuple(k_scale.shape) != blocks or tuple(v_scale.shape) != blocks or k_scale.stride() != v_scale.stride():
            raise ValueError(f"k_scale and v_scale must be {list(blocks)} with the same strides")
        if k_scale.dtype != torch.uint8 or v_scale.dtype != torch.uint8:
            raise ValueError("k_scale and v_scale must be uint8")
        self.index = k.get_device()
        if any(t.get_device() != self.index for t in (v, k_scale, v_scale)):
            raise ValueError("k, v, k_scale and v_scale must lie on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device = k.dtype, k.device
        self.num_pages, self.page_size, self.heads_kv, self.head_dim = k.shape
        self._desc = QgKv8Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *k.shape,
                                *k.stride()[:3], *k_scale.stride())
        self._ref = ctypes.byref(self._desc)

    @staticmethod
    def empty(num_pages: int, page_size: int, heads_kv: int, head_dim: int, device="cuda") -> "KVCache8":
        """Pages with heads first: a head's rows of a page are one contiguous run, and so are its scales."""
        k, v = (torch.empty((num_pages, heads_kv, page_size, head_dim), dtype=torch.float8_e4m3fn,
                            device=device).transpose(1, 2) for _ in range(2))
        ks, vs = (torch.empty((num_pages, heads_kv, page_size // KV8_BLOCK), dtype=torch.uint8,
                              device=device).transpose(1, 2) for _ in range(2))
        return KVCache8(k, v, ks, vs)


class KVBatch:
    """Sequences over one cache (``qg_kv_batch``): own pages table [B, width]
    and own lengths kv_len [B] (new tokens counted), new tokens per sequence
    cu_q [B + 1] (None: one each), all int32 on the device and read when the
    kernels run; pages and length of the prefix they share; and host bounds
    max_kv (own tokens), max_q (new tokens) and tokens (rows of q/k/v;
    default B, one each)."""

    def __init__(self, table: torch.Tensor | None, kv_len: torch.Tensor, max_kv: int, cu_q: torch.Tensor | None = None,
                 max_q: int = 1, tokens: int | None = None, prefix_table: torch.Tensor | None = None,
                 prefix_len: int = 0):
        B = kv_len.numel()
        for name, t, n in (("kv_len", kv_len, B), ("cu_q", cu_q, B + 1), ("prefix_table", prefix_table, None)):
            if t is None:
                continue
            if t.dtype != torch.int32 or not t.is_cuda or t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
                raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
            if n is not None and t.numel() != n:
                raise ValueError(f"{name} must have {n} entries")
        if table is not None:
            if table.dtype != torch.int32 or not table.is_cuda or table.dim() != 2 or table.shape[0] != B or \
                    (table.shape[1] > 1 and table.stride(1) != 1):
                raise ValueError("table must be an int32 CUDA tensor [B, width] with unit inner stride")
        self.index = kv_len.get_device()
        for name, t in (("table", table), ("cu_q", cu_q), ("prefix_table", prefix_table)):
            if t is not None and t.get_device() != self.index:
                raise ValueError(f"{name} must lie on the device of kv_len")
        if cu_q is None and tokens not in (None, B):
            raise ValueError("without cu_q every sequence has one new token")
        if cu_q is not None and tokens is None:
            raise ValueError("tokens (rows of q, k and v) is needed with cu_q")
        self.table, self.kv_len, self.cu_q, self.prefix_table = table, kv_len, cu_q, prefix_table
        self.sequences, self.tokens, self.max_q, self.max_kv = B, B if tokens is None else tokens, max_q, max_kv
        self.prefix_len = prefix_len
        self._width = 0 if table is None else table.shape[1]
        self._shared = 0 if prefix_table is None else prefix_table.numel()
        ld = 0 if table is None else (table.stride(0) if B > 1 else table.shape[1])
        if ld < self._width:
            raise ValueError("rows of table must not overlap")
        self._desc = QgKvBatch(B, self.tokens, max_q, max_kv, ld, prefix_len, _ptr(table), _ptr(kv_len), _ptr(cu_q),
                               _ptr(prefix_table))
        self._ref = ctypes.byref(self._desc)

    def check(self, cache: KVCache):
        """The tables hold an entry for every page the bounds reach, and lie on
        the cache's device."""
        if self.index != cache.index:
            raise ValueError(f"the batch lies on cuda:{self.index}, the cache on cuda:{cache.index}")
        if self._width * cache.page_size < self.max_kv:
            raise ValueError(f"table width {self._width} holds fewer than max_kv={self.max_kv} tokens")
        if self._shared * cache.page_size < self.prefix_len:
            raise ValueError(f"prefix_table of {self._shared} pages holds fewer than prefix_len={self.prefix_len} tokens")


def _rows(t: torch.Tensor, name: str, T: int, heads: int, cache: KVCache) -> int:
    """Token stride of an array [T, heads, head_dim] on the cache's device whose heads are contiguous (heads 0: any
    number)."""
    shape, dim = t.shape, cache.head_dim
    if len(shape) == 3 and t.get_device() == cache.index:
        n, h, d = shape
        if n == T and d == dim and (h == heads or not heads):
            st, sh, sd = t.stride()
            if sd == 1 and (sh == dim or h == 1):
                return st if T > 1 else h * dim
            raise ValueError(f"the heads of a token of {name} must be contiguous")
    raise ValueError(f"{name} must be a tensor [{T}, {heads or 'heads'}, {dim}] on cuda:{cache.index}")


def _launch_stream(cache: KVCache) -> int:
    """The current stream.  The library launches on the current device (with a
    stream argument, the stream's), which must be the cache's."""
    if torch.cuda.current_device() != cache.index:
        raise ValueError(f"the cache lies on cuda:{cache.index}, the current device is cuda:{torch.cuda.current_device()}")
    # the handle alone: torch.cuda.current_stream makes an object for it, 1.4 us of a call that takes 10 on the host
    return torch._C._cuda_getCurrentRawStream(cache.index)


def _norm(q_norm, k_norm, eps: float, cache):
    """The norms' weights [head_dim], as the library takes them (None: nothing is normed)."""
    some = q_norm if q_norm is not None else k_norm
    if some is None:
        return None
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.dtype != some.dtype or w.dtype not in _DTYPES or w.get_device() != cache.index or
                              w.shape != (cache.head_dim,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor [{cache.head_dim}] on cuda:{cache.index}, both norms of one "
                             "dtype (float32, bfloat16 or float16)")
    return QgHeadNorm(None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                      _DTYPES[some.dtype], eps)


@_on_stream
def qkv_append(cache: "KVCache | KVCache8", batch: KVBatch, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
               rope: torch.Tensor | None = None, positions: torch.Tensor | None = None, interleaved: bool = False,
               q_out: torch.Tensor | None = None, stream=None, q_norm: torch.Tensor | None = None,
               k_norm: torch.Tensor | None = None, eps: float = 1e-6, q_dtype: torch.dtype | None = None) -> torch.Tensor | None:
    """Write the batch's new tokens k and v [T, heads_kv, head_dim] (fp32,
    bf16 or fp16) to their pages, k turned by its position; returns q [T,
    heads_q, head_dim] turned, in the cache's type.  rope: fp32 [positions,
    R], row p the R/2 cosines and then the R/2 sines of position p (None: no
    rotation); positions: int32 [T] in place of the batch's own.

    q_norm, k_norm: weights [head_dim] (fp32, bf16 or fp16) of norms applied to
    each head of q and k before the rotation, x * w / sqrt(mean(x^2) + eps).

    With a :class:`KVCache8`, k and v are quantised to its codes and scales, and
    q is returned in q_dtype (default: q's own type, bf16 for fp32)."""
    T, D, xt, eight = batch.tokens, cache.head_dim, k.dtype, isinstance(cache, KVCache8)
    batch.check(cache)
    ldk, ldv = _rows(k, "k", T, cache.heads_kv, cache), _rows(v, "v", T, cache.heads_kv, cache)
    if v.dtype != xt or (q is not None and q.dtype != xt) or xt not in _DTYPES:
        raise ValueError("q, k and v must share one dtype (float32, bfloat16 or float16)")
    if q_dtype is None:
        q_dtype = cache.dtype if not eight else q_out.dtype if q_out is not None else \
            torch.bfloat16 if xt == torch.float32 else xt
    if q_dtype not in (torch.bfloat16, torch.float16) or (not eight and q_dtype != cache.dtype):
        raise ValueError("q is written in the cache's dtype" if not eight else "q is written in bfloat16 or float16")
    heads_q = ldq = ldq_out = 0
    q_at = out_at = None
    if q is not None:
        ldq = _rows(q, "q", T, 0, cache)
        heads_q = q.shape[1]
        if q_out is None:
            q_out = torch.empty((T, heads_q, D), dtype=q_dtype, device=cache.device)
            ldq_out = heads_q * D
        else:
            ldq_out = _rows(q_out, "q_out", T, heads_q, cache)
            if q_out.dtype != q_dtype:
                raise ValueError("q_out must have the cache's dtype" if not eight else "q_out must have q_dtype")
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    elif q_norm is not None:
        raise ValueError("q_norm without q")
    turn = None
    if rope is not None:
        if rope.dtype != torch.float32 or rope.get_device() != cache.index or rope.dim() != 2 or not rope.is_contiguous():
            raise ValueError(f"rope must be a contiguous float32 tensor [positions, R] on cuda:{cache.index}")
        if positions is not None and (positions.dtype != torch.int32 or positions.get_device() != cache.index or
                                      positions.shape != (T,) or not positions.is_contiguous()):
            raise ValueError(f"positions must be a contiguous int32 tensor [{T}] on cuda:{cache.index}")
        turn = QgRope(rope.data_ptr(), _ptr(positions), *rope.shape, interleaved)
    norm = _norm(q_norm, k_norm, eps, cache)
    rows = (q_at, ldq, heads_q, k.data_ptr(), ldk, v.data_ptr(), ldv, _DTYPES[xt], out_at, ldq_out)
    stream = _launch_stream(cache)
    if eight:
        st = lib().qkv8_append(cache._ref, batch._ref, norm, turn, *rows, _DTYPES[q_dtype], stream)
    elif norm is not None:
        st = lib().qkv_append_norm(cache._ref, batch._ref, norm, turn, *rows, stream)
    else:
        st = lib().qkv_append(cache._ref, batch._ref, turn, *rows, stream)
    if st != QG_OK:
        _check(st, "qkv8_append" if eight else "qkv_append" if norm is None else "qkv_append_norm")
    return q_out


@_on_stream
def qkv_read(cache: KVCache8, batch: KVBatch, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
             dtype: torch.dtype | None = None, stream=None) -> tuple:
    """k, v [T, heads_kv, head_dim] (dtype: bf16 by default, fp16 or fp32): the
    values that an 8-bit cache holds for the batch's tokens, the rows that
    qkv_append would write (with cu_q the sums of kv_len, whole sequences)."""
    T, H, D = batch.tokens, cache.heads_kv, cache.head_dim
    batch.check(cache)
    if not isinstance(cache, KVCache8):
        raise ValueError("qkv_read reads a KVCache8")
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else torch.bfloat16
    if k_out is None:
        k_out = torch.empty((T, H, D), dtype=dtype, device=cache.device)
    if v_out is None:
        v_out = torch.empty((T, H, D), dtype=dtype, device=cache.device)
    if k_out.dtype != dtype or v_out.dtype != dtype or dtype not in _DTYPES:
        raise ValueError("k_out and v_out must share one dtype (float32, bfloat16 or float16)")
    ldk, ldv = _rows(k_out, "k_out", T, H, cache), _rows(v_out, "v_out", T, H, cache)
    st = lib().qkv8_read(cache._ref, batch._ref, k_out.data_ptr(), ldk, v_out.data_ptr(), ldv, _DTYPES[dtype],
                         _launch_stream(cache))
    if st != QG_OK:
        _check(st, "qkv8_read")
    return k_out, v_out


def qattn_workspace_size(cache: "KVCache | KVCache8", batch: KVBatch, heads_q: int) -> int:
    b = ctypes.c_size_t()
    name = "qattn8_workspace_size" if isinstance(cache, KVCache8) else "qattn_workspace_size"
    _check(getattr(lib(), name)(cache._ref, batch._ref, heads_q, ctypes.byref(b)), name)
    return b.value


@_on_stream
def qattn_forward(q: torch.Tensor, cache: "KVCache | KVCache8", batch: KVBatch, scale: float | None = None,
                  out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                  lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [T, heads_q, head_dim] (default: of q's type): attention of the new
    tokens q (of the cache's type; bf16 or fp16 with a :class:`KVCache8`) over
    the shared prefix and their own cached tokens.  scale: 1 / sqrt(head_dim) by
    default; lse: fp32 [T, heads_q] to receive the log of each row's sum of
    exponentials."""
    T, D, eight = batch.tokens, cache.head_dim, isinstance(cache, KVCache8)
    batch.check(cache)
    if eight and q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q must be bfloat16 or float16")
    if not eight and q.dtype != cache.dtype:
        raise ValueError("q must have the cache's dtype")
    ldq = _rows(q, "q", T, 0, cache)
    heads_q = q.shape[1]
    if out is None:
        out = torch.empty((T, heads_q, D), dtype=out_dtype or q.dtype, device=cache.device)
        ldo = heads_q * D
    else:
        ldo = _rows(out, "out", T, heads_q, cache)
    if out.dtype not in _DTYPES:
        raise ValueError("out must be float32, bfloat16 or float16")
    if lse is not None and (lse.dtype != torch.float32 or lse.get_device() != cache.index or lse.shape != (T, heads_q) or
                            not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor [{T}, {heads_q}] on cuda:{cache.index}")
    if workspace is None:
        workspace = torch.empty(qattn_workspace_size(cache, batch, heads_q), dtype=torch.uint8, device=cache.device)
    elif workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{cache.index}")
    rest = (D ** -0.5 if scale is None else scale, out.data_ptr(), ldo, _DTYPES[out.dtype],
            None if lse is None else lse.data_ptr(), workspace.data_ptr() or None,
            workspace.numel() * workspace.element_size(), _launch_stream(cache))
    if eight:
        st = lib().qattn8_forward(cache._ref, batch._ref, q.data_ptr(), ldq, heads_q, _DTYPES[q.dtype], *rest)
    else:
        st = lib().qattn_forward(cache._ref, batch._ref, q.data_ptr(), ldq, heads_q, *rest)
    if st != QG_OK:
        _check(st, "qattn8_forward" if eight else "qattn_forward")
    return out
