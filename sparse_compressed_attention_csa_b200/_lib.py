"""ctypes binding of libcsa.so (the C ABI in include/csa.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  Functions take torch CUDA tensors (torch is used for device
memory and streams), check dtype / contiguity / device, and pass raw
pointers and sizes through.  A missing library raises immediately: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

CSA_F32, CSA_BF16 = 0, 1
CSA_OP_COMPRESS, CSA_OP_INDEX_TOPK, CSA_OP_SPARSE_ATTN, CSA_OP_HCA_ATTN, CSA_OP_TOPK_SELECT = range(5)
CSA_OP_SPARSE_ATTN_PAGED, CSA_OP_HCA_ATTN_PAGED = 5, 6

STATUS = {
    0: "CSA_OK", 1: "CSA_ERR_INVALID_ARGUMENT", 2: "CSA_ERR_MISALIGNED",
    3: "CSA_ERR_UNSUPPORTED_SHAPE", 4: "CSA_ERR_UNSUPPORTED_DEVICE",
    5: "CSA_ERR_WORKSPACE_TOO_SMALL", 6: "CSA_ERR_CUDA", 7: "CSA_ERR_DEVICE_TIMEOUT",
    8: "CSA_ERR_DEVICE_BOUNDS",
}


class CsaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


class csa_params_t(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("theta", ctypes.c_float),
                ("scale", ctypes.c_float), ("n_heads", ctypes.c_int32),
                ("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("window", ctypes.c_int32), ("width", ctypes.c_int32),
                ("stride", ctypes.c_int32), ("pos_offset", ctypes.c_int32),
                ("rope_factor", ctypes.c_float), ("rope_orig_ctx", ctypes.c_int32),
                ("rope_beta_fast", ctypes.c_float), ("rope_beta_slow", ctypes.c_float)]


@dataclass(frozen=True)
class Params:
    """Layer constants (defaults: the measured model's CSA layer)."""
    d: int = 512
    rope_dim: int = 64
    theta: float = 10000.0
    scale: float | None = None  # None -> 1/sqrt(d)
    n_heads: int = 128
    idx_heads: int = 64
    idx_dim: int = 128
    topk: int = 1024
    window: int = 128
    width: int = 8
    stride: int = 4
    pos_offset: int = 0
    rope_factor: float = 1.0      # YaRN factor s (1: plain RoPE)
    rope_orig_ctx: int = 0        # YaRN original context L
    rope_beta_fast: float = 32.0  # YaRN beta
    rope_beta_slow: float = 1.0   # YaRN alpha

    def __getstate__(self):
        """The fields alone: what calls keep here (the C struct, a pointer to
        it, workspace sizes) is not copied or pickled."""
        return {f: self.__dict__[f] for f in self.__dataclass_fields__}

    def c(self) -> csa_params_t:
        """The C struct, built once per (immutable) parameter set; the
        library only reads it during a call."""
        cs = self.__dict__.get("_c")
        if cs is None:
            sc = self.scale if self.scale is not None else 1.0 / math.sqrt(self.d)
            cs = csa_params_t(self.d, self.rope_dim, self.theta, sc, self.n_heads,
                              self.idx_heads, self.idx_dim, self.topk, self.window, self.width,
                              self.stride, self.pos_offset, self.rope_factor, self.rope_orig_ctx,
                              self.rope_beta_fast, self.rope_beta_slow)
            object.__setattr__(self, "_c", cs)
        return cs

    def ref(self):
        """A pointer to the C struct, kept with it."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = ctypes.byref(self.c())
            object.__setattr__(self, "_ref", r)
        return r


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_PP = ctypes.POINTER(csa_params_t)


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"CUDA library {LIB_PATH} is not built; run "
                          "sparse_compressed_attention_csa_b200.build.build() (there is no "
                          "CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.csa_abi_version.restype = ctypes.c_int
    lib.csa_status_string.restype = ctypes.c_char_p
    lib.csa_status_string.argtypes = [ctypes.c_int]
    lib.csa_last_error_detail.restype = ctypes.c_char_p
    lib.csa_workspace_size.argtypes = [_PP, ctypes.c_int, _I, _I, _I,
                                       ctypes.POINTER(ctypes.c_size_t)]
    lib.csa_compress.argtypes = [_PP, ctypes.c_int, _P, _P, _I, _I, _P, _P, _P]
    lib.csa_compress_append.argtypes = [_PP, ctypes.c_int, _P, _P, _P, _I, _I, _P, _P, _I, _P, _I,
                                        _P, _P, _I, _P]
    lib.csa_index_scores.argtypes = [_PP, ctypes.c_int, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P]
    lib.csa_topk_select.argtypes = [_PP, _P, _P, _P, _I, _I, _I, _P, _P, ctypes.c_size_t, _P]
    lib.csa_index_topk.argtypes = [_PP, ctypes.c_int, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P,
                                   ctypes.c_size_t, _P]
    lib.csa_sparse_attn.argtypes = [_PP, ctypes.c_int, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P,
                                    _I, _I, _P, _P, ctypes.c_size_t, _P]
    lib.hca_attn.argtypes = list(lib.csa_sparse_attn.argtypes)
    lib.csa_reuse_attn.argtypes = [_PP, ctypes.c_int, _I] + list(lib.csa_sparse_attn.argtypes[2:])
    lib.csa_quantize_fp8.argtypes = [ctypes.c_int, _P, ctypes.c_int64, _I, _P, _P, _P]
    lib.csa_sparse_attn_fp8.argtypes = [_PP, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _I,
                                        _I, _P, _P, ctypes.c_size_t, _P]
    lib.hca_attn_fp8.argtypes = list(lib.csa_sparse_attn_fp8.argtypes)
    lib.csa_index_topk_noalloc.argtypes = [_PP, ctypes.c_int, _P, _P, _P, _P, _P, _I, _I, _I, _P,
                                           _P]
    _L, _Z = ctypes.c_int64, ctypes.c_size_t
    lib.csa_norm_rope.argtypes = [_PP, ctypes.c_int, _I, ctypes.c_float, _P, _L, _I, _I, _P, _P, _P,
                                  _P, _L, _I, _I, _P, _P, _P, _I, _P, _P]
    lib.csa_quantize_mxfp4.argtypes = [ctypes.c_int, _P, _L, _L, _I, _P, _L, _P, _P, _P, _P]
    lib.csa_index_scores_mxfp4.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _I,
                                           _I, _P, _P]
    lib.csa_index_topk_mxfp4.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I,
                                         _P, _P, _Z, _P]
    lib.csa_sparse_attn_paged.argtypes = [_PP, ctypes.c_int, _P, _P, _P, _I, _I, _P, _I, _P, _P, _P,
                                          _P, _I, _P, _I, _I, _P, _P, _Z, _P]
    lib.hca_attn_paged.argtypes = list(lib.csa_sparse_attn_paged.argtypes)
    lib.csa_poll_device_error.argtypes = [_P]
    lib.csa_launch_count.restype = ctypes.c_uint64
    lib.csa_launch_count.argtypes = []
    lib.csa_set_wait_limit_ns.restype = None
    lib.csa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.csa_last_device_error_site.restype = ctypes.c_int32
    lib.csa_last_device_error_site.argtypes = []
    for f in ("csa_workspace_size", "csa_compress", "csa_index_scores", "csa_topk_select",
              "csa_index_topk", "csa_sparse_attn", "hca_attn", "csa_poll_device_error",
              "csa_compress_append", "csa_quantize_fp8", "csa_sparse_attn_fp8", "hca_attn_fp8",
              "csa_reuse_attn", "csa_norm_rope", "csa_quantize_mxfp4", "csa_index_scores_mxfp4",
              "csa_index_topk_mxfp4", "csa_sparse_attn_paged", "hca_attn_paged",
              "csa_index_topk_noalloc"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def lib():
    return _load()


def _check(st: int):
    if st != 0:
        raise CsaError(st, _load().csa_last_error_detail().decode(errors="replace"))


def _ptr(t):
    # a plain int: the c_void_p argtypes convert it
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The cudaStream_t of `stream`, or of the current stream of the current
    device (read through torch's raw-stream query, which skips building a
    Stream object on every call)."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return CSA_BF16
    if t.dtype == torch.float32:
        return CSA_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _req(t, name, dtype=None, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


_ws_sizes = {}


def csa_workspace_size(p: Params, op: int, B: int, Tq: int, n_max: int) -> int:
    """Bytes of workspace the call `op` needs (a pure function of the
    arguments and the current device, so answers are kept per device)."""
    import torch
    key = (p, op, B, Tq, n_max, torch.cuda.current_device() if torch.cuda.is_available() else -1)
    nb = _ws_sizes.get(key)
    if nb is None:
        n = ctypes.c_size_t(0)
        _check(_load().csa_workspace_size(ctypes.byref(p.c()), op, B, Tq, n_max,
                                          ctypes.byref(n)))
        nb = _ws_sizes[key] = int(n.value)
    return nb


def csa_compress(p: Params, x, gate, kv_cmp_out, kv_raw_rot_out=None, stream=None):
    """x, gate [B][T][d] -> kv_cmp_out [B][N][d] (+ kv_raw_rot_out [B][T][d])."""
    _req(x, "x", ndim=3)
    _req(gate, "gate", x.dtype, 3)
    _req(kv_cmp_out, "kv_cmp_out", x.dtype, 3)
    if kv_raw_rot_out is not None:
        _req(kv_raw_rot_out, "kv_raw_rot_out", x.dtype, 3)
    B, T, d = x.shape
    _check(_load().csa_compress(ctypes.byref(p.c()), _dtype_code(x), _ptr(x), _ptr(gate), B, T,
                                _ptr(kv_cmp_out), _ptr(kv_raw_rot_out), _stream(stream)))


def csa_compress_append(p: Params, x, gate, x_pos0, t_old, t_new, max_new: int, kv_cmp,
                        kv_raw=None, raw_pos0=None, stream=None):
    """Entries and raw rows completed by tokens t_old[b] .. t_new[b] - 1:
    x, gate [B][L][d] (row i = token x_pos0[b] + i) -> rows of kv_cmp
    [B][n_cap][d] (entry j at row j) and kv_raw [B][raw_cap][d] (token t at
    row t - raw_pos0[b])."""
    import torch
    _req(x, "x", ndim=3)
    _req(gate, "gate", x.dtype, 3)
    for t, n in ((x_pos0, "x_pos0"), (t_old, "t_old"), (t_new, "t_new")):
        _req(t, n, torch.int32, 1)
    _req(kv_cmp, "kv_cmp", x.dtype, 3)
    if kv_raw is not None:
        _req(kv_raw, "kv_raw", x.dtype, 3)
        _req(raw_pos0, "raw_pos0", torch.int32, 1)
    B, L, d = x.shape
    _check(_load().csa_compress_append(
        ctypes.byref(p.c()), _dtype_code(x), _ptr(x), _ptr(gate), _ptr(x_pos0), B, L, _ptr(t_old),
        _ptr(t_new), int(max_new), _ptr(kv_cmp), kv_cmp.shape[1], _ptr(kv_raw),
        _ptr(raw_pos0), kv_raw.shape[1] if kv_raw is not None else 0, _stream(stream)))


def csa_index_scores(p: Params, q_idx, w, k_idx, q_pos, n_cmp, scores, stream=None):
    """q_idx [B][Tq][H_I][d_I], w [B][Tq][H_I], k_idx [B][n_max][d_I] -> scores [B][Tq][n_max]."""
    import torch
    _req(q_idx, "q_idx", ndim=4)
    _req(w, "w", torch.float32, 3)
    _req(k_idx, "k_idx", q_idx.dtype, 3)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(n_cmp, "n_cmp", torch.int32, 1)
    _req(scores, "scores", torch.float32, 3)
    B, Tq = q_pos.shape
    n_max = k_idx.shape[1]
    _check(_load().csa_index_scores(ctypes.byref(p.c()), _dtype_code(q_idx), _ptr(q_idx), _ptr(w),
                                    _ptr(k_idx), _ptr(q_pos), _ptr(n_cmp), B, Tq, n_max,
                                    _ptr(scores), _stream(stream)))


def csa_topk_select(p: Params, scores, q_pos, n_cmp, idx_out, ws=None, stream=None):
    """scores [B][Tq][n_max] fp32 -> idx_out [B][Tq][topk] int32."""
    import torch
    _req(scores, "scores", torch.float32, 3)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(n_cmp, "n_cmp", torch.int32, 1)
    _req(idx_out, "idx_out", torch.int32, 3)
    B, Tq, n_max = scores.shape
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().csa_topk_select(ctypes.byref(p.c()), _ptr(scores), _ptr(q_pos), _ptr(n_cmp),
                                   B, Tq, n_max, _ptr(idx_out), _ptr(ws), nb, _stream(stream)))


def csa_index_topk(p: Params, q_idx, w, k_idx, q_pos, n_cmp, idx_out, ws, stream=None):
    """Indexer + top-k; ws: csa_workspace_size(CSA_OP_INDEX_TOPK) bytes."""
    import torch
    _req(q_idx, "q_idx", ndim=4)
    _req(w, "w", torch.float32, 3)
    _req(k_idx, "k_idx", q_idx.dtype, 3)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(n_cmp, "n_cmp", torch.int32, 1)
    _req(idx_out, "idx_out", torch.int32, 3)
    B, Tq = q_pos.shape
    n_max = k_idx.shape[1]
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().csa_index_topk(ctypes.byref(p.c()), _dtype_code(q_idx), _ptr(q_idx), _ptr(w),
                                  _ptr(k_idx), _ptr(q_pos), _ptr(n_cmp), B, Tq, n_max,
                                  _ptr(idx_out), _ptr(ws), nb, _stream(stream)))


def csa_index_topk_noalloc(p: Params, q_idx, w, k_idx, q_pos, n_cmp, idx_out, stream=None):
    """Indexer + top-k without a workspace, for callers that cannot allocate
    device memory.  Scores go to an 8 MiB array built into the library
    (B * Tq * n_max <= 2**21); calls that overlap on the GPU share it and race."""
    import torch
    _req(q_idx, "q_idx", ndim=4)
    _req(w, "w", torch.float32, 3)
    _req(k_idx, "k_idx", q_idx.dtype, 3)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(n_cmp, "n_cmp", torch.int32, 1)
    _req(idx_out, "idx_out", torch.int32, 3)
    B, Tq = q_pos.shape
    n_max = k_idx.shape[1]
    _check(_load().csa_index_topk_noalloc(ctypes.byref(p.c()), _dtype_code(q_idx), _ptr(q_idx),
                                          _ptr(w), _ptr(k_idx), _ptr(q_pos), _ptr(n_cmp), B, Tq,
                                          n_max, _ptr(idx_out), _stream(stream)))


def _attn(fn, p, q, q_pos, kv_cmp, sel, kv_raw, raw_pos0, n_raw, sink, out, ws, stream):
    import torch
    _req(q, "q", ndim=4)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(kv_cmp, "kv_cmp", q.dtype, 3)
    _req(kv_raw, "kv_raw", q.dtype, 3)
    _req(raw_pos0, "raw_pos0", torch.int32, 1)
    _req(n_raw, "n_raw", torch.int32, 1)
    _req(sink, "sink", torch.float32, 1)
    _req(out, "out", q.dtype, 4)
    B, Tq = q_pos.shape
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(fn(ctypes.byref(p.c()), _dtype_code(q), _ptr(q), _ptr(q_pos), _ptr(kv_cmp), _ptr(sel),
              kv_cmp.shape[1], _ptr(kv_raw), _ptr(raw_pos0), _ptr(n_raw), kv_raw.shape[1],
              _ptr(sink), B, Tq, _ptr(out), _ptr(ws), nb, _stream(stream)))


def csa_sparse_attn(p: Params, q, q_pos, kv_cmp, idx, kv_raw, raw_pos0, n_raw, sink, out,
                    ws=None, stream=None):
    """q [B][Tq][H][d], idx [B][Tq][topk] -> out [B][Tq][H][d]."""
    import torch
    _req(idx, "idx", torch.int32, 3)
    _attn(_load().csa_sparse_attn, p, q, q_pos, kv_cmp, idx, kv_raw, raw_pos0, n_raw, sink, out,
          ws, stream)


def csa_reuse_attn(p: Params, q, q_pos, kv_cmp, idx, kv_raw, raw_pos0, n_raw, sink, out, ws=None,
                   stream=None):
    """CSA2 Reuse layers: q [R][B][Tq][H][d], sink [R][H] -> out [R][B][Tq][H][d],
    every layer over the same entries, selection (idx [B][Tq][topk]) and window."""
    import torch
    _req(q, "q", ndim=5)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(kv_cmp, "kv_cmp", q.dtype, 3)
    _req(idx, "idx", torch.int32, 3)
    _req(kv_raw, "kv_raw", q.dtype, 3)
    _req(raw_pos0, "raw_pos0", torch.int32, 1)
    _req(n_raw, "n_raw", torch.int32, 1)
    _req(sink, "sink", torch.float32, 2)
    _req(out, "out", q.dtype, 5)
    R = q.shape[0]
    B, Tq = q_pos.shape
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().csa_reuse_attn(ctypes.byref(p.c()), _dtype_code(q), R, _ptr(q), _ptr(q_pos),
                                  _ptr(kv_cmp), _ptr(idx), kv_cmp.shape[1], _ptr(kv_raw),
                                  _ptr(raw_pos0), _ptr(n_raw), kv_raw.shape[1], _ptr(sink), B, Tq,
                                  _ptr(out), _ptr(ws), nb, _stream(stream)))


def hca_attn(p: Params, q, q_pos, kv_cmp, n_cmp, kv_raw, raw_pos0, n_raw, sink, out, ws=None,
             stream=None):
    """Dense attention over every visible entry + window."""
    import torch
    _req(n_cmp, "n_cmp", torch.int32, 1)
    _attn(_load().hca_attn, p, q, q_pos, kv_cmp, n_cmp, kv_raw, raw_pos0, n_raw, sink, out, ws,
          stream)


def csa_launch_count() -> int:
    """Kernels launched (or captured) by the library so far in this process."""
    return int(_load().csa_launch_count())


def csa_set_wait_limit_ns(ns: int = 0):
    """Limit of every bounded wait in the library's kernels (0: the 2 s
    default).  Read at launch; a diagnostic for exercising the timeout path."""
    _load().csa_set_wait_limit_ns(int(ns))


def csa_poll_device_error(stream=None):
    _check(_load().csa_poll_device_error(_stream(stream)))


def csa_last_device_error_site() -> int:
    """Kernel source line of the check behind the last device error polled."""
    return int(_load().csa_last_device_error_site())


def csa_quantize_fp8(rows, codes, scales, stream=None):
    """Cache rows [..., d] (bf16 or fp32, already rotated) -> E4M3 codes
    [..., d] uint8 and one fp32 scale per row [...]."""
    import torch
    _req(rows, "rows")
    _req(codes, "codes", torch.uint8, rows.dim())
    _req(scales, "scales", torch.float32, rows.dim() - 1)
    d = rows.shape[-1]
    n = rows.numel() // d if d else 0
    if tuple(codes.shape) != tuple(rows.shape) or tuple(scales.shape) != tuple(rows.shape[:-1]):
        raise ValueError("codes must match rows and scales its leading dims")
    _check(_load().csa_quantize_fp8(_dtype_code(rows), _ptr(rows), n, d, _ptr(codes), _ptr(scales),
                                    _stream(stream)))


def _attn_fp8(fn, p, q, q_pos, kv_cmp, cmp_scale, sel, kv_raw, raw_scale, raw_pos0, n_raw, sink,
              out, ws, stream):
    import torch
    _req(q, "q", torch.bfloat16, 4)
    _req(q_pos, "q_pos", torch.int32, 2)
    _req(kv_cmp, "kv_cmp", torch.uint8, 3)
    _req(cmp_scale, "cmp_scale", torch.float32, 2)
    _req(kv_raw, "kv_raw", torch.uint8, 3)
    _req(raw_scale, "raw_scale", torch.float32, 2)
    _req(raw_pos0, "raw_pos0", torch.int32, 1)
    _req(n_raw, "n_raw", torch.int32, 1)
    _req(sink, "sink", torch.float32, 1)
    _req(out, "out", torch.bfloat16, 4)
    B, Tq = q_pos.shape
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(fn(ctypes.byref(p.c()), _ptr(q), _ptr(q_pos), _ptr(kv_cmp), _ptr(cmp_scale), _ptr(sel),
              kv_cmp.shape[1], _ptr(kv_raw), _ptr(raw_scale), _ptr(raw_pos0), _ptr(n_raw),
              kv_raw.shape[1], _ptr(sink), B, Tq, _ptr(out), _ptr(ws), nb, _stream(stream)))


def csa_sparse_attn_fp8(p: Params, q, q_pos, kv_cmp, cmp_scale, idx, kv_raw, raw_scale, raw_pos0,
                        n_raw, sink, out, ws=None, stream=None):
    """As csa_sparse_attn over FP8 caches: kv_cmp [B][n_max][d] and kv_raw
    [B][raw_max][d] E4M3 codes with row scales [B][n_max], [B][raw_max]."""
    import torch
    _req(idx, "idx", torch.int32, 3)
    _attn_fp8(_load().csa_sparse_attn_fp8, p, q, q_pos, kv_cmp, cmp_scale, idx, kv_raw, raw_scale,
              raw_pos0, n_raw, sink, out, ws, stream)


def hca_attn_fp8(p: Params, q, q_pos, kv_cmp, cmp_scale, n_cmp, kv_raw, raw_scale, raw_pos0,
                 n_raw, sink, out, ws=None, stream=None):
    """As hca_attn over FP8 caches (codes and row scales)."""
    import torch
    _req(n_cmp, "n_cmp", torch.int32, 1)
    _attn_fp8(_load().hca_attn_fp8, p, q, q_pos, kv_cmp, cmp_scale, n_cmp, kv_raw, raw_scale,
              raw_pos0, n_raw, sink, out, ws, stream)


# ---------------------------------------------------------------------------
# The paged, 4-bit serving path.  These calls also check that every tensor is
# on the current device and that the shapes agree.

def _args(dev, *specs):
    """Addresses of tensors, each given as (tensor, name, dtype, shape), after
    checking that every one is contiguous, of that dtype and shape, and on
    device `dev`."""
    out = []
    try:
        for t, name, dtype, shape in specs:
            if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
                    or not t.is_contiguous()):
                raise AttributeError
            out.append(t.data_ptr())
        return out
    except AttributeError:
        pass
    for t, name, dtype, shape in specs:
        _refuse(t, name, dtype, shape, dev)
    raise AssertionError("unreachable")


def _refuse(t, name, dtype, shape, dev):
    """Raises what is wrong with a tensor, if anything."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(t, name, ndim):
    """The tensor's shape, of `ndim` dims."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    s = t.shape
    if len(s) != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {list(s)}")
    return s


def _device_of(t, name):
    """The tensor's device index, which has to be the current device's (the
    library launches there)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch._C._cuda_getDevice()
    if dev != cur:
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{cur}")
    return dev


def _ws_arg(ws, dev):
    """(pointer, bytes) of a workspace tensor or None."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev:
        raise ValueError(f"ws is on {ws.device}, expected cuda:{dev}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _ws_bytes(p, op, B, Tq, n_max, dev):
    """csa_workspace_size on device `dev`, answers kept with the parameter set."""
    sizes = p.__dict__.get("_ws")
    if sizes is None:
        sizes = {}
        object.__setattr__(p, "_ws", sizes)
    nb = sizes.get((op, B, Tq, n_max, dev))
    if nb is None:
        if len(sizes) >= 4096:  # a server with ever new sizes
            sizes.clear()
        nb = sizes[(op, B, Tq, n_max, dev)] = csa_workspace_size(p, op, B, Tq, n_max)
    return nb


def _head_rows(t, name, dtype, dim, dev):
    """Rows [rows][heads][dim] whose heads are dense, at any row stride."""
    rows, heads, d = _shape(t, name, 3)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if d != dim:
        raise ValueError(f"{name} must have heads of {dim}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    sr, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != dim):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), (sr if rows > 1 else heads * dim), heads, rows


def csa_norm_rope(p: Params, eps: float, q=None, q_weight=None, q_pos=None, q_out=None, k=None,
                  k_weight=None, k_pos=None, k_out=None, k_slots=None, stream=None):
    """RMS norm (fp32 weights [dim], None: ones) of every head of q
    [rows][heads][dim] and k [k_rows][k_heads][dim] and rotation of their
    trailing p.rope_dim dims by q_pos / k_pos (None: none) in one pass.  The
    rows of q and k may be strided (slices of one projection).  q_out as q,
    dense; row r of k goes to row k_slots[r] (-1: skipped; None: r) of k_out
    [n][k_heads][dim].  Either side may be None."""
    import torch
    first, name = (q, "q") if q is not None else (k, "k")
    dev = _device_of(first, name)
    dt = first.dtype
    code = _dtype_code(first)
    dim = _shape(first, name, 3)[2]
    f32, i32 = torch.float32, torch.int32
    qa = ka = (None, 0, 1, 0)
    specs = []
    if q is not None:
        qa = _head_rows(q, "q", dt, dim, dev)
        rows = qa[3]
        specs.append((q_out, "q_out", dt, (rows, qa[2], dim)))
        if q_weight is not None:
            specs.append((q_weight, "q_weight", f32, (dim,)))
        if q_pos is not None:
            specs.append((q_pos, "q_pos", i32, (rows,)))
    n_out = 0
    if k is not None:
        ka = _head_rows(k, "k", dt, dim, dev)
        rows = ka[3]
        n_out = rows if k_slots is None else _shape(k_out, "k_out", 3)[0]
        specs.append((k_out, "k_out", dt, (n_out, ka[2], dim)))
        if k_weight is not None:
            specs.append((k_weight, "k_weight", f32, (dim,)))
        if k_pos is not None:
            specs.append((k_pos, "k_pos", i32, (rows,)))
        if k_slots is not None:
            specs.append((k_slots, "k_slots", i32, (rows,)))
    it = iter(_args(dev, *specs))
    qo = qw = qp = ko = kw = kp = ks = None
    if q is not None:
        qo = next(it)
        qw = None if q_weight is None else next(it)
        qp = None if q_pos is None else next(it)
    if k is not None:
        ko = next(it)
        kw = None if k_weight is None else next(it)
        kp = None if k_pos is None else next(it)
        ks = None if k_slots is None else next(it)
    _check(_load().csa_norm_rope(p.ref(), code, dim, eps, *qa, qw, qp, qo, *ka, kw, kp, ks, n_out,
                                 ko, _stream(stream)))


def csa_quantize_mxfp4(rows, codes, scales, slots=None, values=None, stream=None):
    """Rows [..., d] (bf16 or fp32; a 2-D tensor may have strided rows) ->
    MXFP4 codes [n_out, ..., d / 2] and E8M0 scales [n_out, ..., d / 32]
    uint8.  With slots [n] int32, row i of the 2-D rows goes to row slots[i] of
    the 2-D (or paged [pages][page][...]) codes and scales (-1: skipped).
    values (rows' shape and dtype) receives the values the codes stand for."""
    import torch
    dev = _device_of(rows, "rows")
    code = _dtype_code(rows)
    have = rows.shape
    if not have:
        raise ValueError("rows must have at least 1 dim")
    d = have[-1]
    n = rows.numel() // d if d else 0
    if rows.is_contiguous():
        stride = d
    elif len(have) == 2 and rows.stride(1) == 1:
        stride = rows.stride(0)
    else:
        raise ValueError("rows must be contiguous, or 2-D with contiguous rows")
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch.Tensor")
    lead = tuple(codes.shape[:-1])
    specs = [(codes, "codes", torch.uint8, lead + (d // 2,)),
             (scales, "scales", torch.uint8, lead + (d // 32,))]
    if slots is not None:
        if len(have) != 2:
            raise ValueError("slots need 2-D rows")
        specs.append((slots, "slots", torch.int32, (n,)))
    elif lead != tuple(have[:-1]):
        raise ValueError("without slots, codes and scales must have the rows' leading dims")
    if values is not None:
        specs.append((values, "values", rows.dtype, have))
    it = _args(dev, *specs)
    _check(_load().csa_quantize_mxfp4(code, rows.data_ptr(), stride, n, d,
                                      it[2] if slots is not None else None,
                                      codes.numel() // (d // 2) if d >= 2 else 0, it[0], it[1],
                                      it[-1] if values is not None else None, _stream(stream)))


def _mx_index_args(p, q_codes, q_scales, w, k_codes, k_scales, page_table, q_pos, n_cmp, n_max,
                   out, out_name, out_dtype, out_last):
    """Checked arguments of the two indexer calls, in the C order from
    q_codes to n_max, then the output."""
    import torch
    dev = _device_of(q_codes, "q_codes")
    u8, i32 = torch.uint8, torch.int32
    H, D = p.idx_heads, p.idx_dim
    B, Tq = _shape(q_pos, "q_pos", 2)
    pages, page, _ = _shape(k_codes, "k_codes", 3)
    width, tab = 0, ()
    if page_table is None:
        if pages != B or (n_max is not None and page != n_max):
            raise ValueError(f"contiguous keys must be [B, n_max, ...], got {list(k_codes.shape)}")
        n_max = page
    else:
        width = _shape(page_table, "page_table", 2)[1]
        tab = ((page_table, "page_table", i32, (B, width)),)
        n_max = width * page if n_max is None else n_max
        if width == 0 and n_max > 0:
            # torch gives an empty table the address NULL, which the library
            # takes for contiguous keys
            raise ValueError(f"n_max={n_max} beyond an empty page table")
    a = _args(dev, (q_codes, "q_codes", u8, (B, Tq, H, D // 2)),
              (q_scales, "q_scales", u8, (B, Tq, H, D // 32)), (w, "w", torch.float32, (B, Tq, H)),
              (k_codes, "k_codes", u8, (pages, page, D // 2)),
              (k_scales, "k_scales", u8, (pages, page, D // 32)), (q_pos, "q_pos", i32, (B, Tq)),
              (n_cmp, "n_cmp", i32, (B,)),
              (out, out_name, out_dtype, (B, Tq, n_max if out_last is None else out_last)), *tab)
    return dev, (a[0], a[1], a[2], a[3], a[4], a[8] if tab else None, width, pages, page, a[5], a[6],
                 B, Tq, n_max, a[7])


def csa_index_scores_mxfp4(p: Params, q_codes, q_scales, w, k_codes, k_scales, page_table, q_pos,
                           n_cmp, scores, stream=None):
    """Indexer scores on MXFP4 queries [B][Tq][H_I][d_I/2] and keys
    [n_pages][page][d_I/2] found through page_table [B][width] (None: keys
    [B][n_max][d_I/2]) -> scores [B][Tq][n_max] of the visible entries."""
    import torch
    n_max = _shape(scores, "scores", 3)[2]
    _, a = _mx_index_args(p, q_codes, q_scales, w, k_codes, k_scales, page_table, q_pos, n_cmp,
                          n_max, scores, "scores", torch.float32, None)
    _check(_load().csa_index_scores_mxfp4(p.ref(), *a, _stream(stream)))


def csa_index_topk_mxfp4(p: Params, q_codes, q_scales, w, k_codes, k_scales, page_table, q_pos,
                         n_cmp, idx_out, ws, n_max=None, stream=None):
    """csa_index_scores_mxfp4 + top-k; n_max: entries scored at most (None:
    all the table holds); ws: csa_workspace_size(CSA_OP_INDEX_TOPK, B, Tq,
    n_max) bytes."""
    import torch
    dev, a = _mx_index_args(p, q_codes, q_scales, w, k_codes, k_scales, page_table, q_pos, n_cmp,
                            n_max, idx_out, "idx_out", torch.int32, p.topk)
    _check(_load().csa_index_topk_mxfp4(p.ref(), *a, *_ws_arg(ws, dev), _stream(stream)))


def _attn_paged(fn, p, q, q_pos, kv_pages, page_table, sel, sel_name, sel_shape, kv_raw, raw_pos0,
                n_raw, sink, out, ws, stream):
    import torch
    dev = _device_of(q, "q")
    code = _dtype_code(q)
    dt, i32 = q.dtype, torch.int32
    B, Tq = _shape(q_pos, "q_pos", 2)
    H, d = p.n_heads, p.d
    pages, page, _ = _shape(kv_pages, "kv_pages", 3)
    width = _shape(page_table, "page_table", 2)[1]
    raw_max = _shape(kv_raw, "kv_raw", 3)[1]
    a = _args(dev, (q, "q", dt, (B, Tq, H, d)), (q_pos, "q_pos", i32, (B, Tq)),
              (kv_pages, "kv_pages", dt, (pages, page, d)),
              (page_table, "page_table", i32, (B, width)),
              (sel, sel_name, i32, (B, Tq, p.topk) if sel_shape else (B,)),
              (kv_raw, "kv_raw", dt, (B, raw_max, d)), (raw_pos0, "raw_pos0", i32, (B,)),
              (n_raw, "n_raw", i32, (B,)), (sink, "sink", torch.float32, (H,)),
              (out, "out", dt, (B, Tq, H, d)))
    _check(fn(p.ref(), code, a[0], a[1], a[2], pages, page, a[3], width, a[4], a[5], a[6], a[7],
              raw_max, a[8], B, Tq, a[9], *_ws_arg(ws, dev), _stream(stream)))


def csa_sparse_attn_paged(p: Params, q, q_pos, kv_pages, page_table, idx, kv_raw, raw_pos0, n_raw,
                          sink, out, ws=None, stream=None):
    """csa_sparse_attn over entries in pages: kv_pages [n_pages][page][d],
    page_table [B][width] int32, idx [B][Tq][topk] entry numbers."""
    _attn_paged(_load().csa_sparse_attn_paged, p, q, q_pos, kv_pages, page_table, idx, "idx", True,
                kv_raw, raw_pos0, n_raw, sink, out, ws, stream)


def hca_attn_paged(p: Params, q, q_pos, kv_pages, page_table, n_cmp, kv_raw, raw_pos0, n_raw, sink,
                   out, ws=None, stream=None):
    """hca_attn over entries in pages, at any cache length: kv_pages
    [n_pages][page][d], page_table [B][width] int32, n_cmp [B]."""
    _attn_paged(_load().hca_attn_paged, p, q, q_pos, kv_pages, page_table, n_cmp, "n_cmp", False,
                kv_raw, raw_pos0, n_raw, sink, out, ws, stream)
