"""User-level entry points: allocate outputs and workspace with torch, then
call the C ABI.  Every step runs in the CUDA library.

    decode: csa_decode(p, q, q_idx, w, k_idx, kv_cmp, kv_raw, ...) -> (idx, out)
    prefill: csa_prefill(p, x, gate, q_idx, w, k_idx, q, sink) -> (kv_cmp, kv_raw, idx, out)
    HCA decode: hca_decode(p, q, kv_cmp, kv_raw, ...) -> out
    HCA prefill: hca_prefill(p, x, gate, q, sink) -> (kv_cmp, kv_raw, out)
    CSA2 reuse layer: reuse_attn(p, q, ..., kv_cmp, idx, ...) -> out
    decode-time append: append_tokens(p, x, gate, x_pos0, t_old, t_new, ...)
    FP8 caches: quantize_fp8(rows) -> (codes, scales); csa_decode_fp8(...)
    norm + RoPE of heads: norm_rope(p, q, ...) -> (q_out, k_out)
    paged caches: csa_decode_paged(...) with the indexer in 4 bits,
    sparse_attn_paged(...), hca_decode_paged(...); quantize_mxfp4(rows) ->
    (codes, scales)
"""
from __future__ import annotations

import torch

from . import _lib as L


class _On:
    """What a call allocates is allocated for the stream it runs on (torch's
    allocator hands a freed block to the stream it came from)."""

    def __init__(self, stream):
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


class Workspace:
    """A reusable device scratch buffer that grows on demand.  Calls that share
    one run one after another (on one stream, or ordered by events; replays of
    graphs that were captured with it included).  A buffer that a captured graph
    uses stays until the workspace is dropped, and an outgrown one is not handed
    out again before the calls on it are over, on whichever stream they run."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self._in_graph = False  # a capture has used `buf`
        self._kept = []         # outgrown buffers of captured graphs

    def get(self, nbytes: int):
        """At least `nbytes`, for calls on the current stream."""
        if nbytes == 0:
            return None
        if self.buf is None or self.buf.numel() < nbytes:
            if self._in_graph:
                self._kept.append(self.buf)
                self._in_graph = False
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device or "cuda")
            self._streams = {self._current()}
        if self.buf.is_cuda:
            if torch.cuda.is_current_stream_capturing():
                self._in_graph = True
            elif self._current() not in self._streams:  # once: it counts until the buffer is freed
                self.buf.record_stream(torch.cuda.current_stream(self.buf.device))
                self._streams.add(self._current())
        return self.buf

    def on(self, nbytes: int, stream):
        """get() for a call on `stream` (None: the current one)."""
        if stream is None:
            return self.get(nbytes)
        with _On(stream):
            return self.get(nbytes)

    def _current(self):
        """The current stream's handle."""
        return torch._C._cuda_getCurrentRawStream(self.buf.device.index) if self.buf.is_cuda else 0


def csa_decode(p: L.Params, q, q_pos, q_idx, w, k_idx, n_cmp, kv_cmp, kv_raw, raw_pos0, n_raw,
               sink, ws: Workspace | None = None, idx=None, out=None, stream=None):
    """Indexer + top-k + sparse attention for Tq query tokens per sequence."""
    ws = ws or Workspace(q.device)
    B, Tq = q_pos.shape
    n_max = k_idx.shape[1]
    if idx is None:
        idx = torch.empty((B, Tq, p.topk), dtype=torch.int32, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    nb = L.csa_workspace_size(p, L.CSA_OP_INDEX_TOPK, B, Tq, n_max)
    L.csa_index_topk(p, q_idx, w, k_idx, q_pos, n_cmp, idx, ws.on(nb, stream), stream)
    nb = L.csa_workspace_size(p, L.CSA_OP_SPARSE_ATTN, B, Tq, kv_cmp.shape[1])
    L.csa_sparse_attn(p, q, q_pos, kv_cmp, idx, kv_raw, raw_pos0, n_raw, sink, out, ws.on(nb, stream),
                      stream)
    return idx, out


def csa_prefill(p: L.Params, x, gate, q_idx, w, k_idx, q, sink, ws: Workspace | None = None,
                stream=None):
    """The whole layer on B sequences of T tokens, every token a causal query."""
    ws = ws or Workspace(x.device)
    B, T, d = x.shape
    N = 0 if T < p.width else (T - p.width) // p.stride + 1
    dev = x.device
    kv_cmp = torch.empty((B, N, d), dtype=x.dtype, device=dev)
    kv_raw = torch.empty((B, T, d), dtype=x.dtype, device=dev)
    L.csa_compress(p, x, gate, kv_cmp, kv_raw, stream)
    q_pos = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1).contiguous()
    n_cmp = torch.full((B,), N, dtype=torch.int32, device=dev)
    raw_pos0 = torch.zeros((B,), dtype=torch.int32, device=dev)
    n_raw = torch.full((B,), T, dtype=torch.int32, device=dev)
    idx, out = csa_decode(p, q, q_pos, q_idx, w, k_idx, n_cmp, kv_cmp, kv_raw, raw_pos0, n_raw,
                          sink, ws, stream=stream)
    return kv_cmp, kv_raw, idx, out


def hca_decode(p: L.Params, q, q_pos, kv_cmp, n_cmp, kv_raw, raw_pos0, n_raw, sink,
               ws: Workspace | None = None, out=None, stream=None):
    ws = ws or Workspace(q.device)
    B, Tq = q_pos.shape
    if out is None:
        out = torch.empty_like(q)
    nb = L.csa_workspace_size(p, L.CSA_OP_HCA_ATTN, B, Tq, kv_cmp.shape[1])
    L.hca_attn(p, q, q_pos, kv_cmp, n_cmp, kv_raw, raw_pos0, n_raw, sink, out, ws.on(nb, stream), stream)
    return out


def reuse_attn(p: L.Params, q, q_pos, kv_cmp, idx, kv_raw, raw_pos0, n_raw, sink,
               ws: Workspace | None = None, out=None, stream=None):
    """Reuse layers of CSA2 ("CSA2 encoder layers (2x compression, Full +
    Reuse)": the rest reuse that KV and its top-512 selection): each layer's
    queries q [R][B][Tq][H][d] and sink [R][H] over the entries and indices a
    Full layer produced, all R layers in one call (a single layer:
    q [B][Tq][H][d], sink [H])."""
    ws = ws or Workspace(q.device)
    single = q.dim() == 4
    if single:
        q, sink = q.unsqueeze(0), sink.unsqueeze(0)
    if out is None:
        out = torch.empty_like(q)
    elif single:
        out = out.unsqueeze(0)
    R = q.shape[0]
    B, Tq = q_pos.shape
    nb = L.csa_workspace_size(p, L.CSA_OP_SPARSE_ATTN, R * B, Tq, kv_cmp.shape[1])
    L.csa_reuse_attn(p, q, q_pos, kv_cmp, idx, kv_raw, raw_pos0, n_raw, sink, out, ws.on(nb, stream),
                     stream)
    return out[0] if single else out


def hca_prefill(p: L.Params, x, gate, q, sink, ws: Workspace | None = None, out=None,
                stream=None):
    """HCA on B sequences of T tokens, every token a causal query ("Heavily
    Compressed Attention" row: every 128 tokens pooled into one entry, dense
    attention over all of them plus a 128-token window); p.width and
    p.stride give the pooling."""
    ws = ws or Workspace(x.device)
    B, T, d = x.shape
    N = 0 if T < p.width else (T - p.width) // p.stride + 1
    dev = x.device
    kv_cmp = torch.empty((B, N, d), dtype=x.dtype, device=dev)
    kv_raw = torch.empty((B, T, d), dtype=x.dtype, device=dev)
    L.csa_compress(p, x, gate, kv_cmp, kv_raw, stream)
    q_pos = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1).contiguous()
    n_cmp = torch.full((B,), N, dtype=torch.int32, device=dev)
    raw_pos0 = torch.zeros((B,), dtype=torch.int32, device=dev)
    out = hca_decode(p, q, q_pos, kv_cmp, n_cmp, kv_raw, raw_pos0, n_cmp.new_full((B,), T), sink,
                     ws, out, stream)
    return kv_cmp, kv_raw, out


def append_tokens(p: L.Params, x, gate, x_pos0, t_old, t_new, max_new: int, kv_cmp,
                  kv_raw=None, raw_pos0=None, stream=None):
    """Decode-time compression: write the entries and rotated raw rows that
    tokens t_old[b] .. t_new[b] - 1 complete into the caches (entry j at
    row j of kv_cmp, token t at row t - raw_pos0[b] of kv_raw); x, gate hold
    token x_pos0[b] + i at row i."""
    L.csa_compress_append(p, x, gate, x_pos0, t_old, t_new, max_new, kv_cmp, kv_raw, raw_pos0,
                          stream)


def quantize_fp8(rows, stream=None):
    """Cache rows [..., d] (rotated) -> (E4M3 codes uint8 [..., d], fp32
    scales [...]), one scale per row: the KV cache quantized after RoPE."""
    codes = torch.empty(rows.shape, dtype=torch.uint8, device=rows.device)
    scales = torch.empty(rows.shape[:-1], dtype=torch.float32, device=rows.device)
    L.csa_quantize_fp8(rows, codes, scales, stream)
    return codes, scales


def csa_decode_fp8(p: L.Params, q, q_pos, q_idx, w, k_idx, n_cmp, kv_cmp, cmp_scale, kv_raw,
                   raw_scale, raw_pos0, n_raw, sink, ws: Workspace | None = None, idx=None,
                   out=None, stream=None):
    """csa_decode over FP8 caches (codes and row scales from quantize_fp8)."""
    ws = ws or Workspace(q.device)
    B, Tq = q_pos.shape
    n_max = k_idx.shape[1]
    if idx is None:
        idx = torch.empty((B, Tq, p.topk), dtype=torch.int32, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    nb = L.csa_workspace_size(p, L.CSA_OP_INDEX_TOPK, B, Tq, n_max)
    L.csa_index_topk(p, q_idx, w, k_idx, q_pos, n_cmp, idx, ws.on(nb, stream), stream)
    nb = L.csa_workspace_size(p, L.CSA_OP_SPARSE_ATTN, B, Tq, kv_cmp.shape[1])
    L.csa_sparse_attn_fp8(p, q, q_pos, kv_cmp, cmp_scale, idx, kv_raw, raw_scale, raw_pos0, n_raw,
                          sink, out, ws.on(nb, stream), stream)
    return idx, out


def norm_rope(p: L.Params, q, q_weight=None, q_pos=None, k=None, k_weight=None, k_pos=None,
              k_out=None, k_slots=None, eps: float = 1e-6, stream=None):
    """RMS norm of every head of q [rows][heads][dim] (and k) and rotation of
    the trailing p.rope_dim dims by q_pos (k_pos), in one pass: the indexer's
    queries and keys, token rows, or pooled entries on their way to a cache.
    Returns (q_out, k_out); with k_out and k_slots given, row r of k goes to
    row k_slots[r] of k_out."""
    with _On(stream):
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    L.csa_norm_rope(p, eps, q, q_weight, q_pos, q_out, k, k_weight, k_pos, k_out, k_slots, stream)
    return q_out, k_out


def quantize_mxfp4(rows, stream=None):
    """Rows [..., d] -> (E2M1 codes uint8 [..., d / 2], E8M0 scales uint8
    [..., d / 32]), one scale per 32 values."""
    with _On(stream):
        codes = torch.empty(rows.shape[:-1] + (rows.shape[-1] // 2,), dtype=torch.uint8,
                            device=rows.device)
        scales = torch.empty(rows.shape[:-1] + (rows.shape[-1] // 32,), dtype=torch.uint8,
                             device=rows.device)
    L.csa_quantize_mxfp4(rows, codes, scales, stream=stream)
    return codes, scales


def sparse_attn_paged(p: L.Params, q, q_pos, kv_pages, page_table, idx, kv_raw, raw_pos0, n_raw,
                      sink, ws: Workspace | None = None, out=None, stream=None):
    """Attention over the selected entries idx [B][Tq][topk] of a paged cache
    kv_pages [n_pages][page][d] and the window's raw rows."""
    ws = ws or Workspace(q.device)
    B, Tq = q_pos.shape
    nb = L._ws_bytes(p, L.CSA_OP_SPARSE_ATTN_PAGED, B, Tq, page_table.shape[1] * kv_pages.shape[1],
                     L._device_of(q, "q"))
    with _On(stream):
        if out is None:
            out = torch.empty_like(q)
        buf = ws.get(nb)
    L.csa_sparse_attn_paged(p, q, q_pos, kv_pages, page_table, idx, kv_raw, raw_pos0, n_raw, sink, out, buf,
                           stream)
    return out


def hca_decode_paged(p: L.Params, q, q_pos, kv_pages, page_table, n_cmp, kv_raw, raw_pos0, n_raw,
                     sink, ws: Workspace | None = None, out=None, stream=None):
    """HCA decode over a paged entry cache of any length; with
    Params(width=1, stride=1) every token is its own entry."""
    ws = ws or Workspace(q.device)
    B, Tq = q_pos.shape
    nb = L._ws_bytes(p, L.CSA_OP_HCA_ATTN_PAGED, B, Tq, page_table.shape[1] * kv_pages.shape[1],
                     L._device_of(q, "q"))
    with _On(stream):
        if out is None:
            out = torch.empty_like(q)
        buf = ws.get(nb)
    L.hca_attn_paged(p, q, q_pos, kv_pages, page_table, n_cmp, kv_raw, raw_pos0, n_raw, sink, out, buf,
                    stream)
    return out


def csa_decode_paged(p: L.Params, q, q_pos, q_idx, w, k_codes, k_scales, n_cmp, kv_pages,
                     page_table, kv_raw, raw_pos0, n_raw, sink, ws: Workspace | None = None,
                     idx=None, out=None, n_max: int | None = None, stream=None):
    """CSA decode over paged caches with the indexer in 4 bits: q_idx
    [B][Tq][H_I][d_I] (after its norm and rotation) is quantized to MXFP4,
    scored against the paged MXFP4 keys, and the top-k entries of the paged
    entry cache attended to.  The key and entry pools share page_table; n_max
    bounds the entries scored (None: all the table holds)."""
    if k_codes.shape[1] != kv_pages.shape[1]:
        raise ValueError(f"the pools share a page table: pages of {k_codes.shape[1]} keys and "
                         f"{kv_pages.shape[1]} entries")
    ws = ws or Workspace(q.device)
    B, Tq = q_pos.shape
    q_codes, q_scales = quantize_mxfp4(q_idx, stream)
    if n_max is None:
        n_max = page_table.shape[1] * k_codes.shape[1]
    nb = L._ws_bytes(p, L.CSA_OP_INDEX_TOPK, B, Tq, n_max, L._device_of(q, "q"))
    with _On(stream):
        if idx is None:
            idx = torch.empty((B, Tq, p.topk), dtype=torch.int32, device=q.device)
        buf = ws.get(nb)
    L.csa_index_topk_mxfp4(p, q_codes, q_scales, w, k_codes, k_scales, page_table, q_pos, n_cmp,
                           idx, buf, n_max, stream)
    return idx, sparse_attn_paged(p, q, q_pos, kv_pages, page_table, idx, kv_raw, raw_pos0, n_raw,
                                  sink, ws, out, stream)
