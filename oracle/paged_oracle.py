"""fp64 oracle of the paged, 4-bit serving path: norms of query and key heads
with the partial RoPE, MXFP4 rows (OCP Microscaling Formats v1.0), and rows
looked up through a page table.  The attention and the indexer over them are
the layer's own (csa_oracle)."""
from __future__ import annotations

import numpy as np

from .csa_oracle import rope


def norm_rope(x, weight, pos, rope_dim: int, theta, eps: float) -> np.ndarray:
    """x [rows, heads, dim]: every head row over its root mean square, times
    weight [dim] (None: ones), then rotated at pos [rows] (None: not)."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if pos is None:
        return y
    return rope(y, np.asarray(pos, dtype=np.int64)[:, None], rope_dim, theta)


def e2m1_values() -> np.ndarray:
    """The value of each of the 16 E2M1 codes: sign, two exponent bits with
    bias 1, one mantissa bit."""
    out = np.empty(16, dtype=np.float64)
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = 0.5 * m if e == 0 else 2.0 ** (e - 1) * (1.0 + 0.5 * m)
        out[c] = -v if c & 8 else v
    return out


def e2m1_encode(y) -> np.ndarray:
    """Nearest E2M1 code of each finite value, ties to the even code, past 6
    to 6; the sign of zero is kept."""
    y = np.asarray(y, dtype=np.float64)
    vals = e2m1_values()[:8]
    a = np.minimum(np.abs(y), 6.0)
    gap = np.abs(a[..., None] - vals)
    best = gap.min(axis=-1, keepdims=True)
    tied = gap == best                      # one code, or two neighbours
    first = tied.argmax(axis=-1)
    second = 7 - tied[..., ::-1].argmax(axis=-1)
    code = np.where(first % 2 == 0, first, second)
    return (code + 8 * np.signbit(y)).astype(np.uint8)


def mxfp4_encode(rows):
    """Rows [..., d] -> (codes [..., d / 2], the even dim in the low half;
    scale bytes [..., d / 32])."""
    r = np.asarray(rows, dtype=np.float64)
    blocks = r.reshape(r.shape[:-1] + (r.shape[-1] // 32, 32))
    bad = ~np.isfinite(blocks).all(axis=-1)
    b = np.where(bad[..., None], 0.0, blocks)
    amax = np.abs(b).max(axis=-1)
    exp = np.frexp(np.where(amax > 0, amax, 4.0))[1] - 1 - 2   # floor(log2 amax) - 2
    exp = np.maximum(exp, -127)
    code = e2m1_encode(b / np.exp2(exp.astype(np.float64))[..., None])
    code = np.where(bad[..., None], 0, code).reshape(r.shape).astype(np.uint8)
    scale = np.where(bad, 255, exp + 127).astype(np.uint8)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), scale


def mxfp4_decode(codes, scales) -> np.ndarray:
    """The values that codes [..., d / 2] stand for under scales [..., d / 32]."""
    codes = np.asarray(codes)
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    s = np.asarray(scales).astype(np.int64)
    f = np.where(s == 255, np.nan, np.exp2(np.minimum(s, 254).astype(np.float64) - 127))
    return e2m1_values()[c] * np.repeat(f, 32, axis=-1)


def paged_rows(pool, table_row, n: int) -> np.ndarray:
    """The first n entries of one sequence: pool [n_pages, page, ...]."""
    page = np.shape(pool)[1]
    j = np.arange(n)
    return np.asarray(pool)[np.asarray(table_row)[j // page], j % page]
