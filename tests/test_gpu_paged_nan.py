"""NaN in the generic paged attention (fp32, or d other than 512): one NaN
element of a row makes every dim of every head that attends to the row NaN,
one of a query its head, a NaN sink its head, as a softmax over them does;
other tokens and heads keep their values."""
import numpy as np
import pytest
import torch

from gpu_util import assert_close, host64
from sparse_compressed_attention_csa_b200 import csa_poll_device_error
from test_gpu_paged import _case, _hca, _sparse

pytestmark = pytest.mark.gpu

SHAPES = [
    # dtype, H, d, rope, lens, Tq, page, width, stride, window, topk
    ("f32", 8, 128, 64, [3000, 2900, 2800], 1, 64, 1, 1, 0, 0),      # rows in several splits
    ("f32", 3, 64, 32, [40, 30, 20], 1, 8, 1, 1, 0, 0),              # one split
    ("bf16", 5, 64, 32, [900, 800, 700], 2, 16, 1, 1, 16, 0),
    ("bf16", 8, 128, 64, [50, 40, 30], 1, 8, 1, 1, 4, 0),
    ("f32", 6, 512, 64, [700, 600, 500], 1, 64, 1, 1, 0, 0),
    ("f32", 8, 128, 64, [3000, 2900, 2800], 1, 64, 8, 4, 16, 100),   # selected entries
]


@pytest.mark.parametrize("row", [0, 3, 8])                           # a warp's first row, and a second one
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: str(s)[:48])
def test_nan_spreads_over_its_heads_and_no_further(shape, row):
    dtype, H = shape[0], shape[1]
    topk = shape[10]
    p, t, want = _case(*shape[:10], seed=300 + SHAPES.index(shape), topk=topk)
    call = _sparse if topk else _hca
    page = t["kv"].shape[1]
    j = int(t["idx"][0, 0, row]) if topk else row
    t["kv"][int(t["table"][0, j // page]), j % page, 5] = float("nan")  # one element of one row
    t["q"][1, 0, 2, 3] = float("nan")                                   # of one query head
    t["sink"][1] = float("nan")
    out = host64(call(p, t))
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert np.all(np.isnan(out[0])), "a NaN row"
    assert np.all(np.isnan(out[1, 0, 2])), "a NaN query"
    assert np.all(np.isnan(out[:, :, 1])), "a NaN sink"
    keep = np.ones(H, dtype=bool)
    keep[[1, 2]] = False
    assert_close(out[1:][:, :, keep], want[1:][:, :, keep], dtype, "beside NaN")
