"""More shapes of the paged attention against the oracle: rotated dims that
end inside a warp of the rotation table, on every way a token is split."""
import pytest
import torch

from gpu_util import assert_close, host64
from sparse_compressed_attention_csa_b200 import csa_poll_device_error
from test_gpu_paged import _case, _hca, _sparse

pytestmark = pytest.mark.gpu


def _check(p, t, want, selected, what):
    call = _sparse if selected else _hca
    out = call(p, t)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert_close(host64(out), want, "bf16", what)
    assert torch.equal(out, call(p, t)), f"{what}: not the same twice"


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("rope", [32, 96])
@pytest.mark.parametrize("B", [3, 18, 30, 60, 90])
def test_rotated_dims_that_end_inside_a_warp(B, rope, selected):
    # empty tokens and pairs without tiles among them
    lens = [1, 0, 65] + [37 * i % 250 for i in range(B - 3)]
    p, t, want = _case("bf16", 128, 512, rope, lens, 1, 16, 1, 1, 64, 400 + B + rope, topk=100 if selected else 0)
    _check(p, t, want, selected, f"{B} tokens, {rope} rotated dims")


@pytest.mark.parametrize("c", [
    # H, lens, Tq, page, width, stride, window, topk: chunks of a prompt, many tokens a CTA pair
    (128, [900, 300], 150, 64, 4, 4, 128, 0),
    (128, [700], 300, 16, 128, 128, 128, 0),            # few entries, mostly the window
    (128, [420, 260, 100], 100, 32, 1, 1, 0, 0),        # entries alone; the longest token 7 tiles
    (16, [900, 500], 200, 64, 8, 4, 128, 0),
    (200, [500], 90, 64, 4, 4, 20, 0),                  # two groups of heads
    (128, [1500, 700], 128, 64, 8, 4, 128, 256),
    (128, [400], 400, 8, 8, 4, 128, 64),                # tokens with no entry yet
    (16, [900, 500], 160, 64, 8, 4, 16, 100),
], ids=str)
def test_chunks_of_a_prompt(c):
    H, lens, Tq, page, width, stride, window, topk = c
    p, t, want = _case("bf16", H, 512, 64, lens, Tq, page, width, stride, window, 500 + H + Tq, topk=topk,
                       keep_raw=window + Tq)
    _check(p, t, want, bool(topk), str(c))


@pytest.mark.parametrize("selected", [False, True])
def test_nan_on_several_pairs_of_a_long_token(selected):
    # parts joined by a second launch: a NaN row, a NaN query, a NaN sink
    import numpy as np
    p, t, want = _case("bf16", 128, 512, 64, [9000, 4000, 5000], 1, 64, 1, 1, 128, 540, topk=2048 if selected else 0)
    j = int(t["idx"][0, 0, 1500]) if selected else 7000
    t["kv"][int(t["table"][0, j // 64]), j % 64, 5] = float("nan")
    t["q"][1, 0, 7, 3] = float("nan")
    t["sink"][9] = float("nan")
    out = host64((_sparse if selected else _hca)(p, t))
    csa_poll_device_error()
    assert np.all(np.isnan(out[0])) and np.all(np.isnan(out[1, 0, 7])) and np.all(np.isnan(out[:, 0, 9]))
    keep = np.ones(128, dtype=bool)
    keep[[7, 9]] = False
    assert_close(out[1:][:, :, keep], want[1:][:, :, keep], "bf16", "beside NaN")


@pytest.mark.parametrize("selected", [False, True])
def test_pages_longer_than_a_sequence(selected):
    p, t, want = _case("bf16", 128, 512, 64, [3000, 9000], 1, 16384, 1, 1, 128, 541, topk=512 if selected else 0)
    _check(p, t, want, selected, "pages of 16,384 rows")
