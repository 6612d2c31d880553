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
