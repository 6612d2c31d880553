"""Calls of the paged tensor-core kernels under a wait limit of 1 ns: a wait
that runs out records CSA_ERR_DEVICE_TIMEOUT, every warp waits for the copies
and products that it issued itself and leaves, and the next call is right.  No
wait is endless: each has the limit or, on the way out, 100 ms."""
import pytest
import torch

from sparse_compressed_attention_csa_b200 import (CsaError, Params, csa_index_scores_mxfp4,
                                                  csa_poll_device_error, csa_set_wait_limit_ns)
from test_gpu_mxfp4 import _check_scores, _score_case

pytestmark = pytest.mark.gpu
CSA_ERR_DEVICE_TIMEOUT = 7


def _under_a_tiny_limit(call):
    torch.cuda.synchronize()
    csa_poll_device_error()  # starts clean
    csa_set_wait_limit_ns(1)
    try:
        call()
        try:
            csa_poll_device_error()
        except CsaError as err:
            assert err.status == CSA_ERR_DEVICE_TIMEOUT
    finally:
        csa_set_wait_limit_ns(0)
    csa_poll_device_error()


@pytest.mark.parametrize("lens,Tq", [
    ([160000, 150000, 90000], 1),   # one token: several tiles a CTA, both fetching warps
    ([120000, 50000], 2),           # 16-token units, their tiles in ranges
    ([2600], 2600),                 # more units than CTAs, whole units in turn
], ids=["one token", "few tokens", "prompt"])
def test_indexer(lens, Tq):
    p = Params()
    t, want, bound, vis = _score_case(lens, Tq, 64, 128, 64, 700 + Tq)
    n_max = max(len(x[0]) for x in want)
    scores = torch.empty(len(lens), Tq, n_max, device="cuda")
    _under_a_tiny_limit(lambda: csa_index_scores_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                                             t["page_table"], t["q_pos"], t["n_cmp"], scores))
    _check_scores(p, t, want, bound, vis, n_max)
