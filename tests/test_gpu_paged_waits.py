"""Bounded waits that run out in the paged tensor-core kernels: with a limit
of 1 ns the first wait that is not over at once gives up, the call records
CSA_ERR_DEVICE_TIMEOUT, every warp waits for the copies and products that it
issued itself and leaves, and the next call is right.  No wait is endless:
each has the limit or, on the way out, 100 ms."""
import pytest
import torch

from gpu_util import assert_close, host64
from sparse_compressed_attention_csa_b200 import (CsaError, Params, csa_index_scores_mxfp4,
                                                  csa_last_device_error_site, csa_poll_device_error,
                                                  csa_set_wait_limit_ns)
from test_gpu_mxfp4 import _check_scores, _score_case
from test_gpu_paged import _case, _hca, _sparse

pytestmark = pytest.mark.gpu
CSA_ERR_DEVICE_TIMEOUT = 7


def _runs_out(call):
    torch.cuda.synchronize()
    csa_poll_device_error()  # starts clean
    csa_set_wait_limit_ns(1)
    try:
        call()
        with pytest.raises(CsaError) as err:
            csa_poll_device_error()
        assert err.value.status == CSA_ERR_DEVICE_TIMEOUT
        assert csa_last_device_error_site() > 0
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
    _runs_out(lambda: csa_index_scores_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                                             t["page_table"], t["q_pos"], t["n_cmp"], scores))
    _check_scores(p, t, want, bound, vis, n_max)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("B,n", [(3, 240), (18, 240), (30, 240), (60, 240), (90, 240), (2, 9000)],
                         ids=["4 pairs a token", "3 pairs", "2 pairs", "1 pair", "several tokens a pair",
                              "ranges of a long token"])
def test_attention(B, n, selected):
    # the last two are joined by a second launch, the first three in a cluster
    lens = [n - 7 * (i % 5) for i in range(B)]
    topk = 0 if not selected else (100 if n < 1000 else 1024)
    p, t, want = _case("bf16", 128, 512, 64, lens, 1, 64, 1, 1, 128, 720 + B, topk=topk)
    call = _sparse if selected else _hca
    _runs_out(lambda: call(p, t))
    out = call(p, t)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert_close(host64(out), want, "bf16", "after a failed launch")
