"""The paged calls at the last position that 32 bits hold, 2^31 - 1, where
every token is its own entry."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_close, host64
from sparse_compressed_attention_csa_b200 import (CSA_OP_INDEX_TOPK, Params, csa_index_topk_mxfp4,
                                                  csa_poll_device_error, csa_workspace_size)
from test_gpu_mxfp4 import _check_scores, _score_case
from test_gpu_paged import _case, _hca, _sparse

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("dtype,H,d", [("bf16", 128, 512), ("f32", 3, 64), ("bf16", 5, 128)])
def test_attention_at_the_last_position(dtype, H, d, selected):
    window, n_raw, topk = 16, 12, 40 if selected else 0
    p, t, _ = _case(dtype, H, d, 32, [300, 200], 1, 16, 1, 1, window, 900 + H, topk=topk, keep_raw=n_raw)
    t["q_pos"].fill_(LAST)
    t["pos0"].fill_(LAST - n_raw + 1)
    out = host64((_sparse if selected else _hca)(p, t))
    csa_poll_device_error()
    f = lambda a: a.double().cpu().numpy()  # noqa: E731
    for b, n in enumerate([300, 200]):
        rows = oracle.paged_rows(f(t["kv"]), t["table"][b].cpu().numpy(), n)
        args = (f(t["raw"][b]), LAST - n_raw + 1, n_raw, t["sink"].cpu().numpy(), 1 / np.sqrt(d), window)
        if selected:
            want = oracle.sparse_attn(f(t["q"][b]), [LAST], rows, t["idx"][b].cpu().numpy(), *args, 32, 1e4)
        else:
            want = oracle.hca_attn(f(t["q"][b]), [LAST], rows, n, *args, 1, 1, 32, 1e4)
        assert_close(out[b], want, dtype, "last position")


@pytest.mark.parametrize("H,D", [(64, 128), (4, 32)])
def test_indexer_at_the_last_position(H, D):
    p = Params(width=1, stride=1, idx_heads=H, idx_dim=D, topk=50)
    t, want, bound, _ = _score_case([900, 33], 1, H, D, 64, 950 + H, width=1, stride=1)
    t["q_pos"].fill_(LAST)
    n_max = 900
    scores = _check_scores(p, t, want, bound, [[900], [33]], n_max).cpu().numpy()
    idx = torch.empty(2, 1, 50, dtype=torch.int32, device="cuda")
    ws = torch.empty(csa_workspace_size(p, CSA_OP_INDEX_TOPK, 2, 1, n_max), dtype=torch.uint8, device="cuda")
    csa_index_topk_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"], t["page_table"],
                         t["q_pos"], t["n_cmp"], idx, ws, n_max)
    csa_poll_device_error()
    got = idx.cpu().numpy()[:, 0]
    top = np.argsort(-scores[0, 0], kind="stable")[:50]
    assert sorted(top.tolist()) == got[0].tolist()
    assert got[1].tolist() == list(range(33)) + [-1] * 17
