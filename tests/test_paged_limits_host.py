"""The most entries that a call may be sized for (CPU): sizes whose rounding
up to a tile would pass 32 bits are refused before anything is launched."""
import ctypes

import pytest

import sparse_compressed_attention_csa_b200 as csa
from sparse_compressed_attention_csa_b200 import _lib as L
from sparse_compressed_attention_csa_b200 import build as B

OK = ctypes.c_void_p(1 << 20)      # an aligned address that no accepted call reaches
MOST = 2 ** 31 - 2 ** 15


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def _pp(**kw):
    return ctypes.byref(csa.Params(**kw).c())


@pytest.mark.parametrize("op", [csa.CSA_OP_INDEX_TOPK, csa.CSA_OP_SPARSE_ATTN_PAGED, csa.CSA_OP_HCA_ATTN_PAGED])
def test_workspace_sizes_up_to_the_limit(lib, op):
    p = csa.Params(n_heads=3)
    assert csa.csa_workspace_size(p, op, 1, 1, MOST) > 0
    for n in (MOST + 1, 2 ** 31 - 1):
        with pytest.raises(csa.CsaError) as ei:
            csa.csa_workspace_size(p, op, 1, 1, n)
        assert ei.value.status == 3


@pytest.mark.parametrize("n_max", [MOST + 1, 2 ** 31 - 64, 2 ** 31 - 1])
def test_indexer_and_selection(lib, n_max):
    width, none = (1 << 25) - 1, None       # pages of 64: all the table may hold
    for table, w in ((OK, width), (none, 0)):
        if table is OK and n_max > width * 64:
            continue
        args = (OK, OK, OK, OK, OK, table, w, 9, 64, OK, OK, 1, 1, n_max, OK)
        assert lib.csa_index_scores_mxfp4(_pp(), *args, None) == 3, lib.csa_last_error_detail()
        assert lib.csa_index_topk_mxfp4(_pp(), *args, OK, 1 << 40, None) == 3
    assert lib.csa_topk_select(_pp(), OK, OK, OK, 1, 1, n_max, OK, OK, 1 << 40, None) == 3


@pytest.mark.parametrize("call", ["csa_sparse_attn_paged", "hca_attn_paged"])
@pytest.mark.parametrize("width,page", [((1 << 25) - 1, 64), ((1 << 28) - 1, 8), ((1 << 28) - (1 << 12) + 1, 8)])
def test_page_tables(lib, call, width, page):
    assert width * page > MOST
    for n_heads, dtype in ((128, 1), (3, 0)):
        st = getattr(lib, call)(_pp(n_heads=n_heads), dtype, OK, OK, OK, 9, page, OK, width, OK, OK, OK, OK, 4, OK,
                                1, 1, OK, OK, 1 << 40, None)
        assert st == 3, lib.csa_last_error_detail()
        assert b"entries" in lib.csa_last_error_detail()
