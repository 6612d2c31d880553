"""Refusals of the paged, 4-bit calls (CPU): bad sizes, NULL and misaligned
pointers, short workspaces, host tensors, shapes that disagree.  Nothing
reaches a device."""
import ctypes

import pytest
import torch

import sparse_compressed_attention_csa_b200 as csa
from sparse_compressed_attention_csa_b200 import _lib as L
from sparse_compressed_attention_csa_b200 import build as B
from sparse_compressed_attention_csa_b200 import layer

P = ctypes.c_void_p
OK = P(1 << 20)      # an aligned address that no accepted call reaches
BAD = P((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def _pp(**kw):
    return ctypes.byref(csa.Params(**kw).c())


def _norm(lib, dtype=1, dim=128, eps=1e-6, q=OK, qs=128 * 4, qh=4, qr=3, qw=OK, qp=OK, qo=OK, k=OK,
          ks=128, kh=1, kr=3, kw=OK, kp=OK, slots=None, n_out=3, ko=OK, **params):
    return lib.csa_norm_rope(_pp(**params), dtype, dim, eps, q, qs, qh, qr, qw, qp, qo, k, ks, kh,
                             kr, kw, kp, slots, n_out, ko, None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dtype=5)), (3, dict(dim=4)), (3, dict(dim=100)), (3, dict(dim=2048)),
    (3, dict(dim=32)),                                   # rope_dim 64 > dim
    (1, dict(eps=0.0)), (1, dict(eps=float("nan"))), (1, dict(eps=float("inf"))),
    (1, dict(q=None)), (2, dict(q=BAD)), (1, dict(qo=None)), (2, dict(qw=BAD)), (2, dict(qp=BAD)),
    (1, dict(qs=511)), (2, dict(qs=516)), (3, dict(qr=-1)), (3, dict(qh=0)),
    (1, dict(k=None)), (1, dict(n_out=2)), (2, dict(slots=BAD)), (1, dict(ko=None)),
])
def test_norm_rope_refusals(lib, want, kw):
    assert _norm(lib, **kw) == want, lib.csa_last_error_detail()


def test_norm_rope_with_no_rows_does_nothing(lib):
    assert _norm(lib, qr=0, q=None, qo=None, kr=0, k=None, ko=None) == 0


@pytest.mark.parametrize("want,kw", [
    (1, dict(dtype=2)), (3, dict(d=48)), (3, dict(d=2048)), (3, dict(n=-1)), (1, dict(rows=None)),
    (2, dict(rows=BAD)), (1, dict(codes=None)), (1, dict(scales=None)), (2, dict(values=BAD)),
    (1, dict(stride=127)), (2, dict(stride=132)), (1, dict(n_out=3)), (2, dict(slots=BAD)),
])
def test_quantize_mxfp4_refusals(lib, want, kw):
    a = dict(dtype=1, rows=OK, stride=128, n=4, d=128, slots=None, n_out=4, codes=OK, scales=OK,
             values=None)
    a.update(kw)
    assert lib.csa_quantize_mxfp4(a["dtype"], a["rows"], a["stride"], a["n"], a["d"], a["slots"],
                                  a["n_out"], a["codes"], a["scales"], a["values"], None) == want


def test_quantize_mxfp4_of_no_rows_does_nothing(lib):
    assert lib.csa_quantize_mxfp4(1, None, 128, 0, 128, None, 0, None, None, None, None) == 0


def _scores(lib, table=OK, width=4, pages=9, page=64, n_max=200, Bn=2, Tq=1, qc=OK, kc=OK, w=OK,
            out=OK, **params):
    return lib.csa_index_scores_mxfp4(_pp(**params), qc, OK, w, kc, OK, table, width, pages, page,
                                      OK, OK, Bn, Tq, n_max, out, None)


@pytest.mark.parametrize("want,kw", [
    (3, dict(page=4)), (3, dict(page=48)), (3, dict(page=1 << 21)), (3, dict(pages=-1)),
    (3, dict(pages=1 << 28)), (3, dict(width=1 << 26)), (1, dict(n_max=257)), (1, dict(table=None)),
    (2, dict(table=BAD)), (3, dict(idx_dim=48)), (3, dict(idx_heads=200)), (3, dict(Bn=0)),
    (3, dict(Bn=40000, Tq=2)), (1, dict(qc=None)), (2, dict(kc=BAD)), (1, dict(w=None)),
    (1, dict(out=None)),
    (3, dict(table=None, width=0, Bn=30000, n_max=100000)),
])
def test_index_scores_mxfp4_refusals(lib, want, kw):
    assert _scores(lib, **kw) == want, lib.csa_last_error_detail()


def test_index_topk_mxfp4_wants_its_workspace(lib):
    nb = csa.csa_workspace_size(csa.Params(), csa.CSA_OP_INDEX_TOPK, 2, 1, 200)
    args = (_pp(), OK, OK, OK, OK, OK, OK, 4, 9, 64, OK, OK, 2, 1, 200, OK)
    assert lib.csa_index_topk_mxfp4(*args, OK, nb - 1, None) == 5
    assert lib.csa_index_topk_mxfp4(*args, None, nb, None) == 1
    assert lib.csa_index_topk_mxfp4(_pp(topk=0), *args[1:], OK, nb, None) == 3


@pytest.mark.parametrize("call", ["csa_sparse_attn_paged", "hca_attn_paged"])
@pytest.mark.parametrize("want,kw", [
    (3, dict(page=7)), (3, dict(page=24)), (3, dict(pages=1 << 27)), (3, dict(d=96)),
    (1, dict(table=None)), (1, dict(sel=None)), (2, dict(sel=BAD)), (1, dict(sink=None)),
    (1, dict(raw=None)), (1, dict(raw_max=-1)), (2, dict(out=BAD)), (1, dict(kv=None)),
    (3, dict(Bn=300, Tq=300)), (1, dict(dtype=9)),
])
def test_paged_attention_refusals(lib, call, want, kw):
    a = dict(dtype=1, q=OK, kv=OK, pages=9, page=64, table=OK, width=4, sel=OK, raw=OK, raw_max=4,
             sink=OK, Bn=2, Tq=1, out=OK)
    params = {k: v for k, v in kw.items() if k == "d"}
    a.update({k: v for k, v in kw.items() if k != "d"})
    st = getattr(lib, call)(_pp(**params), a["dtype"], a["q"], OK, a["kv"], a["pages"], a["page"],
                            a["table"], a["width"], a["sel"], a["raw"], OK, OK, a["raw_max"],
                            a["sink"], a["Bn"], a["Tq"], a["out"], OK, 1 << 40, None)
    assert st == want, lib.csa_last_error_detail()


@pytest.mark.parametrize("op", [csa.CSA_OP_SPARSE_ATTN_PAGED, csa.CSA_OP_HCA_ATTN_PAGED])
def test_paged_workspace_sizes(lib, op):
    for p in (csa.Params(), csa.Params(n_heads=3, d=64, rope_dim=32), csa.Params(n_heads=16)):
        for n in (0, 8, 1000, 1 << 20):
            nb = csa.csa_workspace_size(p, op, 3, 1, n)
            assert nb >= 0 and nb % 16 == 0
            assert nb <= 1 << 30


def test_binding_refuses_host_tensors():
    p = csa.Params()
    x = torch.zeros(2, 4, 128)
    with pytest.raises(ValueError):
        layer.norm_rope(p, x)
    with pytest.raises(ValueError):
        layer.quantize_mxfp4(x)
    with pytest.raises(TypeError):
        csa.csa_quantize_mxfp4(None, None, None)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        csa.csa_index_scores_mxfp4(p, x, x, x, x, x, i, i, i[0], torch.zeros(1, 1, 8))
    with pytest.raises(ValueError):
        csa.hca_attn_paged(p, x, i, x, i, i[0], x, i[0], i[0], x[0, 0], x)
    with pytest.raises(ValueError):
        csa.csa_sparse_attn_paged(p, x, i, x, i, i, x, i[0], i[0], x[0, 0], x)
