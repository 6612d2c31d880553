"""The binding of the paged calls on the CPU: what reaches the library, with
the device checks answered for host tensors and a library that records."""
import pytest
import torch

import sparse_compressed_attention_csa_b200 as csa
from sparse_compressed_attention_csa_b200 import _lib as L

I32, U8 = torch.int32, torch.uint8


class _Recorder:
    """A library whose calls succeed and are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def recorded(monkeypatch):
    """Host tensors (device index -1) pass the device checks."""
    lib = _Recorder()
    monkeypatch.setattr(L, "_load", lambda: lib)
    monkeypatch.setattr(L, "_device_of", lambda t, name: -1)
    monkeypatch.setattr(L, "_stream", lambda s: None)
    return lib


def _keys(B, width, pages=3, page=16):
    z = torch.zeros
    return dict(q_codes=z(B, 1, 64, 64, dtype=U8), q_scales=z(B, 1, 64, 4, dtype=U8), w=z(B, 1, 64),
                k_codes=z(pages, page, 64, dtype=U8), k_scales=z(pages, page, 4, dtype=U8),
                page_table=z(B, width, dtype=I32), q_pos=z(B, 1, dtype=I32), n_cmp=z(B, dtype=I32))


def test_an_empty_page_table_is_not_contiguous_keys(recorded):
    # the pool's pages are as many as sequences, its rows fewer than n_max
    p = csa.Params(topk=4)
    t = _keys(3, 0)
    with pytest.raises(ValueError, match="empty page table"):
        csa.csa_index_scores_mxfp4(p, *t.values(), torch.zeros(3, 1, 40))
    idx = torch.zeros(3, 1, 4, dtype=I32)
    with pytest.raises(ValueError, match="empty page table"):
        csa.csa_index_topk_mxfp4(p, *t.values(), idx, None, 40)
    assert not recorded.calls
    # with nothing to score it is an ordinary call of no keys
    csa.csa_index_scores_mxfp4(p, *t.values(), torch.zeros(3, 1, 0))
    csa.csa_index_topk_mxfp4(p, *t.values(), idx, None)
    for _, args in recorded.calls:
        assert args[12:15] == (3, 1, 0)                        # B, Tq, n_max
    # and a table with entries reaches the library as one
    t = _keys(3, 3)
    csa.csa_index_scores_mxfp4(p, *t.values(), torch.zeros(3, 1, 40))
    args = recorded.calls[-1][1]
    assert args[6] == t["page_table"].data_ptr() and args[7:10] == (3, 3, 16)


def test_params_travel_after_a_call(recorded):
    # what a call keeps with the parameter set stays behind
    import copy
    import pickle
    p = csa.Params(topk=4, rope_factor=16.0, rope_orig_ctx=65536)
    t = _keys(3, 3)
    csa.csa_index_scores_mxfp4(p, *t.values(), torch.zeros(3, 1, 40))
    L._ws_bytes(p, csa.CSA_OP_HCA_ATTN_PAGED, 1, 1, 64, -1)
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and hash(q) == hash(p)
        csa.csa_index_scores_mxfp4(q, *t.values(), torch.zeros(3, 1, 40))
        assert q.c() is not p.c() and bytes(q.c()) == bytes(p.c())


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:1."""

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda", 1)


@pytest.mark.parametrize("call", ["hca_decode_paged", "sparse_attn_paged", "csa_decode_paged"])
def test_a_call_for_another_device_leaves_no_workspace_size(monkeypatch, call):
    # sizes are asked of the current device; a tensor elsewhere is refused before
    from sparse_compressed_attention_csa_b200 import layer
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    asked = []
    monkeypatch.setattr(L, "csa_workspace_size", lambda *a: asked.append(a) or 256)
    monkeypatch.setattr(layer, "quantize_mxfp4", lambda rows, stream=None: (rows, rows))
    p = csa.Params(topk=4)
    z = torch.zeros
    q = z(2, 1, 128, 512).as_subclass(_OnDevice)
    i1, i2, kv = z(2, dtype=I32), z(2, 1, dtype=I32), z(3, 16, 512)
    tail = (z(2, 4, 512), i1, i1, z(128))
    ws = layer.Workspace("cpu")
    with pytest.raises(ValueError, match="current device is cuda:0"):
        if call == "csa_decode_paged":
            t = _keys(2, 2)
            layer.csa_decode_paged(p, q, i2, z(2, 1, 64, 128), t["w"], t["k_codes"], t["k_scales"], i1, kv,
                                   t["page_table"], *tail, ws=ws)
        else:
            sel = i1 if call == "hca_decode_paged" else z(2, 1, 4, dtype=I32)
            getattr(layer, call)(p, q, i2, kv, z(2, 2, dtype=I32), sel, *tail, ws=ws)
    assert not asked and not p.__dict__.get("_ws")
