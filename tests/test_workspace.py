"""layer.Workspace: a buffer that a captured graph uses outlives its growth,
and one that another stream uses is not handed out again under that stream's
calls."""
import weakref

import pytest
import torch

from sparse_compressed_attention_csa_b200 import layer


class _Buffer(torch.Tensor):
    """A host tensor that says it is on cuda:0 and keeps who used it."""

    is_cuda = True
    device = torch.device("cuda", 0)

    def record_stream(self, stream):
        self.used_on = getattr(self, "used_on", []) + [stream]


@pytest.fixture
def fake(monkeypatch):
    state = dict(stream=0, capturing=False)
    empty = torch.empty
    monkeypatch.setattr(layer.torch, "empty", lambda n, dtype, device: empty(n, dtype=dtype).as_subclass(_Buffer))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: state["stream"], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: state["stream"])
    return state


def test_an_outgrown_buffer_of_a_graph_is_kept(fake):
    ws = layer.Workspace("cuda")
    first = ws.get(100)
    ref = weakref.ref(first)
    del first
    ws.get(200)
    assert ref() is None                     # only eager calls used it
    fake["capturing"] = True
    second = weakref.ref(ws.get(150))
    fake["capturing"] = False
    assert ws.get(200) is second()
    ws.get(300)
    assert second() is not None              # the graph replays with it
    third = weakref.ref(ws.get(300))
    ws.get(400)
    assert third() is None and second() is not None
    del ws
    assert second() is None


def test_a_buffer_used_on_another_stream_is_recorded_there(fake):
    ws = layer.Workspace("cuda")
    buf = ws.get(100)
    ws.get(50)
    assert not hasattr(buf, "used_on")
    fake["stream"] = 7
    assert ws.get(60) is buf and buf.used_on == [7]
    assert ws.get(120) is not buf and not hasattr(ws.get(120), "used_on")


@pytest.mark.gpu
def test_a_graph_replays_after_its_workspace_grew():
    from gpu_util import assert_close, host64
    from test_gpu_paged import _case, _hca
    p, t, want = _case("bf16", 128, 512, 64, [9000, 4000], 1, 64, 1, 1, 128, 83)
    big = _case("bf16", 128, 512, 64, [9000, 30000, 20000], 1, 64, 1, 1, 128, 84)
    small = layer.Workspace("cuda")
    out = torch.empty_like(t["q"])
    _hca(p, t, ws=small, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _hca(p, t, ws=small, out=out)
    used = small.buf
    n, at = used.numel(), used.data_ptr()
    del used
    small.get(4 * n)                         # a larger call's
    other = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(o.data_ptr() != at for o in other)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in other)
    assert_close(host64(out), want, "bf16", "replay")
    got = _hca(*big[:2], ws=small)
    assert_close(host64(got), big[2], "bf16", "the larger call")
