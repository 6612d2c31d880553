"""Attention over paged caches against the fp64 oracle, at the layer's own
bounds (bf16: max-abs 2e-2 and relative L2 5e-3; fp32: 1e-5).  The pool's
unused rows hold NaN and unused table entries a page outside the pool."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_close, host64
from sparse_compressed_attention_csa_b200 import (CSA_OP_HCA_ATTN_PAGED, CsaError, Params,
                                                  csa_poll_device_error, csa_workspace_size,
                                                  hca_attn_paged, layer)
from test_gpu_mxfp4 import paged

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _case(dtype, H, d, rope, lens, Tq, page, width, stride, window, seed, topk=0, keep_raw=None,
          scale_q=1.0):
    rng = np.random.default_rng(seed)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    val = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(tdt)  # noqa: E731
    B = len(lens)
    n_cmp = [oracle.n_compressed(t, width, stride) for t in lens]
    kv = [val(n, d) for n in n_cmp]
    raw_max = max(1, window + Tq if keep_raw is None else keep_raw)
    raw = val(B, raw_max, d)
    pos0 = [max(0, t - raw_max) for t in lens]
    n_raw = [min(t, raw_max) for t in lens]
    for b in range(B):
        raw[b, n_raw[b]:] = float("nan")
    q = val(B, Tq, H, d) * scale_q
    sink = rng.standard_normal(H).astype(np.float32)
    q_pos = np.array([[t - Tq + i for i in range(Tq)] for t in lens], dtype=np.int32)
    pool, table = paged([k.float().numpy() for k in kv], page, seed, np.nan)
    c = lambda a, dt: torch.as_tensor(a).to(dt).cuda()  # noqa: E731
    t = dict(q=q.cuda(), q_pos=c(q_pos, I32), kv=c(pool, tdt), table=c(table, I32), raw=raw.cuda(),
             pos0=c(pos0, I32), n_raw=c(n_raw, I32), sink=c(sink, torch.float32), n_cmp=c(n_cmp, I32))
    p = Params(d=d, rope_dim=rope, n_heads=H, topk=max(topk, 1), window=window, width=width, stride=stride)
    idx = None
    if topk:
        idx = np.full((B, Tq, topk), -1, dtype=np.int32)
        for b in range(B):
            for i in range(Tq):
                n = oracle.n_visible(int(q_pos[b, i]), n_cmp[b], width, stride)
                pick = np.sort(rng.permutation(n)[:topk])
                idx[b, i, :len(pick)] = pick
        t["idx"] = c(idx, I32)
    scale = 1.0 / np.sqrt(d)
    want = []
    for b in range(B):
        f = lambda a: a.double().numpy()  # noqa: E731
        args = (f(raw[b]), pos0[b], n_raw[b], sink, scale, window)
        if topk:
            want.append(oracle.sparse_attn(f(q[b]), q_pos[b], f(kv[b]), idx[b], *args, rope, 1e4))
        else:
            want.append(oracle.hca_attn(f(q[b]), q_pos[b], f(kv[b]), n_cmp[b], *args, width, stride, rope, 1e4))
    return p, t, np.stack(want)


def _hca(p, t, **kw):
    return layer.hca_decode_paged(p, t["q"], t["q_pos"], t["kv"], t["table"], t["n_cmp"], t["raw"], t["pos0"],
                                  t["n_raw"], t["sink"], **kw)


def _sparse(p, t, **kw):
    return layer.sparse_attn_paged(p, t["q"], t["q_pos"], t["kv"], t["table"], t["idx"], t["raw"], t["pos0"],
                                   t["n_raw"], t["sink"], **kw)


HCA = [
    # dtype, H, d, rope, lens, Tq, page, width, stride, window
    ("bf16", 128, 512, 64, [1], 1, 64, 1, 1, 0),
    ("bf16", 128, 512, 64, [64, 65, 63, 1], 1, 8, 1, 1, 0),
    ("bf16", 128, 512, 64, [2000, 37], 1, 16, 1, 1, 0),
    ("bf16", 128, 512, 64, [40000, 5, 129 * 128], 1, 64, 128, 128, 128),
    ("bf16", 128, 512, 64, [9001, 300, 4097], 2, 32, 1, 1, 128),
    ("bf16", 128, 512, 64, [30000], 1, 128, 1, 1, 16),
    ("bf16", 128, 512, 128, [3000, 2999], 1, 256, 4, 4, 100),
    ("bf16", 128, 512, 0, [777], 3, 64, 1, 1, 128),
    ("bf16", 16, 512, 64, [5000, 17], 1, 64, 1, 1, 128),
    ("bf16", 64, 512, 64, [3000], 2, 64, 2, 2, 128),
    ("bf16", 5, 512, 64, [1300, 2], 1, 64, 1, 1, 8),
    ("bf16", 200, 512, 64, [900, 64], 1, 64, 1, 1, 128),
    ("bf16", 128, 512, 64, [100] * 9, 7, 64, 1, 1, 20),
    ("bf16", 128, 512, 64, [10, 90, 100, 127], 1, 64, 128, 128, 128),     # no entry yet
    ("bf16", 128, 512, 64, [700] * 160, 1, 64, 1, 1, 0),
    ("bf16", 3, 64, 32, [500, 1], 1, 16, 1, 1, 16),
    ("bf16", 8, 128, 64, [5000], 2, 64, 1, 1, 128),
    ("bf16", 4, 256, 64, [700], 1, 8, 1, 1, 0),
    ("bf16", 2, 1024, 64, [700], 1, 64, 1, 1, 3),
    ("f32", 3, 64, 32, [256, 9, 100], 2, 8, 4, 4, 16),
    ("f32", 8, 128, 64, [3000], 1, 64, 1, 1, 0),
    ("f32", 128, 512, 64, [400, 130], 1, 64, 1, 1, 128),
    ("f32", 1, 1024, 0, [90], 1, 16, 1, 1, 4),
]


@pytest.mark.parametrize("c", HCA, ids=lambda c: str(c)[:60])
def test_hca_paged(c):
    p, t, want = _case(*c, seed=HCA.index(c))
    out = _hca(p, t)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert_close(host64(out), want, c[0], str(c))


SPARSE = [
    # dtype, H, d, rope, lens, Tq, page, width, stride, window, topk
    ("bf16", 128, 512, 64, [20000, 5003], 1, 64, 8, 4, 128, 1024),
    ("bf16", 128, 512, 64, [5003, 2001, 40], 2, 16, 8, 4, 128, 1024),
    ("bf16", 128, 512, 64, [3000], 1, 8, 2, 2, 128, 512),
    ("bf16", 128, 512, 64, [9000] * 3, 1, 256, 8, 4, 0, 64),
    ("bf16", 128, 512, 64, [7, 3, 9], 1, 64, 8, 4, 128, 64),
    ("bf16", 128, 512, 64, [30000], 1, 64, 8, 4, 128, 4096),              # past one pair's row list
    ("bf16", 16, 512, 64, [3000], 1, 64, 8, 4, 128, 256),
    ("f32", 3, 64, 32, [256, 20], 2, 16, 8, 4, 5, 7),
    ("f32", 8, 128, 64, [3000], 1, 64, 8, 4, 128, 100),
]


@pytest.mark.parametrize("c", SPARSE, ids=str)
def test_sparse_paged(c):
    p, t, want = _case(*c[:10], seed=50 + SPARSE.index(c), topk=c[10])
    out = _sparse(p, t)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert_close(host64(out), want, c[0], str(c))


def test_paged_agrees_with_a_contiguous_cache():
    # the same rows through pages and from a contiguous cache
    from sparse_compressed_attention_csa_b200 import CSA_OP_SPARSE_ATTN, csa_sparse_attn
    p, t, _ = _case("bf16", 128, 512, 64, [9000, 4001], 1, 64, 8, 4, 128, 70, topk=1024)
    n_max = t["table"].shape[1] * 64
    flat = torch.zeros(2, n_max, 512, dtype=torch.bfloat16, device="cuda")
    for b in range(2):
        n = int(t["n_cmp"][b])
        flat[b, :n] = t["kv"][t["table"][b, :-(-n // 64)].long()].flatten(0, 1)[:n]
    out = torch.empty_like(t["q"])
    ws = torch.empty(max(256, csa_workspace_size(p, CSA_OP_SPARSE_ATTN, 2, 1, n_max)), dtype=torch.uint8,
                     device="cuda")
    csa_sparse_attn(p, t["q"], t["q_pos"], flat, t["idx"], t["raw"], t["pos0"], t["n_raw"], t["sink"], out, ws)
    got = _sparse(p, t)
    assert_close(host64(got), host64(out), "bf16", "paged against contiguous")


def test_large_logits_and_sinks():
    # one row dominates (the running maximum moves far), and sinks of +-inf scale
    p, t, want = _case("bf16", 128, 512, 64, [3000, 70], 1, 64, 1, 1, 128, 71, scale_q=6.0)
    out = _hca(p, t)
    assert_close(host64(out), want, "bf16", "large logits")
    t["sink"].fill_(-float("inf"))
    out = _hca(p, t)
    assert torch.isfinite(out).all()
    # nothing visible, no window and no sink: zeros
    p0 = Params(window=0, width=128, stride=128)
    t["q_pos"].fill_(5)
    out = _hca(p0, t)
    assert torch.all(out == 0)
    csa_poll_device_error()


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_scales_of_any_sign(scale):
    p, t, _ = _case("bf16", 128, 512, 64, [700, 70], 1, 64, 1, 1, 20, 77)
    p = Params(window=20, width=1, stride=1, scale=scale)
    out = host64(_hca(p, t))
    f = lambda a: a.double().cpu().numpy()  # noqa: E731
    for b in range(2):
        n = int(t["n_cmp"][b])
        want = oracle.hca_attn(f(t["q"][b]), t["q_pos"][b].cpu().numpy(),
                               oracle.paged_rows(t["kv"].float().cpu().numpy(), t["table"][b].cpu().numpy(), n), n,
                               f(t["raw"][b]), int(t["pos0"][b]), int(t["n_raw"][b]), t["sink"].cpu().numpy(),
                               scale, 20, 1, 1, 64, 1e4)
        assert_close(out[b], want, "bf16", f"scale {scale}")


@pytest.mark.parametrize("H,d,dtype", [(128, 512, "bf16"), (3, 64, "f32")])
def test_pages_outside_the_pool_are_reported_and_skipped(H, d, dtype):
    rope = 64 if d == 512 else 32
    p, t, want = _case(dtype, H, d, rope, [1000, 640], 1, 16, 1, 1, 0, 72)
    t["table"][0, 2] = -1                                   # entries 32 .. 47 of sequence 0
    t["table"][0, 40] = t["kv"].shape[0]                    # entries 640 .. 655
    out = _hca(p, t)
    with pytest.raises(CsaError) as ei:
        csa_poll_device_error()
    assert ei.value.status == 8
    n = 1000
    keep = [j for j in range(n) if not (32 <= j < 48 or 640 <= j < 656)]
    rows = t["kv"].flatten(0, 1).double().cpu().numpy()
    tab = t["table"][0].cpu().numpy().astype(np.int64)
    ent = np.stack([rows[tab[j // 16] * 16 + j % 16] for j in keep])
    want0 = oracle.attend(t["q"][0, 0].double().cpu().numpy(), 999, ent, t["sink"].cpu().numpy(),
                          1 / np.sqrt(d), rope, 1e4)
    assert_close(host64(out)[0, 0], want0, dtype, "bad pages")
    assert_close(host64(out)[1], want[1], dtype, "the other sequence")


def test_bad_selection_pages_are_reported_and_skipped():
    p, t, want = _case("bf16", 128, 512, 64, [4000, 4000], 1, 16, 8, 4, 128, 73, topk=128)
    t["table"][0, int(t["idx"][0, 0, 5]) // 16] = -3
    t["idx"][0, 0, 9] = t["table"].shape[1] * 16
    out = _sparse(p, t)
    with pytest.raises(CsaError) as ei:
        csa_poll_device_error()
    assert ei.value.status == 8
    assert torch.isfinite(out).all()
    assert_close(host64(out)[1], want[1], "bf16", "the other sequence")


def test_results_repeat_in_place_on_streams_and_from_two_graphs():
    p, t, want = _case("bf16", 128, 512, 64, [9000, 41, 4000], 1, 64, 1, 1, 128, 74)
    first = _hca(p, t)
    assert_close(host64(first), want, "bf16", "first")
    for _ in range(5):
        assert torch.equal(_hca(p, t), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = _hca(p, t)
    side.synchronize()
    assert torch.equal(a, first)
    # two graphs that share a workspace, replayed one after the other
    ws = layer.Workspace("cuda")
    outs = [torch.zeros_like(first) for _ in range(2)]
    _hca(p, t, ws=ws, out=outs[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _hca(p, t, ws=ws, out=o)
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
    csa_poll_device_error()


def test_no_pages_and_negative_counts():
    # an empty pool and table: the window and the sink alone; then nothing at all
    p, t, _ = _case("bf16", 128, 512, 64, [300, 7], 1, 64, 128, 128, 128, 78)
    f = lambda a: a.double().cpu().numpy()  # noqa: E731
    want = [oracle.hca_attn(f(t["q"][b]), t["q_pos"][b].cpu().numpy(), np.zeros((0, 512)), 0, f(t["raw"][b]),
                            int(t["pos0"][b]), int(t["n_raw"][b]), t["sink"].cpu().numpy(), 1 / np.sqrt(512), 128,
                            128, 128, 64, 1e4) for b in range(2)]
    empty = dict(t, kv=t["kv"][:0], table=t["table"][:, :0].contiguous())
    assert_close(host64(_hca(p, empty)), np.stack(want), "bf16", "no pages")
    idx = torch.full((2, 1, 1), -1, dtype=I32, device="cuda")
    assert_close(host64(_sparse(p, dict(empty, idx=idx))), np.stack(want), "bf16", "no pages, selection")
    for dt in (torch.bfloat16, torch.float32):
        u = {k: (v.to(dt) if v.dtype == torch.bfloat16 else v) for k, v in t.items()}
        u["n_cmp"] = torch.full_like(t["n_cmp"], -3)
        u["n_raw"] = torch.full_like(t["n_raw"], -1)
        assert torch.all(_hca(p, u) == 0)
    csa_poll_device_error()


def test_padded_batch_and_no_raw_rows():
    # a padding row of a batch (position -1) gives zeros, the others their own;
    # a cache without raw rows has no window
    p, t, want = _case("bf16", 128, 512, 64, [600, 500, 2000], 1, 64, 1, 1, 128, 84)
    t["q_pos"][1] = -1
    out = _hca(p, t)
    assert torch.all(out[1] == 0)
    assert_close(host64(out)[[0, 2]], want[[0, 2]], "bf16", "beside padding")
    p0, t0, want0 = _case("bf16", 128, 512, 64, [600, 70], 1, 64, 1, 1, 0, 85)
    none = dict(t0, raw=t0["raw"][:, :0].contiguous(), n_raw=torch.zeros_like(t0["n_raw"]))
    assert_close(host64(_hca(Params(width=1, stride=1), none)), want0, "bf16", "no raw rows")
    csa_poll_device_error()


@pytest.mark.parametrize("B,rope,window", [(3, 64, 128), (15, 128, 128), (18, 64, 0), (30, 128, 128), (50, 64, 128),
                                           (74, 128, 0), (80, 64, 128)])
@pytest.mark.parametrize("selected", [False, True])
def test_a_token_on_one_to_four_pairs(B, rope, window, selected):
    # short tokens in batches that leave a token four CTA pairs, three, two, one
    # and a share of one: empty tokens, and pairs that get no tile, among them
    rng = np.random.default_rng(B)
    lens = [1, 0, 65] + [int(n) for n in rng.integers(0, 250, B - 3)]
    p, t, want = _case("bf16", 128, 512, rope, lens, 1, 16, 1, 1, window, 200 + B, topk=100 if selected else 0)
    out = (_sparse if selected else _hca)(p, t)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert_close(host64(out), want, "bf16", f"{B} tokens")
    assert torch.equal(out, (_sparse if selected else _hca)(p, t))


@pytest.mark.parametrize("heads", [40, 256])
def test_head_groups_on_several_pairs(heads):
    p, t, want = _case("bf16", heads, 512, 64, [300, 90], 2, 16, 1, 1, 128, 240 + heads)
    out = _hca(p, t)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert_close(host64(out), want, "bf16", f"{heads} heads")


def test_nan_rows_reach_their_own_token_only():
    # one row of one pair's share; a query; a sink
    p, t, want = _case("bf16", 128, 512, 64, [350, 340, 330, 320], 1, 16, 1, 1, 0, 260)
    kv = t["kv"].clone()
    page, row = int(t["table"][0, 5]), 3
    kv[page, row] = float("nan")
    t["kv"] = kv
    t["q"][1, 0, 7] = float("nan")
    t["sink"][9] = float("nan")
    out = host64(_hca(p, t))
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert np.all(np.isnan(out[0])) and np.all(np.isnan(out[1, 0, 7]))
    assert np.all(np.isnan(out[:, 0, 9]))
    keep = np.ones(128, dtype=bool)
    keep[[7, 9]] = False
    assert_close(out[1:][:, :, keep], want[1:][:, :, keep], "bf16", "beside NaN")


def test_two_calls_at_once_on_two_streams():
    a = _case("bf16", 128, 512, 64, [20000, 300], 1, 64, 1, 1, 128, 86)
    b = _case("bf16", 128, 512, 64, [9000, 4000, 50], 1, 64, 8, 4, 128, 87, topk=512)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        with torch.cuda.stream(streams[0]):
            x = _hca(a[0], a[1])
        with torch.cuda.stream(streams[1]):
            y = _sparse(b[0], b[1])
        outs.append((x, y))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, outs[0][0]) and torch.equal(y, outs[0][1])
    assert_close(host64(outs[0][0]), a[2], "bf16", "one stream")
    assert_close(host64(outs[0][1]), b[2], "bf16", "the other")


def test_another_token_with_nan_queries_and_fewer_heads_than_a_tile():
    # the matrix tile of a 16-head token reaches into the next tokens' queries
    p, t, want = _case("bf16", 16, 512, 64, [900, 800, 700], 1, 64, 1, 1, 64, 79)
    t["q"][1] = float("nan")
    out = _hca(p, t)
    assert torch.isnan(out[1]).all()
    assert_close(host64(out)[[0, 2]], want[[0, 2]], "bf16", "the other tokens")


def test_the_same_entry_twice_counts_twice():
    p, t, _ = _case("bf16", 128, 512, 64, [2000], 1, 64, 8, 4, 16, 80, topk=100)
    t["idx"][0, 0, 50:] = t["idx"][0, 0, :50].flip(0)
    t["idx"][0, 0, 10] = -1                              # unused places anywhere
    f = lambda a: a.double().cpu().numpy()  # noqa: E731
    n = int(t["n_cmp"][0])
    want = oracle.sparse_attn(f(t["q"][0]), t["q_pos"][0].cpu().numpy(),
                              oracle.paged_rows(t["kv"].float().cpu().numpy(), t["table"][0].cpu().numpy(), n),
                              t["idx"][0].cpu().numpy(), f(t["raw"][0]), int(t["pos0"][0]), int(t["n_raw"][0]),
                              t["sink"].cpu().numpy(), 1 / np.sqrt(512), 16, 64, 1e4)
    assert_close(host64(_sparse(p, t))[0], want, "bf16", "duplicates")


@pytest.mark.parametrize("sparse", [False, True])
def test_pages_past_four_gigabytes(sparse):
    # a pool of 5.2 GB whose used pages are its last: element offsets past 2^31
    p, t, want = _case("bf16", 128, 512, 64, [3000], 1, 64, 8, 4, 128, 81, topk=256 if sparse else 0)
    total, used = 80000, t["kv"].shape[0]
    pool = torch.empty((total, 64, 512), dtype=torch.bfloat16, device="cuda")
    pool[total - used:] = t["kv"]
    live = t["table"] < used
    t["table"][live] += total - used
    big = dict(t, kv=pool)
    out = _sparse(p, big) if sparse else _hca(p, big)
    assert_close(host64(out), want, "bf16", "far pages")
    csa_poll_device_error()


def test_calls_on_a_given_stream_allocate_for_it():
    p, t, want = _case("bf16", 128, 512, 64, [4000, 41], 1, 64, 8, 4, 128, 82, topk=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):                                   # results held, workspaces freed at once
        outs.append(_sparse(p, t, stream=side))
        torch.empty(1 << 22, device="cuda").fill_(7.0)   # another stream's use of freed memory
    side.synchronize()
    assert_close(host64(outs[0]), want, "bf16", "side stream")
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_waits_that_run_out_end_the_call_and_the_next_one_is_right():
    # a limit of 1 ns: a wait that is not over at its first try gives up; every
    # role winds down within its bounded drains
    from sparse_compressed_attention_csa_b200 import csa_set_wait_limit_ns
    p, t, want = _case("bf16", 128, 512, 64, [9000, 4000], 1, 64, 1, 1, 128, 83)
    _hca(p, t)
    torch.cuda.synchronize()
    csa_set_wait_limit_ns(1)
    try:
        _hca(p, t)
        torch.cuda.synchronize()
        try:
            csa_poll_device_error()
        except CsaError as e:
            assert e.status == 7
    finally:
        csa_set_wait_limit_ns(0)
    out = _hca(p, t)
    csa_poll_device_error()
    assert_close(host64(out), want, "bf16", "after a failed launch")


def test_workspace_too_small_is_refused():
    p, t, _ = _case("bf16", 128, 512, 64, [9000], 1, 64, 1, 1, 0, 75)
    nb = csa_workspace_size(p, CSA_OP_HCA_ATTN_PAGED, 1, 1, t["table"].shape[1] * 64)
    assert nb > 0
    with pytest.raises(CsaError) as ei:
        hca_attn_paged(p, t["q"], t["q_pos"], t["kv"], t["table"], t["n_cmp"], t["raw"], t["pos0"], t["n_raw"],
                       t["sink"], torch.empty_like(t["q"]), torch.empty(nb - 16, dtype=torch.uint8, device="cuda"))
    assert ei.value.status == 5


def test_a_decode_step_through_every_operator():
    """Norm and rotation of new keys and entries into pages, 4-bit keys, then
    the decode over both caches: each step against the oracle on what the
    step before it gave."""
    rng = np.random.default_rng(76)
    B, T, page, topk = 3, [2600, 1411, 90], 32, 256
    p = Params(topk=topk)
    bf = torch.bfloat16
    n_cmp = [oracle.n_compressed(t, 8, 4) for t in T]
    per = [-(-n // page) for n in n_cmp]
    table = np.zeros((B, max(per)), dtype=np.int32)
    order, at = rng.permutation(sum(per)), 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
    slots = np.concatenate([table[b][np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(n_cmp)])
    pos = np.concatenate([4 * np.arange(n) for n in n_cmp])
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    val = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(bf)  # noqa: E731
    N = len(slots)
    keys, entries = val(N, 1, 128), val(N, 1, 512)
    q_idx, q = val(B, 64, 128), val(B, 128, 512)
    kw, qw = 1 + 0.1 * torch.randn(128, device="cuda"), 1 + 0.1 * torch.randn(128, device="cuda")
    q_pos = np.array([[t - 1] for t in T], dtype=np.int32)
    slots_d, pos_d = c(slots), c(pos)
    # caches: normed and rotated entries straight into pages; keys normed, rotated, quantized into pages
    kv = torch.full((sum(per), page, 512), float("nan"), dtype=bf, device="cuda")
    layer.norm_rope(p, q, None, None, entries, None, pos_d, kv.view(-1, 1, 512), slots_d)
    q_idx_n, keys_n = layer.norm_rope(p, q_idx, qw, c(q_pos[:, 0]), keys, kw, pos_d)
    k_codes = torch.zeros(sum(per), page, 64, dtype=torch.uint8, device="cuda")
    k_scales = torch.full((sum(per), page, 4), 255, dtype=torch.uint8, device="cuda")
    from sparse_compressed_attention_csa_b200 import csa_quantize_mxfp4
    csa_quantize_mxfp4(keys_n[:, 0], k_codes, k_scales, slots=slots_d)
    raw, w, sink = val(B, 128, 512), torch.rand(B, 1, 64, device="cuda"), torch.randn(128, device="cuda")
    pos0 = c([max(0, t - 128) for t in T])
    n_raw = c([min(t, 128) for t in T])
    idx, out = layer.csa_decode_paged(p, q[:, None], c(q_pos), q_idx_n[:, None], w, k_codes, k_scales, c(n_cmp),
                                      kv, c(table), raw, pos0, n_raw, sink)
    torch.cuda.synchronize()
    csa_poll_device_error()
    at = 0
    for b in range(B):
        n = n_cmp[b]
        ent = oracle.paged_rows(kv.float().cpu().numpy(), table[b], n)
        ent_o = oracle.norm_rope(entries[at:at + n].double().cpu().numpy(), None, pos[at:at + n], 64, 1e4, 1e-6)[:, 0]
        assert_close(ent, ent_o, "bf16", "entries in pages")
        kc, ks = oracle.mxfp4_encode(keys_n[at:at + n, 0].double().cpu().numpy())
        np.testing.assert_array_equal(oracle.paged_rows(k_codes.cpu().numpy(), table[b], n), kc)
        qv = oracle.mxfp4_decode(*oracle.mxfp4_encode(q_idx_n[b].double().cpu().numpy()))
        s = oracle.index_scores(qv[None], w[b].cpu().numpy(), oracle.mxfp4_decode(kc, ks))[0]
        got = idx[b, 0].cpu().numpy()
        got = got[got >= 0]
        assert len(got) == min(topk, n) and np.all(np.diff(got) > 0)
        if n > topk:  # every kept score reaches the k-th best, up to the fp32 sums
            cut = np.sort(s)[-topk]
            assert np.all(s[got] >= cut - 1e-4 * np.abs(s).max())
        want = oracle.sparse_attn(q[b:b + 1].double().cpu().numpy(), q_pos[b], ent, idx[b].cpu().numpy(),
                                  raw[b].double().cpu().numpy(), int(pos0[b]), int(n_raw[b]), sink.cpu().numpy(),
                                  1 / np.sqrt(512), 128, 64, 1e4)
        assert_close(host64(out)[b], want, "bf16", "decode")
        at += n
