"""MXFP4 on the GPU: the quantizer bit for bit against the oracle, and the
indexer's product on 4-bit queries and (paged) keys.

Scores: a product of two E2M1 values and their scales is exact; a score sums
d_I products per head and then H_I weighted heads in fp32.  With every
addition off by at most 2^-23 of the sum of magnitudes so far (the matrix
unit may truncate; a rounded addition is off by half of that), a score is
within (d_I + 2 H_I) 2^-23 sum_h |w_h| sum_c |q_hc k_c|."""
import numpy as np
import pytest
import torch

import oracle
from sparse_compressed_attention_csa_b200 import (CSA_OP_INDEX_TOPK, CsaError, Params,
                                                  csa_index_scores_mxfp4, csa_index_topk_mxfp4,
                                                  csa_poll_device_error, csa_quantize_mxfp4,
                                                  csa_topk_select, csa_workspace_size, layer)

pytestmark = pytest.mark.gpu
U8, I32 = torch.uint8, torch.int32


# ------------------------------------------------------------------ quantizer
def _rows(n, d, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * np.exp2(rng.integers(-40, 40, (n, 1)).astype(float))
    # exact ties and saturating values
    x[::5] = np.round(x[::5] / np.abs(x[::5]).max(-1, keepdims=True) * 32) / 4
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 32), (3, 128), (333, 96), (2048, 128), (65, 512), (40, 1024),
                                 (7001, 64)])
def test_quantizer_matches_the_oracle_bit_for_bit(n, d, dtype):
    x = _rows(n, d, dtype, n + d)
    if n > 8:
        x[6] = 0
        x[7, 3] = float("nan")
        x[8, d - 1] = float("-inf")
        x[5, :32] = 1e-38                                     # near the smallest scale
        x[4, :32] = 2.0 ** -130
        x[3, :32] = 3e38
    codes = torch.empty(n, d // 2, dtype=U8, device="cuda")
    scales = torch.empty(n, d // 32, dtype=U8, device="cuda")
    values = torch.empty_like(x)
    csa_quantize_mxfp4(x, codes, scales, values=values)
    wc, ws = oracle.mxfp4_encode(x.double().cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), ws)
    np.testing.assert_array_equal(codes.cpu().numpy(), wc)
    np.testing.assert_array_equal(values.double().cpu().numpy(), oracle.mxfp4_decode(wc, ws))
    c2, s2 = layer.quantize_mxfp4(x)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    csa_poll_device_error()


def test_quantizer_writes_slots_of_a_paged_cache_from_strided_rows():
    x = _rows(50, 256, torch.bfloat16, 3)[:, 64:192]
    slots = torch.randperm(64, device="cuda")[:50].to(I32)
    slots[9] = -1
    codes = torch.full((4, 16, 64), 0xAB, dtype=U8, device="cuda")
    scales = torch.full((4, 16, 4), 0xCD, dtype=U8, device="cuda")
    csa_quantize_mxfp4(x, codes, scales, slots=slots)
    wc, ws = oracle.mxfp4_encode(x.double().cpu().numpy())
    want_c = np.full((64, 64), 0xAB, np.uint8)
    want_s = np.full((64, 4), 0xCD, np.uint8)
    s = slots.cpu().numpy()
    want_c[s[s >= 0]], want_s[s[s >= 0]] = wc[s >= 0], ws[s >= 0]
    np.testing.assert_array_equal(codes.cpu().numpy().reshape(64, 64), want_c)
    np.testing.assert_array_equal(scales.cpu().numpy().reshape(64, 4), want_s)
    csa_poll_device_error()
    slots[0], slots[1] = 64, -7
    before = codes.clone()
    csa_quantize_mxfp4(x[:2], codes, scales, slots=slots[:2].contiguous())
    with pytest.raises(CsaError) as ei:
        csa_poll_device_error()
    assert ei.value.status == 8 and torch.equal(before, codes)


# ------------------------------------------------------------------ scores
def paged(seqs, page, seed, fill):
    """Rows of every sequence (list of [n, ...] arrays) scattered into a pool
    in random page order; the rest of the pool holds `fill`, unused table
    entries a page outside it.  Returns (pool, table)."""
    rng = np.random.default_rng(seed)
    per = [-(-len(s) // page) for s in seqs]
    width, total = max(per + [1]), sum(per) + 2
    order = rng.permutation(total)
    pool = np.full((total, page) + seqs[0].shape[1:], fill, dtype=seqs[0].dtype)
    table = np.full((len(seqs), width), 2 ** 31 - 1, dtype=np.int32)
    at = 0
    for b, s in enumerate(seqs):
        for i in range(per[b]):
            part = s[i * page:(i + 1) * page]
            pool[order[at], :len(part)] = part
            table[b, i] = order[at]
            at += 1
    return pool, table


def _score_case(lens, Tq, H, D, page, seed, width=8, stride=4, integer=False):
    rng = np.random.default_rng(seed)
    n_cmp = [oracle.n_compressed(t, width, stride) for t in lens]
    B = len(lens)
    q = rng.standard_normal((B, Tq, H, D)) * np.exp2(rng.integers(-3, 3, (B, Tq, H, 1)).astype(float))
    ks = [rng.standard_normal((n, D)) * np.exp2(rng.integers(-3, 3, (n, 1)).astype(float)) for n in n_cmp]
    if integer:
        q = rng.integers(-4, 5, q.shape).astype(float)
        ks = [rng.integers(-4, 5, k.shape).astype(float) for k in ks]
    qc, qs = oracle.mxfp4_encode(q)
    kc, ksc = zip(*[oracle.mxfp4_encode(k) for k in ks])
    w = np.exp2(rng.integers(-2, 3, (B, Tq, H))).astype(np.float32) * rng.choice([-1, 1], (B, Tq, H)).astype(np.float32)
    if not integer:
        w *= rng.uniform(0.5, 1.5, w.shape).astype(np.float32)
    q_pos = np.array([[max(0, t - Tq + i) for i in range(Tq)] for t in lens], dtype=np.int32)
    kcp, table = paged(list(kc), page, seed, 0x77)
    ksp, _ = paged(list(ksc), page, seed, 0xFF)               # NaN scales behind the last key
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t = dict(q_codes=c(qc), q_scales=c(qs), w=c(w), k_codes=c(kcp), k_scales=c(ksp), page_table=c(table),
             q_pos=c(q_pos), n_cmp=c(np.array(n_cmp, dtype=np.int32)))
    qv = oracle.mxfp4_decode(qc, qs)
    want, bound = [], []
    for b in range(B):
        kv = oracle.mxfp4_decode(kc[b], ksc[b])
        want.append(oracle.index_scores(qv[b], w[b], kv))
        mag = np.matmul(np.abs(w[b]).astype(float)[:, None, :], np.matmul(np.abs(qv[b]), np.abs(kv).T))[:, 0]
        bound.append((D + 2 * H) * 2.0 ** -23 * mag)
    vis = [[oracle.n_visible(int(q_pos[b, i]), n_cmp[b], width, stride) for i in range(Tq)] for b in range(B)]
    return t, want, bound, vis


def _check_scores(p, t, want, bound, vis, n_max, exact=False):
    B, Tq = t["q_pos"].shape
    scores = torch.full((B, Tq, n_max), -123.0, device="cuda")
    csa_index_scores_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                           t["page_table"], t["q_pos"], t["n_cmp"], scores)
    torch.cuda.synchronize()
    csa_poll_device_error()
    got = scores.cpu().numpy().astype(np.float64)
    for b in range(B):
        for i in range(Tq):
            n = min(vis[b][i], n_max)
            assert np.all(got[b, i, n:] == -123.0)            # invisible entries left as they were
            err = np.abs(got[b, i, :n] - want[b][i, :n])
            if exact:
                assert np.all(err == 0)
            assert np.all(err <= bound[b][i, :n]), (b, i, float(np.nanmax(err)))
    return scores


@pytest.mark.parametrize("lens,Tq,H,D,page", [
    ([2000], 1, 64, 128, 64), ([5003, 9, 3, 4097], 1, 64, 128, 16), ([800, 515], 3, 64, 128, 8),
    ([520, 8], 8, 64, 128, 256), ([333], 333, 64, 128, 32), ([40000, 12, 33000], 1, 64, 128, 128),
    ([700], 2, 4, 32, 16), ([600, 90], 1, 5, 96, 64), ([4000], 1, 128, 128, 64), ([1000], 1, 64, 64, 64),
    ([2048], 5, 64, 128, 512), ([7], 1, 64, 128, 64),
    ([500 + 7 * (i % 90) for i in range(300)], 1, 64, 128, 64),   # more units than CTAs
    ([2600], 2600, 64, 128, 32), ([900, 40, 1500], 33, 64, 128, 64),
], ids=lambda v: str(v)[:24])
def test_index_scores(lens, Tq, H, D, page):
    p = Params(idx_heads=H, idx_dim=D)
    t, want, bound, vis = _score_case(lens, Tq, H, D, page, sum(lens) + Tq)
    _check_scores(p, t, want, bound, vis, max(1, max(len(x[0]) for x in want)))


def test_index_scores_of_whole_numbers_are_exact():
    p = Params()
    t, want, bound, vis = _score_case([9000, 1234], 2, 64, 128, 64, 11, integer=True)
    _check_scores(p, t, want, bound, vis, max(len(x[0]) for x in want), exact=True)


@pytest.mark.parametrize("lens", [[3000, 2999, 2997], [2991, 2000, 2992], [9, 8, 10], [530] * 3], ids=str)
def test_contiguous_keys_equal_paged_keys(lens):
    # the arrays' row counts leave every remainder by four, and few keys
    p = Params()
    t, want, bound, vis = _score_case(lens, 1, 64, 128, 64, 12)
    n_max = max(len(x[0]) for x in want)
    a = _check_scores(p, t, want, bound, vis, n_max)
    kc = torch.zeros(3, n_max, 64, dtype=U8, device="cuda")
    ks = torch.full((3, n_max, 4), 255, dtype=U8, device="cuda")
    for b in range(3):
        n = int(t["n_cmp"][b])
        pages = t["page_table"][b, :-(-n // 64)].long()
        kc[b, :n] = t["k_codes"][pages].flatten(0, 1)[:n]
        ks[b, :n] = t["k_scales"][pages].flatten(0, 1)[:n]
    flat = dict(t, k_codes=kc, k_scales=ks, page_table=None)
    b = _check_scores(p, flat, want, bound, vis, n_max)
    assert torch.equal(a, b)


def test_nan_keys_give_nan_scores_of_their_own():
    p = Params()
    t, want, bound, vis = _score_case([1000], 1, 64, 128, 64, 13)
    n = len(want[0][0])
    page, row = int(t["page_table"][0, 2]), 7
    t["k_scales"][page, row, 1] = 255
    scores = torch.zeros(1, 1, n, device="cuda")
    csa_index_scores_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                           t["page_table"], t["q_pos"], t["n_cmp"], scores)
    bad = torch.isnan(scores[0, 0])
    assert bad.nonzero().flatten().tolist() == [2 * 64 + row]
    ok = ~bad.cpu().numpy()
    assert np.all(np.abs(scores[0, 0].double().cpu().numpy() - want[0][0])[ok] <= bound[0][0][ok])


def test_pages_outside_the_pool_are_reported_and_skipped():
    p = Params()
    t, want, bound, vis = _score_case([2000, 2000], 1, 64, 128, 16, 14)
    n = len(want[0][0])
    t["page_table"][0, 3] = t["k_codes"].shape[0]
    t["page_table"][1, 0] = -1
    scores = torch.full((2, 1, n), -5.0, device="cuda")
    csa_index_scores_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                           t["page_table"], t["q_pos"], t["n_cmp"], scores)
    with pytest.raises(CsaError) as ei:
        csa_poll_device_error()
    assert ei.value.status == 8
    got = scores.double().cpu().numpy()
    skip = [slice(48, 64), slice(0, 16)]
    for b in range(2):
        assert np.all(got[b, 0, skip[b]] == -5.0)
        keep = np.ones(n, bool)
        keep[skip[b]] = False
        assert np.all(np.abs(got[b, 0] - want[b][0])[keep] <= bound[b][0][keep])


@pytest.mark.parametrize("lens,topk", [([9000, 700, 40], 64), ([70000] * 2, 1024)])
def test_topk_is_the_selection_on_the_scores(lens, topk):
    p = Params(topk=topk)
    t, want, bound, vis = _score_case(lens, 1, 64, 128, 64, 15)
    n_max = max(len(x[0]) for x in want)
    scores = _check_scores(p, t, want, bound, vis, n_max)
    B = len(lens)
    nb = csa_workspace_size(p, CSA_OP_INDEX_TOPK, B, 1, n_max)
    ws = torch.empty(nb + 256, dtype=U8, device="cuda")
    idx = torch.empty(B, 1, topk, dtype=I32, device="cuda")
    csa_index_topk_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                         t["page_table"], t["q_pos"], t["n_cmp"], idx, ws, n_max)
    again = torch.empty_like(idx)
    csa_topk_select(p, scores, t["q_pos"], t["n_cmp"], again, ws)
    assert torch.equal(idx, again)
    csa_poll_device_error()


def test_scores_repeat_on_another_stream_and_from_a_graph():
    p = Params()
    t, want, bound, vis = _score_case([9000, 5000], 1, 64, 128, 64, 16)
    n = max(len(x[0]) for x in want)
    first = _check_scores(p, t, want, bound, vis, n)
    call = lambda out: csa_index_scores_mxfp4(  # noqa: E731
        p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"], t["page_table"], t["q_pos"],
        t["n_cmp"], out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = torch.full_like(first, -123.0)
        call(a)
    side.synchronize()
    assert torch.equal(a, first)
    b = torch.full_like(first, -123.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(b)
    for _ in range(3):
        b.fill_(-123.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b, first)


def test_rows_past_four_gigabytes():
    # codes of a pool of 80M keys (5.1 GB): the last rows
    rows = 80_000_000
    codes = torch.empty(rows, 64, dtype=U8, device="cuda")
    scales = torch.empty(rows, 4, dtype=U8, device="cuda")
    x = _rows(128, 128, torch.bfloat16, 17)
    slots = (rows - 1 - torch.arange(128, device="cuda")).to(I32)
    csa_quantize_mxfp4(x, codes, scales, slots=slots)
    wc, ws = oracle.mxfp4_encode(x.double().cpu().numpy())
    np.testing.assert_array_equal(codes[-128:].flip(0).cpu().numpy(), wc)
    # and scores of keys there, in pages of 128
    p = Params()
    table = torch.tensor([[rows // 128 - 1]], dtype=I32, device="cuda")
    t, want, bound, vis = _score_case([4 * 128 + 4], 1, 64, 128, 128, 18)
    codes.view(-1, 128, 64)[-1] = t["k_codes"][t["page_table"][0, 0].long()]
    scales.view(-1, 128, 4)[-1] = t["k_scales"][t["page_table"][0, 0].long()]
    far = dict(t, k_codes=codes.view(-1, 128, 64), k_scales=scales.view(-1, 128, 4), page_table=table)
    _check_scores(p, far, want, bound, vis, 128)


def test_scores_with_no_keys():
    p = Params()
    t, _, _, _ = _score_case([40, 40], 1, 64, 128, 64, 19)
    scores = torch.full((2, 1, 16), 5.0, device="cuda")
    none = dict(t, n_cmp=torch.tensor([-2, 0], dtype=I32, device="cuda"))
    csa_index_scores_mxfp4(p, none["q_codes"], none["q_scales"], none["w"], none["k_codes"], none["k_scales"],
                           none["page_table"], none["q_pos"], none["n_cmp"], scores)
    assert torch.all(scores == 5.0)
    csa_index_scores_mxfp4(p, t["q_codes"], t["q_scales"], t["w"], t["k_codes"], t["k_scales"],
                           t["page_table"], t["q_pos"], t["n_cmp"], torch.empty(2, 1, 0, device="cuda"))
    csa_poll_device_error()


@pytest.mark.parametrize("B", [147, 149, 513])
def test_batches_around_the_number_of_sms_and_the_plan(B):
    p = Params()
    lens = [40 + 37 * (i % 29) for i in range(B)]
    t, want, bound, vis = _score_case(lens, 1, 64, 128, 64, B)
    _check_scores(p, t, want, bound, vis, max(len(x[0]) for x in want))
