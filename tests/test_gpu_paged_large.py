"""The variants of the quantizer and the norm that only large calls take, and
the way of new entries from the compressor into pages."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_close, host64
from sparse_compressed_attention_csa_b200 import (Params, csa_compress, csa_index_topk_mxfp4,
                                                  csa_poll_device_error, csa_quantize_mxfp4, layer)
from test_gpu_mxfp4 import _rows
from test_gpu_norm_rope import _case, _close

pytestmark = pytest.mark.gpu
U8, I32 = torch.uint8, torch.int32


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantizer_with_two_chunks_a_thread(dtype):
    # from 4 * 2048 chunks of 8 values an SM on; the last block half full
    d = 128
    n = 4 * _sms() * 2048 * 8 // d + 225
    assert n * d // 8 % 512 not in (0, 256)
    x = _rows(n, d, dtype, 3)
    x[7, 3], x[n - 1, d - 1], x[8] = float("nan"), float("-inf"), 0
    slots = torch.randperm(n + 100, device="cuda")[:n].to(I32)
    slots[5::1000] = -1
    codes = torch.full((n + 100, d // 2), 0xAB, dtype=U8, device="cuda")
    scales = torch.full((n + 100, d // 32), 0xCD, dtype=U8, device="cuda")
    values = torch.empty_like(x)
    csa_quantize_mxfp4(x, codes, scales, slots=slots, values=values)
    csa_poll_device_error()
    wc, ws = oracle.mxfp4_encode(x.double().cpu().numpy())
    s = slots.cpu().numpy()
    want_c, want_s = np.full((n + 100, d // 2), 0xAB, np.uint8), np.full((n + 100, d // 32), 0xCD, np.uint8)
    want_c[s[s >= 0]], want_s[s[s >= 0]] = wc[s >= 0], ws[s >= 0]
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(values.double().cpu().numpy(), oracle.mxfp4_decode(wc, ws))


@pytest.mark.parametrize("dtype,heads,dim", [
    (torch.bfloat16, 100, 512), (torch.bfloat16, 70, 128), (torch.bfloat16, 100, 96), (torch.float32, 100, 128),
    (torch.float32, 70, 256),
])
def test_norm_with_many_heads_a_lane_group(dtype, heads, dim):
    rows = 8200
    # heads per group: doubled while 2 h <= heads and the groups fill the GPU 16 times
    lanes, per = 1, 128 // torch.finfo(dtype).bits
    while lanes < dim // per and lanes < 32:
        lanes *= 2
    h = 1
    while h < 32 and 2 * h <= heads and rows * heads // (2 * h) >= 16 * _sms() * (256 // lanes):
        h *= 2
    assert h > 4 and heads % h
    p = Params(d=1024, rope_dim=64)
    x, w, pos = _case(rows, heads, dim, dtype, heads + dim)
    out, _ = layer.norm_rope(p, x, w, pos)
    some = torch.cat([torch.arange(8), torch.randint(0, rows, (40,)), torch.arange(rows - 8, rows)]).cuda()
    _close(out[some], x[some], w, pos[some], p, 1e-6)
    assert torch.isfinite(out).all()
    csa_poll_device_error()


def test_an_empty_page_table_selects_nothing():
    p = Params(topk=4)
    z = lambda *s: torch.zeros(s, dtype=U8, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=I32, device="cuda")  # noqa: E731
    idx = i(3, 1, 4) + 9
    csa_index_topk_mxfp4(p, z(3, 1, 64, 64), z(3, 1, 64, 4), torch.zeros(3, 1, 64, device="cuda"), z(3, 16, 64),
                         z(3, 16, 4), i(3, 0), i(3, 1) + 100, i(3) + 20, idx, None)
    torch.cuda.synchronize()
    csa_poll_device_error()
    assert torch.all(idx == -1)


def test_from_the_compressor_into_pages():
    """Tokens are pooled without rotation (the compressor with rope_dim 0), the
    pooled rows normed and rotated into their pages, at first for a whole
    prompt and then for the entry that four more tokens complete; each step
    against the oracle on what the step before it gave."""
    rng = np.random.default_rng(31)
    B, T, page, topk = 2, 724, 16, 64
    bf = torch.bfloat16
    p = Params(topk=topk)
    bare, bare_i = Params(rope_dim=0), Params(d=128, rope_dim=0)
    val = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(bf)  # noqa: E731
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    f = lambda a: a.double().cpu().numpy()  # noqa: E731
    x, gate, xi, gate_i = val(B, T, 512), val(B, T, 512), val(B, T, 128), val(B, T, 128)
    kw, kiw = 1 + 0.1 * torch.randn(512, device="cuda"), 1 + 0.1 * torch.randn(128, device="cuda")
    n_all = oracle.n_compressed(T, 8, 4)
    width = -(-n_all // page)
    table = rng.permutation(B * width + 3)[:B * width].reshape(B, width).astype(np.int32)
    kv = torch.full((B * width + 3, page, 512), float("nan"), dtype=bf, device="cuda")
    codes = torch.zeros(B * width + 3, page, 64, dtype=U8, device="cuda")
    scales = torch.full((B * width + 3, page, 4), 255, dtype=U8, device="cuda")

    def add(t0, t1, j0):
        """Entries j0 .. of the tokens t0 .. t1 - 1 (t0 = 4 j0), both caches."""
        n = oracle.n_compressed(t1 - t0, 8, 4)
        j = j0 + np.arange(n)
        slots = c(np.stack([table[b][j // page] * page + j % page for b in range(B)]).ravel())
        pos = c(np.tile(4 * j, B))
        for pb, src, g, wt, dim in ((bare, x, gate, kw, 512), (bare_i, xi, gate_i, kiw, 128)):
            src, g = src[:, t0:t1].contiguous(), g[:, t0:t1].contiguous()
            pooled = torch.empty(B, n, dim, dtype=bf, device="cuda")
            csa_compress(pb, src, g, pooled)
            for b in range(B):
                assert_close(host64(pooled[b]), oracle.compress(f(src[b]), f(g[b]), 8, 4, 0, 1e4), "bf16", "pooled")
            rows = pooled.view(B * n, 1, dim)
            want = oracle.norm_rope(f(rows), wt.cpu().numpy(), np.tile(4 * j, B), 64, 1e4, 1e-6)[:, 0]
            if dim == 512:
                layer.norm_rope(p, rows, k=rows, k_weight=wt, k_pos=pos, k_out=kv.view(-1, 1, 512), k_slots=slots)
                assert_close(f(kv.view(-1, 512)[slots.long()]), want, "bf16", "entries")
            else:
                normed, _ = layer.norm_rope(p, rows, wt, pos)
                csa_quantize_mxfp4(normed[:, 0], codes, scales, slots=slots)
                wc, ws = oracle.mxfp4_encode(f(normed[:, 0]))
                np.testing.assert_array_equal(codes.view(-1, 64)[slots.long()].cpu().numpy(), wc)
                np.testing.assert_array_equal(scales.view(-1, 4)[slots.long()].cpu().numpy(), ws)
                assert_close(f(normed[:, 0]), want, "bf16", "keys")
        return j0 + n

    j = add(0, T - 4, 0)
    assert add(4 * j, T, j) == n_all == j + 1
    # the window's rows: the last tokens' own, normed and rotated as well
    last = x[:, T - 128:].reshape(-1, 1, 512)
    raw, _ = layer.norm_rope(p, last, kw, c(np.tile(np.arange(T - 128, T), B)))
    raw = raw.view(B, 128, 512)
    q, q_idx, w = val(B, 1, 128, 512), val(B, 1, 64, 128), torch.rand(B, 1, 64, device="cuda")
    sink, n_cmp, q_pos = torch.randn(128, device="cuda"), c([n_all] * B), c([[T - 1]] * B)
    idx, out = layer.csa_decode_paged(p, q, q_pos, q_idx, w, codes, scales, n_cmp, kv, c(table), raw, c([T - 128] * B),
                                      c([128] * B), sink)
    torch.cuda.synchronize()
    csa_poll_device_error()
    for b in range(B):
        got = idx[b, 0].cpu().numpy()
        keys = oracle.mxfp4_decode(oracle.paged_rows(codes.cpu().numpy(), table[b], n_all),
                                   oracle.paged_rows(scales.cpu().numpy(), table[b], n_all))
        s = oracle.index_scores(oracle.mxfp4_decode(*oracle.mxfp4_encode(f(q_idx[b]))), w[b].cpu().numpy(), keys)[0]
        assert len(got) == topk and np.all(np.diff(got) > 0)
        assert np.all(s[got] >= np.sort(s)[-topk] - 1e-4 * np.abs(s).max())
        want = oracle.sparse_attn(f(q[b]), [T - 1], oracle.paged_rows(f(kv), table[b], n_all), idx[b].cpu().numpy(),
                                  f(raw[b]), T - 128, 128, sink.cpu().numpy(), 1 / np.sqrt(512), 128, 64, 1e4)
        assert_close(host64(out[b]), want, "bf16", "decode")
