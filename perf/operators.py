"""Operators of the paged, 4-bit serving path of the sparse-attention layer:
what a pass through each of them is, in plain torch (`own` false) and through
the library's calls (`own` true).

  norm_rope       RMS norm of every query and key head with the partial RoPE
                  in the same pass; key rows go to the rows of a paged cache
                  that a slot list names
  quantize_mxfp4  rows to microscaled 4-bit floats: E2M1 codes and one E8M0
                  scale per 32 values, written to the rows of a paged cache,
                  and the values that the codes stand for
  index_scores    the lightning indexer's product on such 4-bit queries and
                  paged keys: sum_h w_h max(0, q_h . k_j) of every visible key
  sparse_paged    shared-KV attention of new tokens over the selected entries
                  of a paged cache and a window of raw rows
  hca_paged       the same over every visible entry, split over the cache's
                  length and joined
"""
import math

import torch

own = False

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _norm(name, rows, heads, k_rows, k_heads, dim, rope, dtype, max_pos, fused):
    return dict(name=name, op="norm_rope", rows=rows, heads=heads, k_rows=k_rows, k_heads=k_heads,
                dim=dim, rope=rope, dtype=dtype, max_pos=max_pos, fused=fused)


def _quant(name, n, d, cap, dtype):
    return dict(name=name, op="quantize_mxfp4", n=n, d=d, cap=cap, dtype=dtype)


def _index(name, B, Tq, T, width, stride, heads, dim, page, ragged):
    return dict(name=name, op="index_scores", B=B, Tq=Tq, T=T, width=width, stride=stride,
                heads=heads, dim=dim, page=page, ragged=ragged)


def _sparse(name, B, Tq, T, topk, window, page, ragged, heads=128, d=512, rope=64, dtype="bf16"):
    return dict(name=name, op="sparse_paged", B=B, Tq=Tq, T=T, width=8, stride=4, topk=topk,
                window=window, page=page, ragged=ragged, heads=heads, d=d, rope=rope, dtype=dtype)


def _hca(name, B, Tq, T, width, stride, window, page, ragged, heads=128, d=512, rope=64,
         dtype="bf16"):
    return dict(name=name, op="hca_paged", B=B, Tq=Tq, T=T, width=width, stride=stride,
                window=window, page=page, ragged=ragged, heads=heads, d=d, rope=rope, dtype=dtype)


def listed():
    return [
        # a decode step's indexer heads: 32 sequences, 64 query heads and one new key each
        _norm("norm_rope_decode_idx", 32, 64, 32, 1, 128, 64, "bf16", 1 << 20, False),
        # a prefill of 8,192 tokens: 128 query heads and the shared KV row of a fused projection
        _norm("norm_rope_prefill", 8192, 128, 8192, 1, 512, 64, "bf16", 8192, True),
        # fp32 with odd sizes
        _norm("norm_rope_f32_odd", 1237, 5, 311, 3, 96, 32, "f32", 65536, False),
        # a decode step's indexer queries: 32 x 64 heads x 128 dims
        _quant("quantize_decode_queries", 2048, 128, 2048, "bf16"),
        # the key cache of 32 sequences at 64K context, quantized whole
        _quant("quantize_key_cache", 32 * 16383, 128, 32 * 16384, "bf16"),
        # one new token of 32 sequences at 64K context
        _index("index_decode_64k", 32, 1, 65536, 8, 4, 64, 128, 64, False),
        # one new token of 4 sequences of up to 1M context, ragged
        _index("index_decode_1m_ragged", 4, 1, 1048576, 8, 4, 64, 128, 256, True),
        # every token of an 8,192-token prefill
        _index("index_prefill_8k", 1, 8192, 8192, 8, 4, 64, 128, 128, False),
        # top-1,024 of 16,383 entries, 32 sequences
        _sparse("sparse_decode_64k", 32, 1, 65536, 1024, 128, 64, False),
        # a few short ragged sequences, two tokens each, fewer entries than k
        _sparse("sparse_short_ragged", 3, 2, 5003, 1024, 128, 16, True),
        # HCA decode at 128K context, batch 16: 1,024 entries and the window
        _hca("hca_decode_128k", 16, 1, 131072, 128, 128, 128, 64, False),
        # every token its own entry: one new token of 8 ragged sequences of up to 64K tokens
        _hca("hca_dense_64k_ragged", 8, 1, 65536, 1, 1, 0, 64, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "quantize_mxfp4", "index_scores", "index_scores", "sparse_paged",
                     "hca_paged", "hca_paged"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "norm_rope":
        dim = rng.choice([64, 96, 128, 256, 512])
        heads = rng.choice([1, 5, 16, 64, 128])
        rows = _log(rng, 1, max(2, (1 << 28) // (dim * heads)) if dim * heads > 32768 else 8192)
        fused = rng.random() < 0.5
        c = _norm("", rows, heads, rows if fused else _log(rng, 1, 4096), rng.choice([1, 2, 3]),
                  dim, rng.choice([0, 32, 64]), rng.choice(["bf16", "bf16", "f32"]),
                  _log(rng, 128, 1 << 20), fused)
    elif op == "quantize_mxfp4":
        d = rng.choice([32, 64, 96, 128, 512])
        n = _log(rng, 1, 50_000_000 // d)
        c = _quant("", n, d, n + rng.randrange(0, 4096), rng.choice(["bf16", "bf16", "f32"]))
    elif op == "index_scores":
        if rng.random() < 0.3:
            T = _log(rng, 64, 6144)
            c = _index("", 1, T, T, 8, 4, 64, 128, page, False)
        else:
            B = _log(rng, 1, 40)
            c = _index("", B, rng.choice([1, 1, 1, 2, 3]), _log(rng, 64, (1 << 20) // B), 8, 4, 64,
                       128, page, rng.random() < 0.5)
    elif op == "sparse_paged":
        B = _log(rng, 1, 48)
        c = _sparse("", B, rng.choice([1, 1, 2, 3]), _log(rng, 64, (1 << 21) // B), rng.choice([64, 512, 1024]),
                    rng.choice([16, 128]), page, rng.random() < 0.5)
    else:
        B = _log(rng, 1, 24)
        if rng.random() < 0.2:  # fp32, small heads
            c = _hca("", B, rng.choice([1, 2]), _log(rng, 16, 4096), 4, 4, 16, page, True,
                     heads=rng.choice([1, 3, 8]), d=rng.choice([64, 128]), rope=32, dtype="f32")
        else:
            w = rng.choice([1, 4, 128])
            c = _hca("", B, rng.choice([1, 1, 2]), _log(rng, 64, min(262144, (400_000 // B) * w)), w, w,
                     rng.choice([0, 128]), page, rng.random() < 0.6,
                     heads=rng.choice([16, 32, 64, 128, 128]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _entries(T, c):
    return 0 if T < c["width"] else (T - c["width"]) // c["stride"] + 1


def _lengths(c, gen):
    """Context length of every sequence: all T, or spread from about T / 16 to T."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    u = torch.rand(c["B"], generator=gen, dtype=torch.float64).tolist()
    lens = [max(c["Tq"], int(c["T"] * 16.0 ** (x - 1.0))) for x in u]
    lens[0] = c["T"]
    return lens


def _pages(c, lens, gen, dev):
    """A page table over a pool in random order, every sequence holding its own pages."""
    per = [-(-max(1, _entries(t, c)) // c["page"]) for t in lens]
    width, total = max(per), sum(per)
    order = torch.randperm(total, generator=gen).tolist()
    table = torch.full((c["B"], width), 0, dtype=I32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=I32)
        at += n
    return table.to(dev), total


def _randn(gen, shape, dev, dtype):
    return torch.randn(shape, generator=gen, device=dev, dtype=F32).to(dtype)


def _pow2(e, dtype):
    """2^e of whole e in [-127, 127], exactly."""
    lo = torch.div(e, 2, rounding_mode="floor")
    bits = lambda n: ((n.to(I32) + 127) << 23).view(F32)  # noqa: E731
    return bits(lo).to(dtype) * bits(e - lo).to(dtype)


def _mx_encode(x):
    """E2M1 codes (0..15) and E8M0 exponents of x [..., d]: blocks of 32 values share the scale
    2^(floor(log2 max|x|) - 2); nearest code, ties to the even one, values past 6 at 6."""
    blocks = x.to(F32).unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.zeros_like(amax, dtype=I32)).clamp(-127, 127)
    a = blocks.abs() * _pow2(-e, F32)[..., None]
    code = ((a > 0.25).to(U8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    code = code + 8 * torch.signbit(blocks).to(U8)
    return code.flatten(-2), (e + 127).to(U8)


def _mx_pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _mx_values(codes, scales, dtype):
    """The values of packed codes [..., d/2] under scales [..., d/32]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device, dtype=dtype)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    s = _pow2(scales.to(I32) - 127, dtype)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm_rope":
        dt = BF16 if c["dtype"] == "bf16" else F32
        hq, hk, dim = c["heads"], c["k_heads"], c["dim"]
        if c["fused"]:  # queries and keys side by side in the rows of one projection
            both = 3.0 * torch.randn((c["rows"], (hq + hk) * dim), generator=g, device=dev, dtype=dt)
            s["q"] = both[:, :hq * dim].unflatten(-1, (hq, dim))
            s["k"] = both[:, hq * dim:].unflatten(-1, (hk, dim))
        else:
            s["q"] = 3.0 * torch.randn((c["rows"], hq, dim), generator=g, device=dev, dtype=dt)
            s["k"] = 3.0 * torch.randn((c["k_rows"], hk, dim), generator=g, device=dev, dtype=dt)
        s["q_weight"] = 1.0 + 0.2 * torch.randn(dim, generator=g, device=dev)
        s["k_weight"] = 1.0 + 0.2 * torch.randn(dim, generator=g, device=dev)
        pos = lambda n: torch.randint(0, c["max_pos"], (n,), generator=g, device=dev, dtype=I32)  # noqa: E731
        s["q_pos"], s["k_pos"] = pos(c["rows"]), pos(c["k_rows"])
        cap = -(-c["k_rows"] // 64) * 64
        s["slots"] = torch.randperm(cap, generator=g, device=dev)[:c["k_rows"]].to(I32)
        s["k_cache"] = torch.zeros((cap, hk, dim), device=dev, dtype=dt)
        s["q_out"] = torch.empty((c["rows"], hq, dim), device=dev, dtype=dt)
        return s
    if c["op"] == "quantize_mxfp4":
        dt = BF16 if c["dtype"] == "bf16" else F32
        # rows of different sizes, as heads have them
        size = torch.exp2(torch.randint(-3, 4, (c["n"], 1), generator=g, device=dev).to(F32))
        s["rows"] = (torch.randn((c["n"], c["d"]), generator=g, device=dev) * size).to(dt)
        s["slots"] = torch.randperm(c["cap"], generator=g, device=dev)[:c["n"]].to(I32)
        s["codes"] = torch.zeros((c["cap"], c["d"] // 2), device=dev, dtype=U8)
        s["scales"] = torch.zeros((c["cap"], c["d"] // 32), device=dev, dtype=U8)
        s["values"] = torch.empty((c["n"], c["d"]), device=dev, dtype=dt)
        return s
    lens = _lengths(c, gc)
    s["table"], n_pages = _pages(c, lens, gc, dev)
    s["n_cmp"] = torch.tensor([_entries(t, c) for t in lens], dtype=I32, device=dev)
    s["n_max"] = s["table"].shape[1] * c["page"]
    s["q_pos"] = torch.tensor([[t - c["Tq"] + i for i in range(c["Tq"])] for t in lens], dtype=I32,
                              device=dev)
    if c["op"] == "index_scores":
        H, D = c["heads"], c["dim"]
        pack = lambda x: (lambda e: (_mx_pack(e[0]), e[1]))(_mx_encode(x))  # noqa: E731
        s["q_codes"], s["q_scales"] = pack(torch.randn((c["B"], c["Tq"], H, D), generator=g, device=dev))
        s["k_codes"], s["k_scales"] = pack(torch.randn((n_pages, c["page"], D), generator=g, device=dev))
        s["w"] = torch.rand((c["B"], c["Tq"], H), generator=g, device=dev) / math.sqrt(H * D)
        s["n_max"] = int(max(s["n_cmp"].tolist() + [1]))
        s["scores"] = torch.zeros((c["B"], c["Tq"], s["n_max"]), device=dev)
        return s
    dt = BF16 if c["dtype"] == "bf16" else F32
    d = c["d"]
    s["q"] = _randn(g, (c["B"], c["Tq"], c["heads"], d), dev, dt)
    s["kv"] = _randn(g, (n_pages, c["page"], d), dev, dt)
    raw_max = max(1, c["window"] + c["Tq"])
    s["kv_raw"] = _randn(g, (c["B"], raw_max, d), dev, dt)
    s["raw_pos0"] = torch.tensor([max(0, t - raw_max) for t in lens], dtype=I32, device=dev)
    s["n_raw"] = torch.tensor([min(t, raw_max) for t in lens], dtype=I32, device=dev)
    s["sink"] = torch.randn(c["heads"], generator=g, device=dev)
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "sparse_paged":
        rows = []
        for b, t in enumerate(lens):
            for i in range(c["Tq"]):
                n = min(_entries(t - c["Tq"] + i + 1, c), _entries(t, c))
                k = min(n, c["topk"])
                pick = torch.randperm(n, generator=gc)[:k].sort()[0] if n else torch.empty(0)
                rows.append(torch.cat((pick.to(I32), torch.full((c["topk"] - k,), -1, dtype=I32))))
        s["idx"] = torch.stack(rows).view(c["B"], c["Tq"], c["topk"]).to(dev)
    return s


# ------------------------------------------------------------------ the plain forms
def _cos_sin(pos, rope):
    """cos and sin of pos * 10000^(-2i/rope), angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rope, 2, device=pos.device, dtype=torch.float64) / rope)
    a = pos.to(torch.float64)[..., None] * f
    return a.cos().to(F32), a.sin().to(F32)


def _rotate(x, cos, sin):
    """The last 2 * cos.shape[-1] dims of x, in interleaved pairs, rotated."""
    r = 2 * cos.shape[-1]
    if r == 0:
        return x
    head, tail = x[..., :x.shape[-1] - r], x[..., x.shape[-1] - r:]
    a, b = tail[..., 0::2], tail[..., 1::2]
    return torch.cat((head, torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)), -1)


def _norm_rotate(x, weight, pos, rope):
    v = x.to(F32)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * weight
    cos, sin = _cos_sin(pos, rope)
    return _rotate(v, cos[:, None], sin[:, None])


def _visible(s):
    """[B, Tq]: entries that each query sees."""
    c = s["case"]
    n = torch.div(s["q_pos"] - (c["width"] - 1), c["stride"], rounding_mode="floor") + 1
    return torch.minimum(n.clamp(min=0), s["n_cmp"][:, None])


def _attend(s, rows, valid):
    """rows [B, n, d] or [B, Tq, n, d], valid [B, Tq, n]: attention with the window and the sink."""
    c = s["case"]
    cos, sin = _cos_sin(s["q_pos"], c["rope"])
    q = _rotate(s["q"].to(F32), cos[:, :, None], sin[:, :, None])
    shared = rows.dim() == 3
    raw = s["kv_raw"].to(F32)
    p = s["raw_pos0"][:, None] + torch.arange(raw.shape[1], device=raw.device)
    t = s["q_pos"][:, :, None]
    win = (p[:, None] <= t) & (p[:, None] > t - c["window"]) & (p < (s["raw_pos0"] + s["n_raw"])[:, None])[:, None]
    scale = 1.0 / math.sqrt(c["d"])
    z = torch.matmul(q.flatten(1, 2), rows.transpose(1, 2)).unflatten(1, q.shape[1:3]) if shared else torch.matmul(q, rows.transpose(2, 3))
    zw = torch.matmul(q.flatten(1, 2), raw.transpose(1, 2)).unflatten(1, q.shape[1:3])
    z = (z * scale).masked_fill(~valid[:, :, None], -math.inf)
    zw = (zw * scale).masked_fill(~win[:, :, None], -math.inf)
    sink = s["sink"][None, None, :, None]
    m = torch.maximum(torch.maximum(z.amax(-1, keepdim=True) if z.shape[-1] else sink, zw.amax(-1, keepdim=True)), sink)
    e, ew = torch.exp(z - m), torch.exp(zw - m)
    den = e.sum(-1, keepdim=True) + ew.sum(-1, keepdim=True) + torch.exp(sink - m)
    o = torch.matmul(e.flatten(1, 2), rows).unflatten(1, q.shape[1:3]) if shared else torch.matmul(e, rows)
    o = (o + torch.matmul(ew.flatten(1, 2), raw).unflatten(1, q.shape[1:3])) / den
    return _rotate(o, cos[:, :, None], -sin[:, :, None]).to(s["q"].dtype)


def _paged(cache, table):
    """[B, n_max, ...]: the rows of every sequence in order."""
    return cache[table.long()].flatten(1, 2)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm_rope":
        q = _norm_rotate(s["q"], s["q_weight"], s["q_pos"], c["rope"])
        k = _norm_rotate(s["k"], s["k_weight"], s["k_pos"], c["rope"])
        cache = s["k_cache"].clone()
        cache[s["slots"].long()] = k.to(cache.dtype)
        return q.to(s["q"].dtype), cache
    if c["op"] == "quantize_mxfp4":
        code, scale = _mx_encode(s["rows"])
        codes, scales = s["codes"].clone(), s["scales"].clone()
        codes[s["slots"].long()] = _mx_pack(code)
        scales[s["slots"].long()] = scale
        return _mx_values(codes[s["slots"].long()], scales[s["slots"].long()], F32).to(s["rows"].dtype)
    if c["op"] == "index_scores":
        q = _mx_values(s["q_codes"], s["q_scales"], F32)
        k = _paged(_mx_values(s["k_codes"], s["k_scales"], F32), s["table"])[:, :s["n_max"]]
        z = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).clamp_(min=0).unflatten(1, q.shape[1:3])
        score = torch.matmul(s["w"][:, :, None], z)[:, :, 0]
        seen = torch.arange(s["n_max"], device=q.device) < _visible(s)[:, :, None]
        return torch.where(seen, score, s["scores"])
    if c["op"] == "sparse_paged":
        idx = s["idx"].long()
        j = idx.clamp(min=0)
        b = torch.arange(c["B"], device=j.device)[:, None, None]
        page = s["table"].long()[b, j // c["page"]]
        rows = s["kv"].flatten(0, 1)[page * c["page"] + j % c["page"]].to(F32)
        return _attend(s, rows, idx >= 0)
    rows = _paged(s["kv"], s["table"])[:, :max(1, int(s["n_max"]))].to(F32)
    seen = torch.arange(rows.shape[1], device=rows.device) < _visible(s)[:, :, None]
    return _attend(s, rows, seen)


# ------------------------------------------------------------------ the library's calls
def _handles(s):
    """What a program sets up once: the layer's constants and a workspace."""
    from sparse_compressed_attention_csa_b200 import Params, layer
    c = s["case"]
    if "params" not in s:
        get = c.get
        s["params"] = Params(d=get("d", 512), rope_dim=get("rope", 64), n_heads=get("heads", 128) if "d" in c else 128,
                             idx_heads=get("heads", 64) if c["op"] == "index_scores" else 64,
                             idx_dim=get("dim", 128) if c["op"] == "index_scores" else 128,
                             topk=get("topk", 1024), window=get("window", 128), width=get("width", 8),
                             stride=get("stride", 4))
        s["ws"] = layer.Workspace("cuda")
    return layer, s["params"]


def _library(s):
    import sparse_compressed_attention_csa_b200 as csa
    layer, p = _handles(s)
    op = s["case"]["op"]
    if op == "norm_rope":
        csa.csa_norm_rope(p, EPS, s["q"], s["q_weight"], s["q_pos"], s["q_out"], s["k"], s["k_weight"],
                          s["k_pos"], s["k_cache"], s["slots"])
        return s["q_out"], s["k_cache"]
    if op == "quantize_mxfp4":
        csa.csa_quantize_mxfp4(s["rows"], s["codes"], s["scales"], slots=s["slots"], values=s["values"])
        return s["values"]
    if op == "index_scores":
        csa.csa_index_scores_mxfp4(p, s["q_codes"], s["q_scales"], s["w"], s["k_codes"], s["k_scales"],
                                   s["table"], s["q_pos"], s["n_cmp"], s["scores"])
        return s["scores"]
    if op == "sparse_paged":
        return layer.sparse_attn_paged(p, s["q"], s["q_pos"], s["kv"], s["table"], s["idx"], s["kv_raw"],
                                       s["raw_pos0"], s["n_raw"], s["sink"], s["ws"], s["out"])
    return layer.hca_decode_paged(p, s["q"], s["q_pos"], s["kv"], s["table"], s["n_cmp"], s["kv_raw"],
                                  s["raw_pos0"], s["n_raw"], s["sink"], s["ws"], s["out"])


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def _seen_counts(c):
    """Entries seen by each query and window rows of it, from the sizes alone (ragged batches:
    the lengths' mean)."""
    if c["ragged"]:
        mean = (c["T"] + (c["B"] - 1) * c["T"] * (1 - 1 / 16) / math.log(16)) / c["B"]
    else:
        mean = c["T"]
    if c["Tq"] >= mean:  # a causal prefill
        n = sum(max(0, (t - c["width"] + 1) // c["stride"] + 1) if t >= c["width"] - 1 else 0
                for t in range(c["Tq"])) / c["Tq"]
    else:
        n = max(0.0, (mean - c["width"]) / c["stride"] + 1)
    return n, mean


def work(case):
    c = case
    if c["op"] == "norm_rope":
        e = 2 if c["dtype"] == "bf16" else 4
        n = (c["rows"] * c["heads"] + c["k_rows"] * c["k_heads"]) * c["dim"]
        return {"bytes": 2 * n * e + 8 * c["dim"] + 4 * c["rows"] + 8 * c["k_rows"], "flops": 5 * n}
    if c["op"] == "quantize_mxfp4":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["n"] * c["d"]
        return {"bytes": n * (2 * e) + n // 2 + n // 32 + 4 * c["n"], "flops": 3 * n}
    n, mean = _seen_counts(c)
    q = c["B"] * c["Tq"]
    if c["op"] == "index_scores":
        keys = c["B"] * max(0.0, (mean - c["width"]) / c["stride"] + 1)
        D = c["dim"]
        by = keys * (D / 2 + D / 32 + 4 / c["page"]) + q * c["heads"] * (D / 2 + D / 32 + 4) + 4 * q * n
        return {"bytes": int(by), "flops": int(q * n * c["heads"] * (2 * D + 2))}
    e = 2 if c["dtype"] == "bf16" else 4
    d, H = c["d"], c["heads"]
    win = min(mean, c["window"])
    io = 2 * q * H * d * e + 4 * H
    if c["op"] == "sparse_paged":
        rows = q * (min(n, c["topk"]) + win)
        return {"bytes": int(rows * d * e + io + 4 * q * c["topk"]), "flops": int(4 * rows * H * d)}
    return {"bytes": int(c["B"] * (n + win) * d * e + io), "flops": int(4 * q * (n + win) * H * d)}


# ------------------------------------------------------------------ 64 bits
def _x_rope(x, pos, rope):
    """x [..., h, d] at pos [...]: the trailing dims as complex numbers times e^(i pos f)."""
    if rope == 0:
        return x
    f = torch.exp(torch.arange(rope // 2, device=x.device, dtype=torch.float64) * (-2.0 * math.log(10000.0) / rope))
    turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64), pos.double().unsqueeze(-1) * f).unsqueeze(-2)
    z = torch.view_as_complex(x[..., -rope:].reshape(x.shape[:-1] + (rope // 2, 2)).contiguous())
    return torch.cat((x[..., :-rope], torch.view_as_real(z * turn).reshape(x.shape[:-1] + (rope,))), -1)


def _x_e2m1(codes, scales):
    """Packed codes to values by their bits: sign, two exponent bits (bias 1), one mantissa bit."""
    c = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), device=codes.device, dtype=torch.int64)
    c[..., 0::2] = codes.long() % 16
    c[..., 1::2] = codes.long() // 16
    e, m = (c // 2) % 4, (c % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).double()) * (1 - 2 * (c // 8)).double()
    return v * (2.0 ** (scales.double() - 127)).repeat_interleave(32, -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm_rope":
        def one(x, w, pos):
            y = x.double()
            y = y / torch.sqrt(torch.einsum("rhd,rhd->rh", y, y) / c["dim"] + EPS)[..., None] * w.double()
            return _x_rope(y, pos, c["rope"])
        cache = s["k_cache"].double()
        cache.index_copy_(0, s["slots"].long(), one(s["k"], s["k_weight"], s["k_pos"]))
        return one(s["q"], s["q_weight"], s["q_pos"]), cache
    if c["op"] == "quantize_mxfp4":
        x = s["rows"].double().reshape(c["n"], c["d"] // 32, 32)
        power = torch.frexp(x.abs().max(-1, keepdim=True)[0])[1].double() - 3
        unit = torch.exp2(power)
        y = (x / unit).clamp(-6, 6)
        # steps of 0.5 below 2, of 1 below 4, of 2 above; torch.round takes ties to even, and the
        # even multiple of a step is the even code
        step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
        return (torch.round(y / step) * step * unit).reshape(c["n"], c["d"])
    if c["op"] == "index_scores":
        q, k = _x_e2m1(s["q_codes"], s["q_scales"]), _x_e2m1(s["k_codes"], s["k_scales"])
        out = s["scores"].double()
        k_flat, t = k.reshape(-1, c["dim"]), torch.arange(s["n_max"], device=out.device)
        for b in range(c["B"]):
            kb = k_flat[s["table"][b].long()[t // c["page"]] * c["page"] + t % c["page"]]
            for i in range(0, c["Tq"], 512):
                z = torch.einsum("thd,nd->thn", q[b, i:i + 512], kb).relu_()
                sc = torch.einsum("th,thn->tn", s["w"][b, i:i + 512].double(), z)
                last = t * c["stride"] + c["width"] - 1
                seen = (last <= s["q_pos"][b, i:i + 512, None]) & (t < s["n_cmp"][b])
                out[b, i:i + 512][seen] = sc[seen]
        return out
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    flat = s["kv"].reshape(-1, c["d"])
    q = _x_rope(s["q"].double(), s["q_pos"], c["rope"])
    for b in range(c["B"]):
        for i in range(c["Tq"]):
            t = int(s["q_pos"][b, i])
            if c["op"] == "sparse_paged":
                j = s["idx"][b, i].long()
                j = j[j >= 0]
            else:
                n = int(s["n_cmp"][b])
                j = torch.arange(n, device="cuda")
                j = j[j * c["stride"] + c["width"] - 1 <= t]
            rows = flat[s["table"][b].long()[j // c["page"]] * c["page"] + j % c["page"]]
            p0 = int(s["raw_pos0"][b])
            lo, hi = max(0, t - c["window"] + 1, p0), min(t + 1, p0 + int(s["n_raw"][b]))
            rows = torch.cat((rows, s["kv_raw"][b, lo - p0:hi - p0] if hi > lo else rows[:0])).double()
            z = torch.cat((q[b, i] @ rows.T / math.sqrt(c["d"]), s["sink"].double()[:, None]), 1)
            out[b, i] = torch.softmax(z, 1)[:, :-1] @ rows
    return _x_rope(out, -s["q_pos"], c["rope"])
