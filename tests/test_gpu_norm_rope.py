"""csa_norm_rope against the fp64 oracle: types, head counts, dims that fill
part of a lane group, strided rows, key slots, no rotation, no weights.

Tolerance, per value: half a step of the output type relative to the value,
plus the fp32 arithmetic before it.  That is at most 37 roundings in the sum
of squares (up to 32 terms per lane, 5 shuffle steps), halved by the root,
some 10 more for the mean, the root and the products, and 2 each for sine and
cosine: below 32 units of 2^-24 of the rotated pair's magnitude sum."""
import numpy as np
import pytest
import torch

import oracle
from sparse_compressed_attention_csa_b200 import Params, csa_norm_rope, csa_poll_device_error, layer

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _close(got, x, weight, pos, p, eps):
    """got against the oracle on the values of x."""
    xs = x.double().cpu().numpy()
    w = None if weight is None else weight.cpu().numpy()
    t = None if pos is None else pos.cpu().numpy()
    want = oracle.norm_rope(xs, w, t, p.rope_dim, _theta(p), eps)
    plain = np.abs(oracle.norm_rope(xs, w, None, 0, 1.0, eps))
    mag = plain + plain.reshape(plain.shape[:-1] + (-1, 2))[..., ::-1].reshape(plain.shape)
    tol = HALF[got.dtype] * np.abs(want) + 32 * 2.0 ** -24 * mag + 1e-45
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err - tol).max())


def _theta(p):
    if p.rope_factor > 1:
        return oracle.YaRN(theta=p.theta, factor=p.rope_factor, orig_ctx=p.rope_orig_ctx)
    return p.theta


def _case(rows, heads, dim, dtype, seed, max_pos=1 << 20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (3 * torch.randn((rows, heads, dim), generator=g, device="cuda")).to(dtype)
    w = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    pos = torch.randint(0, max_pos, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return x, w, pos


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,heads,dim,rope", [
    (1, 1, 128, 64), (32, 64, 128, 64), (7, 5, 96, 32), (3, 128, 512, 64), (130, 1, 512, 64),
    (5, 3, 8, 8), (9, 2, 64, 0), (2, 17, 1024, 128), (70, 3, 72, 8), (1, 300, 24, 24),
    (400, 24, 256, 64), (3, 2, 512, 512),
    (3001, 33, 128, 64), (1200, 70, 512, 64),        # several heads per lane group
])
def test_queries(rows, heads, dim, rope, dtype):
    p = Params(d=1024, rope_dim=rope) if rope in (0, 32, 64, 128, 512) else Params(d=64, rope_dim=64)
    if p.rope_dim > dim:
        p = Params(d=64, rope_dim=0)
    x, w, pos = _case(rows, heads, dim, dtype, rows + heads)
    out, _ = layer.norm_rope(p, x, w, pos)
    _close(out, x, w, pos, p, 1e-6)
    bare, _ = layer.norm_rope(p, x)           # no weights, no rotation
    _close(bare, x, None, None, p, 1e-6)
    csa_poll_device_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_queries_and_keys_of_one_projection_into_slots(dtype):
    rows, hq, hk, dim = 77, 6, 2, 128
    p = Params(rope_factor=16.0, rope_orig_ctx=65536, theta=160000.0)
    x, w, pos = _case(rows, hq + hk + 1, dim, dtype, 5)
    proj = x.flatten(1)
    q = proj[:, :hq * dim].unflatten(-1, (hq, dim))
    k = proj[:, hq * dim:(hq + hk) * dim].unflatten(-1, (hk, dim))
    slots = torch.randperm(128, device="cuda")[:rows].to(torch.int32)
    slots[3] = -1
    cache = torch.full((128, hk, dim), 7.0, device="cuda", dtype=dtype)
    q_out, k_out = layer.norm_rope(p, q, w, pos, k, None, pos, cache, slots, eps=1e-5)
    assert k_out is cache
    _close(q_out, q, w, pos, p, 1e-5)
    live = slots >= 0
    _close(cache[slots[live].long()], k[live], None, pos[live], p, 1e-5)
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[slots[live].long()] = False
    assert torch.all(cache[rest] == 7.0)      # rows that no slot names
    csa_poll_device_error()


def test_slots_outside_the_cache_are_reported_and_skipped():
    from sparse_compressed_attention_csa_b200 import CsaError
    x, w, pos = _case(40, 2, 128, torch.bfloat16, 6)
    slots = torch.arange(40, device="cuda", dtype=torch.int32)
    slots[5], slots[39] = 41, -2
    guard = torch.full((42, 2, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    p = Params()
    csa_norm_rope(p, 1e-6, k=x, k_weight=w, k_pos=pos, k_out=guard[:41], k_slots=slots)
    torch.cuda.synchronize()
    with pytest.raises(CsaError) as ei:
        csa_poll_device_error()
    assert ei.value.status == 8
    assert torch.all(guard[41] == 3.0) and torch.all(guard[5] == 3.0) and torch.all(guard[39] == 3.0)
    keep = [i for i in range(40) if i not in (5, 39)]
    _close(guard[keep], x[keep], w, pos[keep], p, 1e-6)


def test_in_place_zero_rows_and_large_values():
    p = Params()
    x, w, pos = _case(33, 4, 128, torch.bfloat16, 7)
    x[3] = 0
    x[4] *= 1e15                                # below 2^63 / sqrt(128)
    want, _ = layer.norm_rope(p, x, w, pos)
    _close(want, x, w, pos, p, 1e-6)
    assert torch.all(want[3] == 0)
    csa_norm_rope(p, 1e-6, x, w, pos, x)
    assert torch.equal(x, want)
    # a NaN stays in its own head row
    y = torch.ones(2, 2, 128, device="cuda")
    y[0, 1, 5] = float("nan")
    out, _ = layer.norm_rope(p, y)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all() and torch.isfinite(out[1]).all()


def test_refusals_on_device_tensors():
    p = Params()
    x, w, pos = _case(4, 2, 128, torch.bfloat16, 8)
    out = torch.empty_like(x)
    with pytest.raises(TypeError):
        csa_norm_rope(p, 1e-6, x.half(), w, pos, out)
    with pytest.raises(ValueError):
        csa_norm_rope(p, 1e-6, x, w[:64], pos, out)
    with pytest.raises(ValueError):
        csa_norm_rope(p, 1e-6, x, w, pos[:3], out)
    with pytest.raises(ValueError):
        csa_norm_rope(p, 1e-6, x.transpose(0, 1), w, pos[:2], out.transpose(0, 1))
    with pytest.raises(TypeError):
        csa_norm_rope(p, 1e-6, x, w, pos.long(), out)
