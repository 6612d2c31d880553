"""Pins of the paged-path oracle (CPU): E2M1 against the format's points and a
search over all codes, the block scale, norms and rotations, page lookup."""
import numpy as np
import pytest

import oracle


def test_e2m1_points():
    v = oracle.e2m1_values()
    assert v[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    np.testing.assert_array_equal(v[8:], -v[:8])


def test_e2m1_ties_go_to_the_even_code():
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert oracle.e2m1_encode(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert oracle.e2m1_encode([-m for m in mid]).tolist() == [8, 10, 10, 12, 12, 14, 14]
    assert oracle.e2m1_encode([7.9, -100.0, 0.0, -0.0]).tolist() == [7, 15, 0, 8]


def test_mxfp4_scale_and_error():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 96)) * np.exp2(rng.integers(-30, 30, (50, 1)).astype(float))
    x[3] = 0.0
    codes, scales = oracle.mxfp4_encode(x)
    y = oracle.mxfp4_decode(codes, scales)
    b, q = x.reshape(50, 3, 32), y.reshape(50, 3, 32)
    s = np.exp2(scales.astype(float) - 127)
    amax = np.abs(b).max(-1)
    live = amax > 0
    assert np.all((amax[live] / s[live] >= 4) & (amax[live] / s[live] < 8))
    assert np.all(scales[3] == 127) and np.all(y[3] == 0)
    # within half a step: 0.25 below 2, 0.5 below 4, 1 below 6, and 2 where 6 saturates
    err = np.abs(b - q) / s[..., None]
    a = np.abs(b) / s[..., None]
    lim = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, np.where(a <= 6, 1.0, 2.0)))
    assert np.all(err <= lim)


def test_mxfp4_values_are_fixed_points():
    # the values that codes stand for encode to themselves when the block's
    # largest code is 4 or 6 (any smaller one would move the scale)
    rng = np.random.default_rng(2)
    c = rng.integers(0, 16, (20, 64)).astype(np.uint8)
    c[:, 0], c[:, 32] = 7, 14
    c[c == 8] = 0
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    scales = rng.integers(100, 150, (20, 2)).astype(np.uint8)
    again, s2 = oracle.mxfp4_encode(oracle.mxfp4_decode(codes, scales))
    np.testing.assert_array_equal(s2, scales)
    np.testing.assert_array_equal(again, codes)


def test_mxfp4_blocks_with_nan_or_infinity():
    x = np.ones((1, 64))
    x[0, 5] = np.inf
    codes, scales = oracle.mxfp4_encode(x)
    assert scales.tolist() == [[255, 125]] and np.all(codes[0, :16] == 0)
    assert np.all(np.isnan(oracle.mxfp4_decode(codes, scales)[0, :32]))


def test_norm_rope_has_unit_rms_and_turns_only_the_tail():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 3, 16)) * 7
    y = oracle.norm_rope(x, None, None, 8, 1e4, 1e-12)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-10)
    z = oracle.norm_rope(x, None, [0, 1, 5, 100], 8, 1e4, 1e-12)
    np.testing.assert_array_equal(z[..., :8], y[..., :8])
    np.testing.assert_allclose(z[0], y[0], rtol=1e-14)
    np.testing.assert_allclose((z * z).sum(-1), (y * y).sum(-1), rtol=1e-12)
    a = np.cos(5.0) * y[2, 1, 8] - np.sin(5.0) * y[2, 1, 9]
    assert z[2, 1, 8] == pytest.approx(a, rel=1e-12)


def test_paged_rows_follow_the_table():
    pool = np.arange(5 * 4).reshape(5, 4)
    assert oracle.paged_rows(pool, [3, 0, 99], 6).tolist() == [12, 13, 14, 15, 0, 1]
