"""Pins of the 4-bit oracle: hand values, the code tables, and its invariants."""
import numpy as np
import pytest
import torch

from oracle import h3_fp4 as o


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.E4M3, t)


def test_rounding_ties_to_the_even_code_and_saturates():
    a = [0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 100.0]
    assert list(o.E2M1[o.nearest_even(a, o.E2M1)]) == [0, 0.5, 1, 1, 2, 2, 3, 4, 4, 6, 6]


def test_mx_scale_by_hand():
    x = np.zeros((5, 32))
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = 6.0, 7.0, 7.25, -0.5
    codes, sc, row, _ = o.quantize(x, "mx")
    # 7 saturates at 6 under scale 1; 7.25 needs scale 2 (7.25 / 2 = 3.625 -> 4); 0.5 = 4 * 2^-3
    assert list(sc[:4, 0] - 127) == [0, 0, 1, -3] and sc[4, 0] == 1 and np.all(row == 1)
    assert list(o.values(codes, sc, row, "mx")[:4, 3]) == [6.0, 6.0, 8.0, -0.5]


def test_nv_scales_by_hand():
    x = np.zeros((3, 32))
    x[0, 0], x[0, 16] = 2688.0, 3.0
    x[1, 0] = 2689.0
    codes, sc, row, _ = o.quantize(x, "nv")
    assert list(row) == [1.0, 2.0, 1.0]
    assert list(o.E4M3[sc[0]]) == [448.0, 0.5] and list(sc[2]) == [0, 0]
    v = o.values(codes, sc, row, "nv")
    assert v[0, 0] == 2688.0 and v[0, 16] == 3.0 and np.all(v[2] == 0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rot", [False, True])
def test_values_are_near_the_input(fmt, rot):
    x = np.random.default_rng(1).standard_normal((7, 256)) * 10.0 ** np.arange(-3, 4)[:, None]
    c, s, r, _ = o.quantize(x, fmt, rot)
    v = o.values(c, s, r, fmt)
    ref = o.rotate(x) / np.sqrt(128) if rot else x
    # half the widest step of a block (2, under amax >= 3.5 scales or, in NV,
    # 6 of 17/16 scales) against its amax
    err = np.abs(v - ref).reshape(7, -1, o.BLOCK[fmt]).max(-1) / np.abs(ref).reshape(7, -1, o.BLOCK[fmt]).max(-1)
    assert err.max() <= 1 / 3.5 + 1e-12 and np.abs(v - ref).mean() < 0.12 * np.abs(ref).mean() * 10
    assert np.all((v == 0) | (np.sign(v) == np.sign(ref)))


def test_non_finite_blocks_are_nan_and_alone():
    x = np.random.default_rng(2).standard_normal((2, 64))
    y = x.copy()
    y[0, 5], y[1, 40] = np.inf, np.nan
    for fmt in ("mx", "nv"):
        c, s, r, bad = o.quantize(y, fmt)
        v = o.values(c, s, r, fmt).reshape(2, -1, o.BLOCK[fmt])
        assert bad.sum() == 2 and np.isnan(v[bad]).all() and np.isfinite(v[~bad]).all()


def test_scale_offsets_fill_the_atoms_once():
    off = o.scale_offsets(256, 8)
    assert sorted(off.ravel()) == list(range(256 * 8))
    assert off[0, 0] == 0 and off[1, 0] == 16 and off[32, 0] == 4 and off[0, 4] == 512 and off[128, 0] == 1024


def test_rotated_product_is_the_product():
    rng = np.random.default_rng(3)
    a, b = rng.standard_normal((3, 256)), rng.standard_normal((4, 256))
    np.testing.assert_allclose((o.rotate(a) / np.sqrt(128)) @ (o.rotate(b) / np.sqrt(128)).T, a @ b.T, atol=1e-12)


def test_sandwich_by_hand():
    x, y = np.array([[3.0, 4.0], [1.0, 1.0]]), np.array([[3.0, -4.0], [5.0, 5.0]])
    t = np.zeros((1, 1, 6, 2))
    t[0, 0, 2], t[0, 0, 3], t[0, 0, 4] = [2.0, 2.0], [0.5, 0.5], [1.0, 1.0]
    x1, h = o.sandwich(x, y, [0, -1], [0, 0], t, 0, post_norm=False, norm_eps=0.0, branch_scale=0.5)
    assert np.array_equal(x1, [[6.0, 0.0], [1.0, 1.0]])
    np.testing.assert_allclose(h, [[2 * np.sqrt(2) + 0.5, 0.5], [1.0, 1.0]])
    x1, h = o.sandwich(x, y, [0, 0], [0, 0], t, 0, post_gain=[1.0, 10.0], post_eps=0.0)
    np.testing.assert_allclose(x1[0], [3 + 2 * 3 / np.sqrt(12.5), 4 - 20 * 4 / np.sqrt(12.5)])
