"""Dequantisation rounds code * block scale * row scale to fp32 and then to bf16. For
every code, scale and row scale that the quantisation writes that is the nearest
bf16 of the exact product: rows of power-of-two scale are exact up to the last
rounding, and of the rotated ones no fp32 value lies where the second rounding
would go the other way."""
import numpy as np
import pytest

from oracle import h3_fp4 as o

ROT = np.float64(np.float32(1 / np.sqrt(128.0)))


def _bf16(x):
    """Nearest bf16 of fp64 values, ties to even, subnormals included (below the largest)."""
    m, e = np.frexp(x)
    step = np.maximum(e - 8, -133)
    return np.ldexp(np.round(np.ldexp(x, -step)), step)


def _check(values, row_scale):
    a = np.float32(values)
    assert np.array_equal(np.float64(a), values)  # code times block scale: exact
    exact = values * row_scale                    # 6 + 24 bits: exact in fp64
    twice = _bf16(np.float64(a * np.float32(row_scale)))
    assert np.array_equal(twice, _bf16(exact))


@pytest.mark.parametrize("rot", [1.0, ROT])
def test_nv(rot):
    v = (o.E2M1[None, :] * o.E4M3[:, None]).ravel()
    for e in range(-126, 118):
        row = np.ldexp(rot, e)
        _check(v[v * row < 3.38e38], row)  # (a value past the largest float is infinite in either type)


@pytest.mark.parametrize("rot", [1.0, ROT])
def test_mx(rot):
    for e in range(-126, 126):
        _check(o.E2M1 * 2.0 ** e, rot)
