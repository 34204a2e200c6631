"""4-bit products and dequantisation where their arithmetic is at its limits,
against fp64."""
import numpy as np
import pytest
import torch

from oracle import h3_fp4 as o
from tests.test_gpu_fp4 import _operands, _tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def j():
    assert torch.cuda.is_available(), "GPU tests need a B200"
    import joint_video_audio_b200
    return joint_video_audio_b200


E2M1 = torch.tensor([.5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6])


def wide_gates(m, f, seed):
    """MX operands [m, 128] and [2 f, 128] whose values are multiples of a
    quarter (gates) and of 2^-6 (ups), so that their fp32 sums are exact; the
    gates reach past +-100."""
    g = torch.Generator().manual_seed(seed)
    a = E2M1[torch.randint(0, 14, (m, 128), generator=g)]
    b = E2M1[torch.randint(0, 14, (2 * f, 128), generator=g)]
    a[:, ::32], b[:, ::32] = 6, -6  # every block's scale is the table's own
    a = a / 2
    b[f:] /= 16
    return a, b


WIDE_GATES = [(5, 1024), (40, 512), (300, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,f", WIDE_GATES)
def test_swiglu_of_wide_gates(j, dtype, m, f):
    """The product is exact, so that what is left is swiglu's own error: two units
    of the last place each (2^-22) for the exponential, which enters numerator and
    denominator by its factor, and for the quotient, one rounding (2^-24) each for
    the sum, the products with g and with u; together below 2^-20, and the output
    type's own. Where the output is bf16 the exponent -|g| log2 e is rounded to fp32:
    half a step of up to 184 is 2^-17, times log 2, and the rounding of log2 e
    itself another 128 * 2^-26: 2^-17 together. An exponential below the normals is
    good to two of the smallest steps, and so are the products and the output."""
    a, b = wide_gates(m, f, m + f)
    ya = a.double().numpy() @ b.double().numpy().T
    g, u = ya[:, :f], ya[:, f:]
    assert g.min() < -100 and g.max() > 100 and ((g > -88.7) & (g < -87.4)).any()
    ref = g / (1 + np.exp(-g)) * u
    qa, qb = (j.quantize_fp4(v.to(torch.bfloat16).cuda(), "mx") for v in (a, b))
    assert torch.equal(j.dequantize_fp4(qa).cpu().float(), a) and torch.equal(j.dequantize_fp4(qb).cpu().float(), b)
    got = j.gemm_fp4(qa, qb, swiglu=True, dtype=dtype).double().cpu().numpy()
    out = torch.finfo(dtype)
    step = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    tol = np.abs(ref) * (out.eps / 2 + 2.0 ** -20 + (2.0 ** -17 if dtype == torch.bfloat16 else 0)) + 2.0 ** -147 * (np.abs(g) + 1) * (np.abs(u) + 1) + step
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{bad.sum()} values, first at g = {g[bad][0]}, u = {u[bad][0]}: {got[bad][0]} not {ref[bad][0]}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_rotated_values_near_the_largest_float(j, dtype):
    """Rotated sums near 2^128 under a block scale of 2^126: code times scale is
    2^128 there, the value 2^128 / sqrt(128) and finite. Two roundings of fp32 (the
    product's and the row scale's), one of the output."""
    x = torch.zeros(3, 256)
    x[0, 0], x[0, 1] = 1.6e38, 1.4e38
    x[1, 130], x[1, 131], x[1, 200] = -1.5e38, 1.1e38, -0.6e38
    x = x.to(torch.bfloat16)
    c, s, r, bad = o.quantize(x, "mx", True)
    assert not bad.any() and s.max() == 253 and (c[s.repeat(32, 1) == 253] & 7).max() >= 6
    ref = o.values(c, s, r, "mx")
    assert np.abs(ref).max() < 2.0 ** 126
    got = j.dequantize_fp4(j.quantize_fp4(x.cuda(), "mx", rotate=True), dtype).double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= np.abs(ref) * (2.0 ** -23 + torch.finfo(dtype).eps / 2))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k,swiglu", [(1, 512, 5376, True), (17, 512, 5472, True), (50, 1024, 4128, True), (64, 256, 7168, True),
                                          (20, 256, 2048, False), (33, 384, 2080, False)])
def test_few_rows_with_split_sums(j, fmt, dtype, m, n, k, swiglu):
    """Up to 64 rows whose K several CTAs share, at each of the kernel's widths
    (16, 32, 64 rows), into a wider buffer whose other bytes stay as they were.
    Bounds as for the other products, with silu' <= 1.1 and swiglu's own error
    (test_swiglu_of_wide_gates) below 2^-17 (bf16) and 2^-20 (fp32)."""
    qa, qb, a, b = _operands(j, m, n, k, fmt)
    cols = n // 2 if swiglu else n
    buf = torch.full((m + 3, cols + 16), 7.0, dtype=dtype, device="cuda")
    out = buf[1:m + 1, 8:8 + cols]
    j.gemm_fp4(qa, qb, swiglu=swiglu, dtype=dtype, out=out)
    got, y = out.double().cpu().numpy(), o.product(a, b)
    if swiglu:
        t = _tolerance(a, b, torch.float32, y)
        g, u, y = y[:, :cols], y[:, cols:], o.product(a, b, True)
        own = 2.0 ** -17 if dtype == torch.bfloat16 else 2.0 ** -20
        tol = 1.1 * t[:, :cols] * np.abs(u) + np.abs(o.silu(g)) * t[:, cols:] + np.abs(y) * (torch.finfo(dtype).eps / 2 + own) + 1e-30
    else:
        tol = _tolerance(a, b, dtype, y)
    assert np.all(np.abs(got - y) <= tol)
    out.fill_(7)
    assert torch.all(buf == 7)
