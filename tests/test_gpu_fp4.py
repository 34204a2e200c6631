"""4-bit linear path on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import h3_fp4 as o

pytestmark = pytest.mark.gpu

FMT = ["mx", "nv"]


@pytest.fixture(scope="module")
def j():
    assert torch.cuda.is_available(), "GPU tests need a B200"
    import joint_video_audio_b200
    return joint_video_audio_b200


def _rows(rows, k, seed, spread=1.0):
    """Rows over many binades, with a zero row and zero blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g) * spread)
    if rows > 2:
        x[rows // 2] = 0
        x[0, :32] = 0
    return x.to(torch.bfloat16)


def unpack(q, o_blocks):
    """(codes 0..15, scale codes [rows, blocks], row scales) of an Fp4Tensor, on the host."""
    c = q.codes.cpu().numpy()
    codes = np.stack([c & 15, c >> 4], -1).reshape(q.shape)
    sc = q.scales.cpu().numpy().reshape(-1)[o.scale_offsets(q.shape[0], o_blocks)]
    return codes, sc, q.row_scale.cpu().numpy().astype(np.float64)


def assert_same_bits(q, ref):
    codes, sc, row = unpack(q, q.shape[1] // o.BLOCK[q.fmt])
    rc, rs, rr, bad = ref
    assert np.array_equal(sc, rs)
    np.testing.assert_allclose(row, rr, rtol=2.0 ** -24)
    keep = ~np.repeat(bad, o.BLOCK[q.fmt], axis=1)
    diff = (codes != rc) & keep
    assert not diff.any(), f"{diff.sum()} codes differ, first at {np.argwhere(diff)[0]}"


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (2, 96), (127, 128), (129, 160), (300, 256), (5, 1024), (5, 1056),
                                    (9, 5376), (3, 7168), (2, 16384), (257, 2016)])
def test_quantize_bits(j, fmt, rows, k):
    x = _rows(rows, k, rows * 31 + k)
    assert_same_bits(j.quantize_fp4(x.cuda(), fmt), o.quantize(x, fmt))


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_every_bf16_value(j, fmt):
    """All 65,536 bit patterns, each beside values that make it a tie, a
    block's largest or a small one; infinities and NaN among them."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.cat([bits.view(-1, 512), bits.flip(0).view(512, 128).T.reshape(-1, 512)], 0)
    assert_same_bits(j.quantize_fp4(x.cuda(), fmt), o.quantize(x, fmt))
    # one value a block against a fixed largest one: ties among the codes
    y = torch.zeros(65536 // 32, 32, 32)
    y[:, :, 0] = 6.0
    y[:, :, 1] = bits.float().view(-1, 32).nan_to_num(0, 0, 0).clamp(-6, 6)
    y = y.view(-1, 1024).to(torch.bfloat16)
    assert_same_bits(j.quantize_fp4(y.cuda(), fmt), o.quantize(y, fmt))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,k", [(20001, 64), (3000, 1056), (1500, 2080), (700, 4128)])
def test_quantize_more_rows_than_ctas(j, fmt, rows, k):
    """Every CTA takes many rows, its ring goes round several times."""
    x = _rows(rows, k, k)
    x[rows // 3, 40] = float("nan")
    assert_same_bits(j.quantize_fp4(x.cuda(), fmt), o.quantize(x, fmt))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,k", [(3, 128), (40, 5376), (1, 1152), (2, 16384)])
def test_quantize_rotated_bits(j, fmt, rows, k):
    """Integers of up to 8 bits: their sums of 128 are exact in fp32, so the
    rotated codes have one answer."""
    g = torch.Generator().manual_seed(k)
    x = torch.randint(-128, 129, (rows, k), generator=g).to(torch.bfloat16)
    assert_same_bits(j.quantize_fp4(x.cuda(), fmt, rotate=True), o.quantize(x, fmt, True))


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_rotated_non_finite(j, fmt):
    """An infinity or a NaN takes its 128 channels and nothing else."""
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-64, 65, (5, 1280), generator=g).to(torch.bfloat16)
    y = x.clone()
    y[1, 300], y[3, 1279] = float("inf"), float("nan")
    y[3, 1100], y[4, 0], y[4, 1] = float("-inf"), float("inf"), float("-inf")
    q = j.quantize_fp4(y.cuda(), fmt, rotate=True)
    v = j.dequantize_fp4(q, torch.float32).double().cpu().numpy()
    bad = np.zeros((5, 10), bool)
    bad[1, 2], bad[3, 9], bad[3, 8], bad[4, 0] = True, True, True, True
    assert np.array_equal(np.isnan(v).reshape(5, 10, 128), np.repeat(bad[..., None], 128, 2))
    c, s, r, _ = o.quantize(y, fmt, True)
    ok = np.repeat(~bad, 128, 1)
    np.testing.assert_allclose(v[ok], o.values(c, s, r, fmt)[ok], rtol=2.0 ** -22)


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_strided_rows_and_pads(j, fmt):
    """Rows inside a wider buffer; the scale bytes past K are finite, those of
    rows past the last are left as they were."""
    wide = _rows(70, 512, 5).cuda()
    x = wide[:, 64:64 + 160]
    q = j.Fp4Tensor(70, 160, fmt)
    q.buffer.fill_(0xEE)
    assert j.quantize_fp4(x, fmt, out=q) is q
    assert_same_bits(q, o.quantize(x.cpu(), fmt))
    blocks = 160 // o.BLOCK[fmt]
    off = o.scale_offsets(128, -(-blocks // 4) * 4)
    sc = q.scales.cpu().numpy().reshape(-1)
    assert np.all(sc[off[:70, blocks:]] < 0x7f)
    assert np.all(sc[off[70:]] == 0xEE)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 32), (130, 96), (33, 5376), (2, 16384)])
def test_dequantize_values(j, fmt, dtype, rows, k):
    x = _rows(rows, k, 3 * k)
    x[0, 1] = float("nan")
    x[-1, -1] = float("inf")
    got = j.dequantize_fp4(j.quantize_fp4(x.cuda(), fmt), dtype).double().cpu().numpy()
    c, s, r, _ = o.quantize(x, fmt)
    v = o.values(c, s, r, fmt)  # 6 significant bits at most: exact in either type
    assert np.array_equal(np.isnan(got), np.isnan(v)) and np.array_equal(got[~np.isnan(v)], v[~np.isnan(v)])


def _tolerance(a, b, dtype, y):
    """Sum of |a b| times the accumulator's steps (one rounding per 64
    channels, 2^-23 for an adder that truncates, and the alignment of the 64
    products inside one), the two row scales' roundings, the output's."""
    acc = np.abs(np.nan_to_num(a)) @ np.abs(np.nan_to_num(b)).T
    return acc * (2.0 ** -20 + (a.shape[1] / 64 + 4) * 2.0 ** -23) + np.abs(y) * (
        torch.finfo(dtype).eps / 2 + 2.0 ** -22) + 1e-30


def _operands(j, m, n, k, fmt, rot=False):
    g = torch.Generator().manual_seed(m * 7 + n * 3 + k)
    a = (torch.randn(m, k, generator=g) * torch.exp(0.5 * torch.randn(m, 1, generator=g))).to(torch.bfloat16)
    b = (torch.randn(n, k, generator=g) / k ** 0.5).to(torch.bfloat16)
    qa, qb = j.quantize_fp4(a.cuda(), fmt, rotate=rot), j.quantize_fp4(b.cuda(), fmt, rotate=rot)
    va, vb = (j.dequantize_fp4(q, torch.float32).double().cpu().numpy() for q in (qa, qb))
    return qa, qb, va, vb


SHAPES = [(1, 8, 32), (1, 128, 64), (2, 136, 96), (16, 384, 256), (17, 96, 288), (33, 128, 1024), (65, 256, 160),
          (128, 128, 512), (129, 264, 5376), (300, 1032, 768), (515, 768, 1312), (1, 5376, 7168), (1025, 520, 2048)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm(j, fmt, dtype, m, n, k):
    qa, qb, a, b = _operands(j, m, n, k, fmt)
    y = o.product(a, b)
    got = j.gemm_fp4(qa, qb, dtype=dtype).double().cpu().numpy()
    assert np.all(np.abs(got - y) <= _tolerance(a, b, dtype, y))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("m,n,k", [(2600, 2000, 256), (2300, 2600, 160), (2600, 2600, 96), (200, 5376, 512), (140, 72, 1024)])
def test_gemm_waves(j, fmt, m, n, k):
    """More tiles than the SMs take at once, the rest in quarters, halves or whole; fewer tiles than SMs."""
    qa, qb, a, b = _operands(j, m, n, k, fmt)
    y = o.product(a, b)
    got = j.gemm_fp4(qa, qb).double().cpu().numpy()
    assert np.all(np.abs(got - y) <= _tolerance(a, b, torch.bfloat16, y))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("m,n,k", [(1, 256, 128), (37, 512, 288), (64, 256, 96), (200, 768, 1024), (700, 1536, 512)])
def test_gemm_swiglu(j, fmt, m, n, k):
    qa, qb, a, b = _operands(j, m, n, k, fmt)
    y = o.product(a, b)
    g, u = y[:, :n // 2], y[:, n // 2:]
    t = _tolerance(a, b, torch.float32, y)
    ref = o.product(a, b, True)
    # silu' <= 1.1; the exponential and the quotient are good to 2^-20
    tol = 1.1 * t[:, :n // 2] * np.abs(u) + np.abs(o.silu(g)) * t[:, n // 2:] + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)
    got = j.gemm_fp4(qa, qb, swiglu=True).double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol + 1e-30)


@pytest.mark.parametrize("m,n,k", [(1, 128, 14336), (130, 256, 14336), (600, 640, 5376)])
def test_gemm_exact_integers(j, m, n, k):
    """Every block's largest is 6 or 4 (scale 1): products are multiples of a
    quarter up to 36, their sums exact in fp32 in any order."""
    g = torch.Generator().manual_seed(k + m)
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6])
    a, b = (t[torch.randint(0, 15, (r, k), generator=g)] for r in (m, n))
    a[:, ::32], b[:, ::32] = 6, -6
    qa, qb = (j.quantize_fp4(v.to(torch.bfloat16).cuda(), "mx") for v in (a, b))
    got = j.gemm_fp4(qa, qb, dtype=torch.float32).double().cpu()
    assert torch.equal(got, a.double() @ b.double().T)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("m", [3, 600])
def test_gemm_nan_stays_in_its_row_and_column(j, fmt, m):
    k, n = 512, 256
    g = torch.Generator().manual_seed(1)
    a = torch.randn(m, k, generator=g).to(torch.bfloat16)
    b = torch.randn(n, k, generator=g).to(torch.bfloat16)
    a[1, 70], b[9, 300] = float("nan"), float("inf")
    y = j.gemm_fp4(j.quantize_fp4(a.cuda(), fmt), j.quantize_fp4(b.cuda(), fmt)).cpu()
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[1], bad[:, 9] = True, True
    assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("m", [5, 700])
@pytest.mark.parametrize("swiglu", [False, True])
def test_gemm_into_a_wider_buffer(j, m, swiglu):
    """A strided output; its other columns and the row behind it stay as they were."""
    qa, qb, _, _ = _operands(j, m, 512, 256, "nv")
    n = 256 if swiglu else 512
    ref = j.gemm_fp4(qa, qb, swiglu=swiglu)
    buf = torch.full((m + 1, n + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    j.gemm_fp4(qa, qb, swiglu=swiglu, out=buf[:m, 8:8 + n])
    assert torch.equal(buf[:m, 8:8 + n], ref)
    assert torch.all(buf[:, :8] == 7) and torch.all(buf[:, 8 + n:] == 7) and torch.all(buf[m] == 7)


@pytest.mark.parametrize("fmt", FMT)
def test_rotated_operands_give_the_product(j, fmt):
    """Rotating both sides leaves the product: the result is as near to it as
    the 4-bit values' own distance from the rotated inputs allows."""
    g = torch.Generator().manual_seed(9)
    a = torch.randn(200, 1024, generator=g)
    a[:, 5] *= 30  # an outlier channel, which the rotation spreads
    b = torch.randn(256, 1024, generator=g) / 32
    a, b = a.to(torch.bfloat16), b.to(torch.bfloat16)
    qa, qb = j.quantize_fp4(a.cuda(), fmt, rotate=True), j.quantize_fp4(b.cuda(), fmt, rotate=True)
    va, vb = (j.dequantize_fp4(q, torch.float32).double().cpu().numpy() for q in (qa, qb))
    y = j.gemm_fp4(qa, qb, dtype=torch.float32).double().cpu().numpy()
    assert np.all(np.abs(y - va @ vb.T) <= _tolerance(va, vb, torch.float32, y))
    full = a.double().numpy() @ b.double().numpy().T
    ra, rb = o.rotate(a.double().numpy()) / 128 ** 0.5, o.rotate(b.double().numpy()) / 128 ** 0.5
    slack = np.abs(va - ra) @ np.abs(rb).T + np.abs(va) @ np.abs(vb - rb).T
    assert np.all(np.abs(y - full) <= slack + 1e-3)


@pytest.mark.parametrize("m", [7, 600])
def test_repeats_graphs_and_streams(j, m):
    """The same bits from every run: eagerly, twice at once on two streams, and
    replayed from a graph whose inputs changed in place."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(m, 768, generator=g).to(torch.bfloat16).cuda()
    x2 = torch.randn(m, 768, generator=g).to(torch.bfloat16).cuda()
    w = j.quantize_fp4((torch.randn(1024, 768, generator=g) / 28).to(torch.bfloat16).cuda(), "nv")
    step = lambda v: j.gemm_fp4(j.quantize_fp4(v, "nv"), w)  # noqa: E731
    ref, ref2 = step(x), step(x2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        for s, v in ((s1, x), (s2, x2)):
            with torch.cuda.stream(s):
                outs.append(step(v))
    torch.cuda.synchronize()
    assert all(torch.equal(y, (ref, ref2)[i % 2]) for i, y in enumerate(outs))
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(buf)
    graph.replay()
    assert torch.equal(y, ref)
    buf.copy_(x2)
    graph.replay()
    assert torch.equal(y, ref2)


def test_empty_operands(j):
    w = j.quantize_fp4(torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda"), "mx")
    q = j.quantize_fp4(torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda"), "mx")
    assert j.dequantize_fp4(q).shape == (0, 128) and j.gemm_fp4(q, w).shape == (0, 64)


@pytest.mark.parametrize("fmt", FMT)
def test_offsets_past_32_bits(j, fmt):
    """270 repeats of 1000 rows: the values' and the product's indices pass 2^31
    and their bytes 2^32, the codes' bytes 2^31. Every repeat gives the bits of
    the first, and those of the 1000 rows alone."""
    reps, rows, k, n = 270, 1000, 16384, 8192
    assert reps * rows * k // 2 > 2 ** 31 < reps * rows * n
    base = _rows(rows, k, 21).cuda()
    one, q = j.quantize_fp4(base, fmt), j.quantize_fp4(base.repeat(reps, 1), fmt)
    assert torch.equal(q.codes.view(reps, -1), one.codes.view(1, -1).expand(reps, -1))
    assert torch.equal(q.row_scale.view(reps, -1), one.row_scale.expand(reps, -1))
    v, first = j.dequantize_fp4(q), j.dequantize_fp4(one)
    assert torch.equal(v.view(reps, -1), first.view(1, -1).expand(reps, -1))
    del v
    g = torch.Generator().manual_seed(22)
    w = j.quantize_fp4((torch.randn(n, k, generator=g) / 128).to(torch.bfloat16).cuda(), fmt)
    y, first = j.gemm_fp4(q, w), j.gemm_fp4(one, w)
    assert torch.equal(y.view(reps, -1), first.view(1, -1).expand(reps, -1))


NARROW = [(1, 128, 128), (15, 256, 256), (17, 256, 296), (16, 384, 384), (9, 384, 400), (7, 512, 512), (70003, 128, 136),
          (20001, 512, 512), (5, 640, 640), (33, 32, 40), (18, 288, 288), (30000, 480, 488)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,k,stride,rotate", [(*c, r) for c in NARROW for r in (False, True) if not r or c[1] % 128 == 0])
def test_narrow_rows(j, fmt, rows, k, stride, rotate):
    """Several rows to a warp: integers, whose rotated sums are exact; a row's
    scale is its own, and non-finite values stay in their block."""
    g = torch.Generator().manual_seed(rows + k)
    wide = torch.randint(-128, 129, (rows, stride), generator=g).to(torch.bfloat16)
    wide *= torch.exp2(torch.randint(-30, 31, (rows, 1), generator=g)).to(torch.bfloat16)
    x = wide[:, :k]
    if rows > 4:
        x[rows // 2] = 0
        if not rotate:
            x[1, 3], x[rows - 1, k - 1] = float("inf"), float("nan")
    q = j.Fp4Tensor(rows, k, fmt)
    q.buffer.fill_(0xEE)
    j.quantize_fp4(wide.cuda()[:, :k], fmt, rotate=rotate, out=q)
    assert_same_bits(q, o.quantize(x, fmt, rotate))
    pads = q.scales.cpu().numpy().reshape(-1)[o.scale_offsets(-(-rows // 128) * 128, k // o.BLOCK[fmt])[rows:]]
    assert np.all(pads == 0xEE)


def test_calls_keep_no_memory(j):
    """Outputs made by the calls are freed with their last reference, and errors leave none."""
    import gc
    import sys
    x = torch.randn(64, 256, device="cuda").to(torch.bfloat16)
    w = j.quantize_fp4(torch.randn(128, 256, device="cuda").to(torch.bfloat16))
    tag, table = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, 6, 256, device="cuda")

    def step():
        q = j.quantize_fp4(x)
        j.quantize_fp4(x, out=q)
        y = j.gemm_fp4(q, w)
        j.gemm_fp4(q, w, out=y)
        v = j.dequantize_fp4(q, torch.float32)
        x1, h = j.sandwich_norm(x, x, tag, tag, table)
        j.sandwich_norm(x1, h, tag, tag, table, h="mx", x_out=x1)
        with pytest.raises(j.H3BlkError):
            j.quantize_fp4(x[:, :160], rotate=True)  # a rotation takes whole blocks of 128
        with pytest.raises(ValueError):
            j.gemm_fp4(q, w, out=v)

    step()
    gc.collect()
    held = (x, w, w.buffer, tag, table)
    before = torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in held]
    for _ in range(20):
        step()
    gc.collect()
    assert (torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in held]) == before


def test_calls_from_two_threads(j):
    """Each thread on its own stream, with its own operands."""
    import threading
    g = torch.Generator().manual_seed(61)
    xs = [torch.randn(200, 512, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    w = j.quantize_fp4((torch.randn(256, 512, generator=g) / 23).to(torch.bfloat16).cuda())
    refs = [j.gemm_fp4(j.quantize_fp4(x), w) for x in xs]
    torch.cuda.synchronize()
    good = [0, 0]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                good[i] += torch.equal(j.gemm_fp4(j.quantize_fp4(xs[i]), w), refs[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert good == [50, 50]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m,n,k", [(65, 256, 256), (100, 1536, 768), (128, 512, 5376), (129, 256, 5472), (200, 512, 7168),
                                   (385, 256, 4128), (1000, 256, 6144), (130, 1280, 14336)])
def test_gemm_rows_between_the_kernels(j, fmt, swiglu, m, n, k):
    """Row counts that either kernel may take, by the sums that K is split into:
    several row tiles with split sums, a ragged K, into a wider buffer whose
    other columns and rows stay as they were."""
    qa, qb, a, b = _operands(j, m, n, k, fmt)
    cols = n // 2 if swiglu else n
    buf = torch.full((m + 3, cols + 16), 7.0, dtype=torch.float32, device="cuda")
    out = buf[1:m + 1, 8:8 + cols]
    j.gemm_fp4(qa, qb, swiglu=swiglu, dtype=torch.float32, out=out)
    got, y = out.double().cpu().numpy(), o.product(a, b)
    tol = _tolerance(a, b, torch.float32, y)
    if swiglu:  # as in test_gemm_swiglu, fp32 out
        g, u, ref = y[:, :cols], y[:, cols:], o.product(a, b, True)
        tol = 1.1 * tol[:, :cols] * np.abs(u) + np.abs(o.silu(g)) * tol[:, cols:] + np.abs(ref) * (2.0 ** -24 + 2.0 ** -20)
        y = ref
    assert np.all(np.abs(got - y) <= tol + 1e-30)
    buf[1:m + 1, 8:8 + cols] = 7
    assert torch.all(buf == 7)
