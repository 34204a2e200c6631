"""Sandwich norm on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import h3_fp4 as o
from tests.test_gpu_fp4 import _tolerance, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def j():
    assert torch.cuda.is_available(), "GPU tests need a B200"
    import joint_video_audio_b200
    return joint_video_audio_b200


def _case(n, c, seed, n_tags=4, n_t=2):
    g = torch.Generator().manual_seed(seed)
    d = {"x": torch.randn(n, c, generator=g).to(torch.bfloat16),
         "y": (torch.randn(n, c, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).to(torch.bfloat16),
         "tag": torch.randint(-1, n_tags, (n,), generator=g, dtype=torch.int32),
         "tidx": torch.randint(0, n_t, (n,), generator=g, dtype=torch.int32),
         "table": 0.4 * torch.randn(n_tags, n_t, 6, c, generator=g),
         "next": 0.4 * torch.randn(n_tags, n_t, 6, c, generator=g),
         "gain": (1 + 0.1 * torch.randn(c, generator=g)).to(torch.bfloat16)}
    if n > 3:
        d["y"][1] = 0
        d["x"][2] = 0
        d["y"][2] = 0
    return d


def _run(j, d, branch, post, gain=True, **kw):
    c = {k: v.cuda() for k, v in d.items()}
    return j.sandwich_norm(c["x"], c["y"], c["tag"], c["tidx"], c["table"], branch=branch, next_table=c["next"],
                           post_norm=post, post_gain=c["gain"] if post and gain else None, branch_scale=0.7, **kw)


def _ref(d, branch, post, gain=True):
    n = {k: v.float().numpy() for k, v in d.items()}
    return o.sandwich(n["x"], n["y"], d["tag"], d["tidx"], n["table"], branch, n["next"], post,
                      n["gain"] if post and gain else None, branch_scale=0.7)


def _check(d, got_x, got_h, x1, h):
    """fp32 arithmetic: the reductions over at most 16384 squares are good to
    2^-18 (32 in a thread, then trees), x1 adds two terms of its size; then
    one rounding to bf16."""
    half = torch.finfo(torch.bfloat16).eps / 2
    xs = np.abs(d["x"].double().numpy())
    gx = got_x.double().cpu().numpy()
    assert np.all(np.abs(gx - x1) <= half * np.abs(x1) + 2.0 ** -18 * (2 * xs + np.abs(x1)) + 1e-30)
    if h is not None:
        gh = got_h.double().cpu().numpy()
        rms = np.sqrt(np.mean(x1 * x1, -1, keepdims=True) + 1e-5)
        lim = half * np.abs(h) + 2.0 ** -17 * (np.abs(h) + 2 + 3 * (2 * xs + np.abs(x1)) / rms)
        assert np.all(np.abs(gh - h) <= lim)


@pytest.mark.parametrize("n,c", [(1, 128), (2, 256), (9, 384), (300, 1024), (33, 1152), (65, 2176), (31, 5376), (5, 16384), (40, 2048), (7, 5632),
                                 (9, 8192)])
@pytest.mark.parametrize("branch", [0, 1])
@pytest.mark.parametrize("post", [False, True])
def test_sandwich(j, n, c, branch, post):
    d = _case(n, c, n + c + branch)
    x1, h = _run(j, d, branch, post)
    _check(d, x1, h, *_ref(d, branch, post))


def test_many_rows_and_no_gain(j):
    d = _case(5000, 640, 8)
    x1, h = _run(j, d, 1, True, gain=False)
    _check(d, x1, h, *_ref(d, 1, True, gain=False))


def test_runs_of_one_key(j):
    """Rows packed in runs, as a sequence is, and every row of one key."""
    for fill in (None, 3):
        d = _case(2500, 768, 11)
        d["tag"] = torch.sort(d["tag"])[0].flip(0).contiguous() if fill is None else torch.full_like(d["tag"], fill)
        d["tidx"] = (d["tag"] == 2).to(torch.int32)
        x1, h = _run(j, d, 0, True)
        _check(d, x1, h, *_ref(d, 0, True))


def test_padding_and_bad_indices_pass_through(j):
    d = _case(40, 512, 3)
    d["tag"][:6] = torch.tensor([-1, 4, -2, 2 ** 31 - 1, 0, 1])
    d["tidx"][4:6] = torch.tensor([2, -1])
    x1, h = _run(j, d, 0, True)
    assert torch.equal(x1[:6].cpu(), d["x"][:6])
    _check(d, x1, h, *_ref(d, 0, True))


def test_no_h_and_in_place(j):
    d = _case(70, 1280, 6)
    ref_x, ref_h = _run(j, d, 1, True)
    x1, h = _run(j, d, 1, True, h=None)
    assert h is None and torch.equal(x1, ref_x)
    x1, h = j.sandwich_norm(*(d[k].cuda() for k in ("x", "y", "tag", "tidx", "table")), branch=1,
                            post_gain=d["gain"].cuda(), branch_scale=0.7)  # the last layer has no next table
    assert h is None and torch.equal(x1, ref_x)
    c = {k: v.cuda() for k, v in d.items()}
    x = c["x"]
    x1, h = j.sandwich_norm(x, c["y"], c["tag"], c["tidx"], c["table"], branch=1, next_table=c["next"],
                            post_gain=c["gain"], branch_scale=0.7, x_out=x)
    assert x1 is x and torch.equal(x, ref_x) and torch.equal(h, ref_h)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("n,c", [(3, 128), (130, 1024), (37, 5376), (2, 16384)])
def test_h_in_4_bits(j, fmt, rotate, n, c):
    """Each stored code is a nearest one of the exact h up to fp32 noise (2^-17
    of the row's largest, seven stages more when rotated), and the scales are
    those of the exact h wherever the noise cannot change them."""
    d = _case(n, c, c + n)
    x1, q = _run(j, d, 0, True, h=fmt, rotate=rotate)
    rx, rh = _ref(d, 0, True)
    _check(d, x1, None, rx, None)
    codes, sc, row = unpack(q, c // o.BLOCK[fmt])
    rc, rs, rr, _ = o.quantize(rh, fmt, rotate)
    assert np.mean(sc == rs) > 0.995 and np.mean(codes == rc) > 0.995
    same = np.repeat((sc == rs) & (np.abs(row / rr - 1) < 1e-6)[:, None], o.BLOCK[fmt], 1)
    flat = o.rotate(rh) / 128 ** 0.5 if rotate else rh
    v, step = o.values(codes, sc, row, fmt), o.values(np.full_like(codes, 2), sc, row, fmt)  # step: the block's 1.0
    noise = 2.0 ** -15 * np.abs(flat).max(-1, keepdims=True)
    ref = o.values(rc, rs, rr, fmt)
    assert np.all(np.abs(v - flat)[same] <= (np.abs(ref - flat) + 2 * noise)[same])
    assert np.all(np.abs(v - flat) <= 2.2 * step + noise)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_h_in_4_bits_is_the_quantised_h(j, fmt):
    """Against the two steps one after the other, over more rows than CTAs: the
    only difference is h's rounding to bf16 in between, half a step of 2^-8,
    which moves a code by one at most and a scale by one of its steps. Where it
    carries a row's largest past 2688 * 2^E, the NV row scale doubles and every
    block scale halves with it, which is 8 codes of e4m3 (three mantissa bits)
    and says nothing about a step: such rows are few and left out."""
    d = _case(3000, 640, 21)
    x1, h = _run(j, d, 0, True)
    x2, q = _run(j, d, 0, True, h=fmt)
    assert torch.equal(x1, x2)
    two = j.quantize_fp4(h, fmt)
    b = 640 // o.BLOCK[fmt]
    (c1, s1, r1), (c2, s2, r2) = unpack(q, b), unpack(two, b)
    assert np.mean(r1 != r2) < 0.01 and np.all((r1 / r2 >= 0.5) & (r1 / r2 <= 2))
    assert np.abs(s1.astype(int) - s2)[r1 == r2].max() <= 1
    same = np.repeat((s1 == s2) & (r1 == r2)[:, None], o.BLOCK[fmt], 1)
    mag1, mag2 = (c1 & 7).astype(int), (c2 & 7).astype(int)
    assert same.mean() > 0.9 and np.abs(mag1 - mag2)[same].max() <= 1 and (c1 == c2)[same].mean() > 0.97


@pytest.mark.parametrize("fmt,rotate", [("mx", False), ("nv", True)])
@pytest.mark.parametrize("n", [5, 300])
def test_feed_forward_half_of_the_block_in_4_bits(j, fmt, rotate, n):
    """The operators as a step uses them: the sandwich norm after attention, FFN
    up with SwiGLU, its output to 4 bits, FFN down, the sandwich norm of the
    next layer; each stage against the oracle from the GPU's own input to it.
    The whole is captured into a graph and replayed with the same result."""
    c, f = 512, 1024
    d = _case(n, c, 77)
    g = torch.Generator().manual_seed(5)
    w13 = j.quantize_fp4((torch.randn(2 * f, c, generator=g) / c ** 0.5).to(torch.bfloat16).cuda(), fmt, rotate=rotate)
    w2 = j.quantize_fp4((torch.randn(c, f, generator=g) / f ** 0.5).to(torch.bfloat16).cuda(), fmt, rotate=rotate)
    t = {k: v.cuda() for k, v in d.items()}

    def step():
        x1, h = j.sandwich_norm(t["x"], t["y"], t["tag"], t["tidx"], t["table"], post_gain=t["gain"], h=fmt, rotate=rotate)
        a = j.gemm_fp4(h, w13, swiglu=True)
        qa = j.quantize_fp4(a, fmt, rotate=rotate)
        y = j.gemm_fp4(qa, w2)
        x2, h2 = j.sandwich_norm(x1, y, t["tag"], t["tidx"], t["table"], branch=1, next_table=t["next"], post_norm=False)
        return x1, h, a, qa, y, x2, h2

    x1, h, a, qa, y, x2, h2 = step()
    val = lambda q: j.dequantize_fp4(q, torch.float32).double().cpu().numpy()  # noqa: E731
    vh, v13, vqa, v2 = val(h), val(w13), val(qa), val(w2)
    up = o.product(vh, v13)
    tol = _tolerance(vh, v13, torch.float32, up)
    ref = o.product(vh, v13, True)
    lim = 1.1 * tol[:, :f] * np.abs(up[:, f:]) + np.abs(o.silu(up[:, :f])) * tol[:, f:] + np.abs(ref) * (2.0 ** -8 + 2.0 ** -20)
    assert np.all(np.abs(a.double().cpu().numpy() - ref) <= lim + 1e-30)
    ref = vqa @ v2.T
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= _tolerance(vqa, v2, torch.bfloat16, ref))
    d2 = dict(d, x=x1.cpu(), y=y.cpu())
    n2 = {k: v.float().numpy() for k, v in d2.items()}
    _check(d2, x2, h2, *o.sandwich(n2["x"], n2["y"], d["tag"], d["tidx"], n2["table"], 1, n2["next"], False))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    graph.replay()
    assert torch.equal(again[5], x2) and torch.equal(again[6], h2)


@pytest.mark.parametrize("h", ["bf16", "mx"])
def test_offsets_past_32_bits(j, h):
    """420 repeats of 1000 rows, more than 2^31 values in each tensor: every
    repeat gives the bits of the first, and those of the 1000 rows alone."""
    reps, n, c = 420, 1000, 5376
    assert reps * n * c > 2 ** 31
    d = _case(n, c, 31)
    x1, h1 = _run(j, d, 0, True, h=h)
    long = dict(d, **{k: d[k].cuda().repeat(reps, *[1] * (d[k].dim() - 1)) for k in ("x", "y", "tag", "tidx")})
    xl, hl = _run(j, long, 0, True, h=h)
    assert torch.equal(xl.view(reps, -1), x1.view(1, -1).expand(reps, -1))
    if h == "bf16":
        assert torch.equal(hl.view(reps, -1), h1.view(1, -1).expand(reps, -1))
    else:
        assert torch.equal(hl.codes.view(reps, -1), h1.codes.view(1, -1).expand(reps, -1))
        assert torch.equal(hl.row_scale.view(reps, -1), h1.row_scale.expand(reps, -1))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("n", [1, 40, 600, 3000])
def test_back_to_back_calls_in_the_same_buffers(j, n, graph):
    """A kernel starts its set-up while the one before it ends. Calls in a row
    that write what the one before reads and read what it writes, with a torch
    kernel or a copy between them at times, give the bits of the same calls one
    at a time."""
    c, f = 512, 1024
    d = {k: v.cuda() for k, v in _case(n, c, 41).items()}
    g = torch.Generator().manual_seed(42)
    up = j.quantize_fp4((torch.randn(f, c, generator=g) / 23).to(torch.bfloat16).cuda(), "nv")
    down = j.quantize_fp4((torch.randn(c, f, generator=g) / 32).to(torch.bfloat16).cuda(), "nv")

    def run(wait):
        x, y = d["x"].clone(), d["y"].clone()
        a, h = torch.empty(n, f, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
        qh, qa = j.Fp4Tensor(n, c, "nv"), j.Fp4Tensor(n, f, "nv")
        seen = []
        for i in range(6):
            for step in (lambda: h.copy_(j.sandwich_norm(x, y, d["tag"], d["tidx"], d["table"], branch_scale=0.5, x_out=x)[1]),
                         lambda: j.quantize_fp4(h, "nv", out=qh),
                         lambda: j.gemm_fp4(qh, up, out=a),
                         lambda: j.quantize_fp4(a, "nv", out=qa),
                         lambda: j.gemm_fp4(qa, down, out=y),
                         lambda: a.zero_() if i % 2 else j.dequantize_fp4(qa, out=a),
                         lambda: j.quantize_fp4(y, "nv", out=qh),
                         lambda: j.dequantize_fp4(qh, out=y)):
                step()
                if wait:
                    torch.cuda.synchronize()
            seen.append((x + 0, y + 0, a + 0))
        return seen

    ref = run(True)
    if graph:
        run(False)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run(False)
        for _ in range(3):
            g.replay()
    else:
        got = [run(False) for _ in range(3)][-1]
    torch.cuda.synchronize()
    for r, s in zip(ref, got):
        assert all(torch.equal(u, v) for u, v in zip(r, s))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("n", [20, 2000])
def test_streams_that_wait_for_one_another(j, n, graph):
    """One stream makes inputs slowly, another one works on them behind an
    event, and the first overwrites them behind an event of the second: a
    kernel that starts early still waits for the events before it."""
    c, steps = 512, 5
    g = torch.Generator().manual_seed(51)
    xs = [torch.randn(n, c, generator=g).to(torch.bfloat16).cuda() for _ in range(steps)]
    slow = torch.randn(2048, 2048, generator=g).cuda()
    w = j.quantize_fp4((torch.randn(c, c, generator=g) / 23).to(torch.bfloat16).cuda(), "nv")
    refs = [j.gemm_fp4(j.quantize_fp4(x, "nv"), w) for x in xs]
    torch.cuda.synchronize()

    def run(s1, s2):
        buf, q = torch.zeros(n, c, dtype=torch.bfloat16, device="cuda"), j.Fp4Tensor(n, c, "nv")
        outs = [torch.zeros(n, c, dtype=torch.bfloat16, device="cuda") for _ in xs]
        s2.wait_stream(s1)
        for x, y in zip(xs, outs):
            acc = slow
            for _ in range(4):
                acc = acc @ slow * 0.01
            buf.copy_(x)
            buf += (acc[0, 0] * 0).nan_to_num().to(torch.bfloat16)  # behind the products
            s2.wait_stream(s1)
            with torch.cuda.stream(s2):
                j.quantize_fp4(buf, "nv", out=q)
            s1.wait_stream(s2)
            buf.fill_(float("nan"))
            with torch.cuda.stream(s2):
                j.gemm_fp4(q, w, out=y)
            s2.wait_stream(s1)
        s1.wait_stream(s2)
        return outs, buf, q

    s2 = torch.cuda.Stream()
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            keep = run(torch.cuda.current_stream(), s2)
        for _ in range(3):
            cg.replay()
    else:
        keep = run(torch.cuda.current_stream(), s2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep[0], refs))
