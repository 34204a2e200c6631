"""Calls of one kernel from several threads at once, each on its own stream and
with rows of its own width. The shared memory that a launch asks for goes by the
width, and the limit that allows it is the kernel's, shared by every thread: a call
must not lower it under another one that is about to launch."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

CALLS = 300


@pytest.fixture(scope="module")
def j():
    assert torch.cuda.is_available(), "GPU tests need a B200"
    import joint_video_audio_b200
    return joint_video_audio_b200


def _in_threads(calls):
    """Every call CALLS times in a thread of its own; its outputs have to be those of a call alone."""
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    errors = []

    def work(call, ref):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for i in range(CALLS):
                try:
                    out = call()
                except Exception as e:  # reported by the test's thread
                    errors.append(repr(e))
                    continue
                if i % 50 == 0 and not all(torch.equal(a, b) for a, b in zip(out, ref)):
                    errors.append("another result")
        s.synchronize()

    threads = [threading.Thread(target=work, args=p) for p in zip(calls, refs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads)
    assert not errors, f"{len(errors)} of {CALLS * len(calls)}: {errors[0]}"


def _rows(rows, k):
    return torch.randn(rows, k, generator=torch.Generator().manual_seed(k)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_of_several_widths(j, fmt):
    def call(x):
        q = j.quantize_fp4(x, fmt)
        return q.codes, q.row_scale

    _in_threads([lambda x=_rows(4, k): call(x) for k in (7168, 14336, 5376, 16384)])


@pytest.mark.parametrize("h", ["bf16", "nv"])
def test_sandwich_norm_of_several_widths(j, h):
    def call(x, i, table):
        x1, out = j.sandwich_norm(x, x, i, i, table, h=h)
        return x1, out if h == "bf16" else out.codes

    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    _in_threads([lambda x=_rows(4, c), t=0.3 * torch.ones(1, 1, 6, c, device="cuda"): call(x, i, t)
                 for c in (2176, 5376, 3968, 4096)])


def test_rotate_quantize_of_several_widths(j):
    _in_threads([lambda x=_rows(4, k): j.rotate_quantize(x) for k in (7168, 14336, 5376, 16384)])


def test_products_of_every_kernel_at_once(j):
    """One row with split sums, 40 rows of SwiGLU, 128 unsplit and the pair kernel's
    many, each behind its own quantisation, which their set-up overlaps, and one
    thread of sandwich norms into a product."""
    g = torch.Generator().manual_seed(3)

    def product(m, n, k, swiglu):
        x = torch.randn(m, k, generator=g).to(torch.bfloat16).cuda()
        w = j.quantize_fp4((torch.randn(n, k, generator=g) / k ** 0.5).to(torch.bfloat16).cuda())
        return lambda: (j.gemm_fp4(j.quantize_fp4(x), w, swiglu=swiglu),)

    def chain():
        x = torch.randn(300, 1024, generator=g).to(torch.bfloat16).cuda()
        i, t = torch.zeros(300, dtype=torch.int32, device="cuda"), (0.3 * torch.randn(1, 1, 6, 1024, generator=g)).cuda()
        w = j.quantize_fp4((torch.randn(512, 1024, generator=g) / 32).to(torch.bfloat16).cuda(), "mx")

        def call():
            x1, h = j.sandwich_norm(x, x, i, i, t, h="mx")
            return x1, j.gemm_fp4(h, w)

        return call

    _in_threads([product(1, 1024, 5376, False), product(40, 2048, 2048, True), product(128, 21504, 512, False),
                 product(2000, 1536, 768, True), chain()])
    assert j.check_fp4() == j.H3BLK_OK
