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
