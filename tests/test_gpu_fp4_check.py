"""A wait of the 4-bit kernels that runs out is reported to the host, without a GPU
fault: the wait here is one of a kernel for this test alone, 50 ms long, which
records it as theirs do."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def j():
    assert torch.cuda.is_available(), "GPU tests need a B200"
    import joint_video_audio_b200
    return joint_video_audio_b200


@pytest.fixture(scope="module")
def x():
    return torch.randn(70, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()


def _calls(j, x):
    i, t = torch.zeros(70, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, 6, 256, device="cuda")
    q = j.quantize_fp4(x)
    return j.gemm_fp4(q, j.quantize_fp4(x[:64])), j.dequantize_fp4(q), j.sandwich_norm(x, x, i, i, t)[1]


def _late(j, stream=None):
    s = stream or torch.cuda.current_stream()
    assert j.capi.h3blk_selftest_fp4_wait(50, s.cuda_stream) == j.H3BLK_OK


def test_calls_that_end_well(j, x):
    assert j.check_fp4() == j.H3BLK_OK
    _calls(j, x)
    assert j.check_fp4() == j.H3BLK_OK


def test_a_wait_that_runs_out(j, x):
    """Seen once, whatever ran before or behind it; the calls go on working."""
    ref = _calls(j, x)
    _late(j)
    again = _calls(j, x)
    assert j.check_fp4() == j.capi.H3BLK_ERR_TIMEOUT
    assert j.check_fp4(torch.device("cuda", torch.cuda.current_device())) == j.H3BLK_OK
    assert all(torch.equal(a, b) for a, b in zip(ref, again))


def test_on_another_stream_and_in_a_graph(j, x):
    s = torch.cuda.Stream()
    _late(j, s)
    s.synchronize()
    assert j.check_fp4() == j.capi.H3BLK_ERR_TIMEOUT
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _late(j)
        out = _calls(j, x)
    assert j.check_fp4() == j.H3BLK_OK  # captured, not run
    for _ in range(2):
        g.replay()
        assert j.check_fp4() == j.capi.H3BLK_ERR_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(out, _calls(j, x)))
    assert j.check_fp4() == j.H3BLK_OK


def test_the_first_call_of_a_process_may_be_captured():
    code = """
import torch
import joint_video_audio_b200 as j
x = torch.randn(8, 256, device="cuda").to(torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q = j.quantize_fp4(x)
    v = j.dequantize_fp4(q)
    y = j.gemm_fp4(q, q)
g.replay()
torch.cuda.synchronize()
assert torch.equal(v, j.dequantize_fp4(j.quantize_fp4(x))) and torch.equal(y, j.gemm_fp4(q, q))
assert j.check_fp4() == j.H3BLK_OK
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
