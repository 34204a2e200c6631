"""Reporting of waits that ran out in the 4-bit kernels: the host side, and, read
from the sources, that every kernel reports."""
import ctypes as C
import re

import pytest

from joint_video_audio_b200 import _binding as B
from tests.test_fp4_host import needs_no_gpu
from tests.test_warp_votes_host import _body


def test_refusals():
    assert B._lib.h3blk_fp4_check(None, None) == B.H3BLK_ERR_INVALID_ARG
    for ms in (0, -1, 2001):
        assert B.h3blk_selftest_fp4_wait(ms, None) == B.H3BLK_ERR_INVALID_ARG


@needs_no_gpu
def test_without_a_device():
    st = C.c_int(77)
    assert B._lib.h3blk_fp4_check(None, C.byref(st)) == B.H3BLK_ERR_CUDA and st.value == 77
    with pytest.raises(B.H3BlkError):
        B.h3blk_fp4_check(None)


@pytest.mark.parametrize("name", ["fp4.cu", "sandwich.cu"])
def test_row_passes_report_before_they_stop(name):
    bodies = [k for k in _body(name) if "fail[par]" in k]
    assert bodies
    for kernel in bodies:
        stop = kernel[kernel.index("if (fail[par]) {"):]
        assert re.match(r"[^}]*atomicOr\((a\.)?err, kErrTimeoutStream\);", stop)


def test_products_report_where_they_set_the_abort_word():
    text = "".join(_body("gemm_fp4.cu"))
    assert not re.search(r"\*v?abort = 1;", text)
    assert len(re.findall(r"give_up\(v?abort, p\.err\);", text)) >= 8
