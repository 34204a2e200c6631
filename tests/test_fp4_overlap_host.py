"""What the 4-bit calls and the sandwich norm write must share no byte with what
they read or write besides: refused before any CUDA call (the pointers are fake)."""
import ctypes as C

import pytest

from joint_video_audio_b200 import _binding as B
from tests.test_fp4_host import BAD, OK, _sandwich, fp4, needs_no_gpu, p

ROWS, HIDDEN = 10, 256
BYTES = ROWS * HIDDEN * 2
TABLE = 4 * 2 * 6 * HIDDEN * 4
INPUTS = {"y": BYTES, "post_gain": HIDDEN * 2, "tag": ROWS * 4, "tidx": ROWS * 4, "mod_table": TABLE, "norm_table": TABLE}
AT = {"x": 1, "y": 2, "post_gain": 3, "tag": 4, "tidx": 5, "mod_table": 6, "norm_table": 7}


def _round(n):
    return -(-n // 16) * 16


@needs_no_gpu
@pytest.mark.parametrize("out", ["x_out", "h"])
@pytest.mark.parametrize("name", INPUTS)
def test_sandwich_outputs_and_inputs(out, name):
    """The output's last 16 bytes on the input's first, and the other way round; next to one another they are fine."""
    at, n = p(AT[name]), _round(INPUTS[name])
    for ptr, status in ((at - BYTES + 16, BAD), (at + n - 16, BAD), (at - BYTES, OK), (at + n, OK)):
        assert B.h3blk_sandwich_norm(_sandwich(**{out: ptr}), None) == status, hex(ptr - at)


@needs_no_gpu
@pytest.mark.parametrize("part", ["codes", "scales", "row_scale"])
@pytest.mark.parametrize("name", [*AT, "x_out"])
def test_sandwich_4_bit_output_and_the_rest(part, name):
    at = p(AT.get(name, 8))
    q = fp4(ROWS, HIDDEN, at=10, **{part: at})
    assert B.h3blk_sandwich_norm(_sandwich(h=None, h_fp4=C.pointer(q)), None) == BAD


@needs_no_gpu
@pytest.mark.parametrize("a,b", [("codes", "scales"), ("codes", "row_scale"), ("scales", "row_scale")])
def test_parts_of_a_written_matrix(a, b):
    q = fp4(ROWS, HIDDEN, at=10, **{b: getattr(fp4(ROWS, HIDDEN, at=10), a)})
    assert B.h3blk_sandwich_norm(_sandwich(h=None, h_fp4=C.pointer(q)), None) == BAD
    assert B.h3blk_quantize_fp4(p(1), HIDDEN, 0, q, None) == BAD


@needs_no_gpu
def test_what_may_be_shared():
    """x_out may be x; one table may serve both purposes, and inputs may be one another."""
    assert B.h3blk_sandwich_norm(_sandwich(x_out=p(1), norm_table=p(6), y=p(1)), None) == BAD  # y is x, and x_out is written
    assert B.h3blk_sandwich_norm(_sandwich(x_out=p(1), norm_table=p(6)), None) == OK
    assert B.h3blk_sandwich_norm(_sandwich(y=p(1), tidx=p(4)), None) == OK
    assert B.h3blk_sandwich_norm(_sandwich(n_tags=2 ** 31 - 1, n_t=2 ** 31 - 1), None) == BAD  # no such table
