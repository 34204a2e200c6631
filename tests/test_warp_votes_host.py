"""Read from the sources, without a GPU: what a whole warp does together must not
hang on a wait that each lane decides by itself. Pipeline waits are bounded; where
one runs out while its barrier flips, some lanes would go on and some not, and
tensor-memory reads and cluster barriers (`.aligned`) are defined for whole warps only."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "joint_video_audio_b200", "csrc")
SOURCES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")))
KERNELS = [s for s in SOURCES if "tmem_ld" in open(os.path.join(CSRC, s)).read()]


def _body(name):
    """The kernels of a source without comments (device functions defined behind one are cut off)."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    return [part.split("__device__ __forceinline__ void", 1)[0] for part in re.split(r"__global__", text)[1:]]


def test_the_sources_are_found():
    assert {"attn.cu", "gemm.cu", "gemm_fp4.cu"} <= set(KERNELS)


@pytest.mark.parametrize("name", KERNELS)
def test_accumulators_are_read_behind_a_vote(name):
    """The wait in front of each tensor-memory read (epilogue_tile reads them in
    gemm.cu) is one whose outcome is the same in every lane."""
    reads = 0
    for kernel in _body(name):
        waits = [(m.start(), m.group(0)) for m in re.finditer(r"__all_sync\(0xffffffffu, mbar_wait\w*\(|mbar_wait\w*\(", kernel)]
        for m in re.finditer(r"\b(tmem_ld\w+|epilogue_tile)(<[^;]*?>)?\(", kernel):
            before = [w for at, w in waits if at < m.start()]
            assert before, f"{name}: {m.group(1)} without a wait"
            assert before[-1].startswith(("mbar_wait_warp(", "__all_sync(")), f"{name}: {m.group(1)} behind {before[-1]}"
            reads += 1
    assert reads


@pytest.mark.parametrize("name", KERNELS)
def test_warps_are_whole_at_a_closing_cluster_barrier(name):
    """Behind the roles, whose single lanes loop by themselves, a __syncwarp
    comes first, with nothing in between that a lane might do alone."""
    for kernel in _body(name):
        for m in re.finditer(r"cluster_sync(_relaxed)?\(\);", kernel):
            head = kernel[:m.start()]
            if "warp == 0" not in head.replace("warp == 0 && lane == 0", ""):
                continue  # before the roles
            tail = head[head.rfind("__syncwarp()"):]
            assert "__syncwarp()" in head and "lane == 0" not in tail, f"{name}: {m.group(0)}"


def test_the_abort_word_is_set_by_waits_alone():
    """Every wait that succeeds passes over the abort word, so that setting it
    stops nothing by itself: it is for those that gave up. The pair kernel's base
    address 0 rests on its allocating all 512 columns, not on such a check."""
    text = open(os.path.join(CSRC, "gemm_fp4.cu")).read()
    assert "tmem_alloc_pair(tmem_slot, 512)" in text
    for kernel in _body("gemm_fp4.cu"):
        assert not re.search(r"if \(\*tmem_slot[^)]*\) \*?\w*abort", kernel)
