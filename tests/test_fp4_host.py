"""Host-side checks of the 4-bit and sandwich-norm entry points: every bad
argument is refused before any CUDA call (the pointers are fake)."""
import ctypes as C

import pytest
import torch

import joint_video_audio_b200 as j
from joint_video_audio_b200 import _binding as B

BASE = 1 << 40
OK = B.H3BLK_ERR_CUDA  # a well-formed call passes every check and fails at the first CUDA call (no device here)
BAD, UNS = B.H3BLK_ERR_INVALID_ARG, B.H3BLK_ERR_UNSUPPORTED
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers")


def fp4(rows=64, K=256, format=B.H3BLK_FP4_NV, at=0, **kw):
    d = dict(codes=BASE + (at << 36), scales=BASE + (at << 36) + (1 << 34), row_scale=BASE + (at << 36) + (1 << 35))
    d.update(kw)
    return B.h3blk_fp4(format=format, K=K, rows=rows, **d)


def p(k):
    return BASE + (k << 36)


@pytest.mark.parametrize("fmt,rows,k,want", [(0, 1, 32, (16, 512, 4)), (1, 1, 32, (16, 512, 4)), (0, 128, 128, (8192, 512, 512)),
                                             (1, 129, 160, (129 * 80, 2 * 3 * 512, 516)), (0, 129, 160, (129 * 80, 2 * 2 * 512, 516)),
                                             (1, 0, 32, (0, 0, 0))])
def test_bytes(fmt, rows, k, want):
    assert B.h3blk_fp4_bytes(fmt, rows, k) == want


@pytest.mark.parametrize("fmt,rows,k", [(2, 1, 32), (-1, 1, 32), (0, -1, 32), (0, 1, 0), (0, 1, 48), (0, 1, -32)])
def test_bytes_refusals(fmt, rows, k):
    with pytest.raises(B.H3BlkError) as e:
        B.h3blk_fp4_bytes(fmt, rows, k)
    assert e.value.status == BAD


@needs_no_gpu
@pytest.mark.parametrize("args,q,status", [
    ({}, {}, OK), ({"ld": 264}, {}, OK), ({"rot": 1}, {}, OK), ({}, {"rows": 0}, OK),
    ({"x": 0}, {}, BAD), ({"x": BASE + 8}, {}, BAD), ({"ld": 248}, {}, BAD), ({"ld": 260}, {}, BAD),
    ({"rot": 1, "ld": 512}, {"K": 288}, BAD), ({}, {"K": 0}, BAD), ({}, {"K": 40}, BAD), ({}, {"format": 2}, BAD),
    ({}, {"rows": -1}, BAD), ({}, {"codes": 0}, BAD), ({}, {"scales": p(2) + 8}, BAD), ({}, {"row_scale": 0}, BAD),
    ({"ld": 32768}, {"K": 16416}, UNS), ({}, {"rows": (1 << 30) + 1}, UNS), ({}, {"codes": p(1) + 64 * 512 - 16}, BAD),
])
def test_quantize_refusals(args, q, status):
    a = {"x": p(1), "ld": 256, "rot": 0, **args}
    assert B.h3blk_quantize_fp4(a["x"], a["ld"], a["rot"], fp4(at=2, **q), None) == status
    assert B.h3blk_quantize_fp4(a["x"], a["ld"], a["rot"], None, None) == BAD


@needs_no_gpu
@pytest.mark.parametrize("out,ld,typ,status", [(p(1), 256, 0, OK), (p(1), 264, 1, OK), (0, 256, 0, BAD), (p(1) + 8, 256, 0, BAD),
                                               (p(1), 252, 0, BAD), (p(1), 248, 0, BAD), (p(1), 256, 2, BAD), (p(2), 256, 0, BAD)])
def test_dequantize_refusals(out, ld, typ, status):
    assert B.h3blk_dequantize_fp4(fp4(at=2), typ, out, ld, None) == status


@needs_no_gpu
@pytest.mark.parametrize("a,b,kw,status", [
    ({}, {}, {}, OK), ({"rows": 1}, {"rows": 8}, {"ld": 8}, OK), ({}, {"rows": 512}, {"epi": 1, "ld": 256}, OK),
    ({}, {"K": 288}, {}, BAD), ({}, {"format": 0}, {}, BAD), ({}, {"rows": 0}, {}, BAD), ({}, {"rows": 4}, {}, UNS),
    ({}, {"rows": 384}, {"epi": 1}, UNS), ({}, {}, {"epi": 2}, BAD), ({}, {}, {"typ": 2}, BAD), ({}, {}, {"out": 0}, BAD),
    ({}, {}, {"out": p(1) + 4}, BAD), ({}, {}, {"ld": 120}, BAD), ({}, {}, {"ld": 132}, BAD), ({}, {}, {"out": p(2)}, BAD), ({"rows": 1}, {}, {"ld": (1 << 36) + 8}, UNS),
    ({}, {}, {"out": p(3) + (1 << 34)}, BAD), ({"codes": 0}, {}, {}, BAD), ({}, {"row_scale": p(3) + 4}, {}, BAD),
])
def test_gemm_refusals(a, b, kw, status):
    k = {"epi": 0, "typ": 0, "out": p(1), "ld": 128, **kw}
    st = B.h3blk_gemm_fp4(fp4(at=2, **a), fp4(at=3, **{"rows": 128, **b}), k["epi"], k["typ"], k["out"], k["ld"], None)
    assert st == status


def _sandwich(**kw):
    d = dict(n_rows=10, hidden=256, n_tags=4, n_t=2, branch=0, post_norm=1, post_eps=1e-5, norm_eps=1e-5,
             branch_scale=1.0, x=p(1), y=p(2), post_gain=p(3), tag=p(4), tidx=p(5), mod_table=p(6), norm_table=p(7),
             x_out=p(8), h=p(9), h_fp4=None, rotate=0)
    d.update(kw)
    return B.h3blk_sandwich(**d)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    ({}, OK), ({"branch": 1}, OK), ({"post_gain": None}, OK), ({"post_norm": 0, "post_gain": None}, OK), ({"x_out": p(1)}, OK),
    ({"norm_table": None, "h": None}, OK), ({"n_rows": 0}, OK), ({"h": None, "h_fp4": C.pointer(fp4(10, 256, at=10))}, OK),
    ({"n_rows": -1}, BAD), ({"hidden": 0}, BAD), ({"branch": 2}, BAD), ({"x": None}, BAD), ({"y": p(2) + 8}, BAD),
    ({"post_norm": 0}, BAD), ({"h": None}, BAD), ({"norm_table": None}, BAD), ({"h_fp4": C.pointer(fp4(10, 256, at=10))}, BAD),
    ({"h": None, "h_fp4": C.pointer(fp4(9, 256, at=10))}, BAD), ({"h": None, "h_fp4": C.pointer(fp4(10, 128, at=10))}, BAD),
    ({"post_eps": -1.0}, BAD), ({"norm_eps": float("nan")}, BAD), ({"x_out": p(2)}, BAD), ({"x_out": p(1) + 512}, BAD),
    ({"h": p(8)}, BAD), ({"h": p(1)}, BAD), ({"hidden": 192}, UNS), ({"hidden": 16512}, UNS), ({"n_t": 0}, BAD), ({"rotate": 1}, BAD),
    ({"h": None, "h_fp4": C.pointer(fp4(10, 256, at=10, codes=p(2)))}, BAD),
])
def test_sandwich_refusals(kw, status):
    assert B.h3blk_sandwich_norm(_sandwich(**kw), None) == status


def test_null_structs():
    assert B._lib.h3blk_sandwich_norm(None, None) == BAD
    assert B._lib.h3blk_gemm_fp4(None, None, 0, 0, p(1), 128, None) == BAD
    assert B._lib.h3blk_dequantize_fp4(None, 0, p(1), 128, None) == BAD


def test_python_refusals():
    cpu = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        j.quantize_fp4(cpu)
    with pytest.raises(ValueError):
        j.Fp4Tensor(4, 256, "fp8", device="cpu")
    a, b = j.Fp4Tensor(4, 256, "nv", device="cpu"), j.Fp4Tensor(8, 256, "mx", device="cpu")
    assert a.codes.shape == (4, 128) and a.scales.shape == (4, 512) and a.row_scale.shape == (4,)
    with pytest.raises(ValueError):
        j.gemm_fp4(a, b)
    with pytest.raises(ValueError):
        j.dequantize_fp4(a, torch.float16)
    c, d = j.Fp4Tensor(4, 256, "nv", device="cpu"), j.Fp4Tensor(8, 256, "nv", device="cpu")
    for call in (lambda: j.gemm_fp4(c, d), lambda: j.dequantize_fp4(c)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    d.rotated = True
    with pytest.raises(ValueError, match="rotated"):
        j.gemm_fp4(c, d)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        j.sandwich_norm(cpu, cpu, i, i, torch.zeros(4, 2, 6, 256))
    for kw in ({"h": "fp8"}, {"h": "bf16", "rotate": True}, {"h": None, "rotate": True}):
        with pytest.raises(ValueError):
            j.sandwich_norm(cpu, cpu, i, i, torch.zeros(4, 2, 6, 256), **kw)


def test_python_refuses_what_is_no_tensor_or_does_not_fit():
    with pytest.raises(TypeError, match="Tensor"):
        j.quantize_fp4([1.0])
    with pytest.raises(ValueError, match="fmt"):
        j.quantize_fp4(torch.zeros(2, 32, dtype=torch.bfloat16), "fp8")
    q = j.Fp4Tensor(4, 256, "nv", device="cpu")
    with pytest.raises(ValueError, match="out"):
        j.quantize_fp4(torch.zeros(4, 128, dtype=torch.bfloat16), out=q)
    with pytest.raises(j.H3BlkError):
        j.Fp4Tensor(4, 100, "nv", device="cpu")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="tag"):
        j.sandwich_norm(torch.zeros(4, 256), torch.zeros(4, 256), None, i, torch.zeros(4, 2, 6, 256))
    with pytest.raises(ValueError, match="hidden"):
        j.sandwich_norm(torch.zeros(4, 256), torch.zeros(4, 256), i, i, torch.zeros(4, 2, 256))


def test_refused_calls_keep_no_references():
    import sys
    from joint_video_audio_b200 import fp4 as F
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, i, t = j.Fp4Tensor(4, 256, "nv", device="cpu"), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 6, 256)
    held = (x, q, q.buffer, i, t, j.H3BlkError)
    before = [sys.getrefcount(o) for o in held]
    for _ in range(50):
        for call in (lambda: j.quantize_fp4(x), lambda: j.gemm_fp4(q, q), lambda: j.dequantize_fp4(q, out=x),
                     lambda: j.sandwich_norm(x, x, i, i, t), lambda: F._host.layout(0, 4, 33), lambda: F._host.layout(0, 4),
                     lambda: F._host.layout("mx", 4, 32)):
            with pytest.raises((ValueError, TypeError, j.H3BlkError)):
                call()
    assert [sys.getrefcount(o) for o in held] == before
