"""torch-tensor marshalling of the 4-bit linear path and the sandwich norm
(no arithmetic here): include/h3blk.h states the formats and the formulas."""
from __future__ import annotations

from ctypes import addressof
from functools import lru_cache
from struct import Struct

import torch

from . import _binding as B

FORMATS = {"mx": B.H3BLK_FP4_MX, "nv": B.H3BLK_FP4_NV}
_OUT = {torch.bfloat16: B.H3BLK_BF16, torch.float32: B.H3BLK_F32}
_quantize, _dequantize = B._lib.h3blk_quantize_fp4, B._lib.h3blk_dequantize_fp4
_gemm, _sandwich = B._lib.h3blk_gemm_fp4, B._lib.h3blk_sandwich_norm
# h3blk_sandwich in its C layout: packing it takes 0.4 us, filling the ctypes structure 1.8 us
_pack_sandwich = Struct("@qiiiiifffPPPPPPPPPPi0P").pack
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _call(fn, i, *args):
    """The library call fn(*args, stream) on device i's current stream, with that device current."""
    if _current_device() == i:
        st = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = fn(*args, _raw_stream(i))
    if st:
        raise B.H3BlkError(fn.__name__, st)


def _rows(t: torch.Tensor, name: str, dtype=torch.bfloat16):
    """(rows, columns, row stride) of a 2-D CUDA tensor with unit column stride; ValueError otherwise."""
    if not t.is_cuda or t.dtype != dtype or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D {dtype} CUDA tensor, got {t.dtype} {tuple(t.shape)} on {t.device}")
    (rows, k), (ld, unit) = t.shape, t.stride()
    if unit != 1 and k > 1:
        raise ValueError(f"{name}: its rows are not contiguous")
    if rows < 2:
        return rows, k, -(-k // 8) * 8
    if ld < k or ld % 8:
        raise ValueError(f"{name}: row stride {ld} is not a multiple of 8 of at least {k}")
    return rows, k, ld


@lru_cache(maxsize=1024)
def _layout(rows: int, K: int, fmt: str):
    """(format code, byte lengths, offsets and total of the three parts), every part on a 256-byte boundary."""
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}, got {fmt!r}")
    lens = B.h3blk_fp4_bytes(FORMATS[fmt], rows, K)
    up = [-(-n // 256) * 256 for n in lens]
    return FORMATS[fmt], lens, (0, up[0], up[0] + up[1]), max(256, sum(up))


class Fp4Tensor:
    """A [rows, K] matrix in microscaled 4-bit floats on the GPU (h3blk_fp4).

    codes      uint8 [rows, K / 2], two e2m1 codes a byte
    scales     uint8 [..., 512] atoms of 128 rows x 4 block scales
    row_scale  fp32 [rows]
    rotated    whether the values went through the Hadamard rotation
    """

    __slots__ = ("fmt", "shape", "rotated", "buffer", "c", "ref")

    def __init__(self, rows: int, K: int, fmt: str = "nv", device="cuda"):
        code, _, (_, scales, row_scale), total = _layout(rows, K, fmt)
        self.fmt, self.shape, self.rotated = fmt, (rows, K), False
        self.buffer = buf = torch.empty(total, dtype=torch.uint8, device=device)
        p = buf.data_ptr()
        self.c = c = B.h3blk_fp4(code, K, rows, p, p + scales, p + row_scale)
        self.ref = addressof(c)

    def _part(self, i):
        _, lens, at, _ = _layout(*self.shape, self.fmt)
        return self.buffer[at[i]:at[i] + lens[i]]

    @property
    def device(self):
        return self.buffer.device

    @property
    def codes(self) -> torch.Tensor:
        return self._part(0).view(self.shape[0], self.shape[1] // 2)

    @property
    def scales(self) -> torch.Tensor:
        return self._part(1).view(-1, 512)

    @property
    def row_scale(self) -> torch.Tensor:
        return self._part(2).view(torch.float32)

    def __repr__(self):
        return f"Fp4Tensor({self.shape[0]}, {self.shape[1]}, {self.fmt!r}{', rotated' * self.rotated}, {self.device})"


def quantize_fp4(x: torch.Tensor, fmt: str = "nv", rotate: bool = False, out: Fp4Tensor | None = None) -> Fp4Tensor:
    """bf16 [rows, K] (rows may be strided) -> microscaled 4-bit floats.

    fmt "mx": blocks of 32 with power-of-two scales; "nv": blocks of 16 with
    e4m3 scales and a power-of-two scale per row. rotate: the block-128 Hadamard
    transform of the W8A8 path first (a product takes two rotated operands or
    two that are not). h3blk_quantize_fp4."""
    rows, K, ld = _rows(x, "x")
    if out is None:
        out = Fp4Tensor(rows, K, fmt, x.device)
    elif out.fmt != fmt or out.shape != (rows, K) or out.device != x.device:
        raise ValueError(f"out: expected {fmt} {(rows, K)} on {x.device}, got {out}")
    if rows:
        _call(_quantize, x.get_device(), x.data_ptr(), ld, rotate, out.ref)
    out.rotated = bool(rotate)
    return out


def dequantize_fp4(q: Fp4Tensor, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values `q` stands for, bf16 or fp32 [rows, K] (h3blk_dequantize_fp4)."""
    rows, K = q.shape
    out, ld = _output(out, rows, K, dtype, q.device)
    if rows:
        _call(_dequantize, out.get_device(), q.ref, _OUT[dtype], out.data_ptr(), ld)
    return out


def _output(out, rows, cols, dtype, device):
    """(output tensor, its row stride), made here where none is given; a
    stride that is no multiple of 8 (columns that are not) is the library's to refuse."""
    if dtype not in _OUT:
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    if device.type != "cuda":
        raise ValueError(f"expected operands on a CUDA device, got {device}")
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=device), cols
    if tuple(out.shape) != (rows, cols) or out.dtype != dtype or out.device != device:
        raise ValueError(f"out: expected {dtype} {(rows, cols)} on {device}, got {out.dtype} {tuple(out.shape)} on {out.device}")
    return out, _rows(out, "out", dtype)[2]


def gemm_fp4(a: Fp4Tensor, b: Fp4Tensor, swiglu: bool = False, dtype=torch.bfloat16,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """A [M, K] B [N, K]^T of two 4-bit matrices -> bf16 or fp32 [M, N]; with
    swiglu, B holds the gate rows, then the up rows, and the result is
    silu(gate) * up [M, N / 2] (h3blk_gemm_fp4)."""
    (rows, K), (cols, Kb) = a.shape, b.shape
    if a.fmt != b.fmt or K != Kb or a.rotated != b.rotated or a.device != b.device:
        raise ValueError(f"operands do not match: {a} and {b}")
    if swiglu:
        cols //= 2
    out, ld = _output(out, rows, cols, dtype, a.device)
    if rows:
        _call(_gemm, out.get_device(), a.ref, b.ref, B.H3BLK_FP4_SWIGLU if swiglu else B.H3BLK_FP4_STORE, _OUT[dtype],
              out.data_ptr(), ld)
    return out


def sandwich_norm(x, y, tag, tidx, table, branch: int = 0, next_table=None, post_norm: bool = True, post_gain=None,
                  post_eps: float = 1e-5, norm_eps: float = 1e-5, branch_scale: float = 1.0, h: str | None = "bf16",
                  rotate: bool = False, x_out=None):
    """The norms after and before a block fused with its gate and residual:

      x_out = x + branch_scale * gate * (rmsnorm(y) * post_gain)    (y itself without post_norm)
      h     = rmsnorm(x_out) * (1 + scale) + shift

    branch 0 follows attention (gate1, then shift2 / scale2 of `table`); branch
    1 follows the feed-forward step (gate2, then shift1 / scale1 of
    `next_table`, the next layer's). h: "bf16", "mx" / "nv" (an Fp4Tensor, as
    quantize_fp4 of h's fp32 values; rotate as there) or None; without a next
    table there is no h after branch 1. x_out may be x. Returns (x_out, h).
    h3blk_sandwich_norm."""
    if x.dim() != 2 or table.dim() != 4:
        raise ValueError("expected x [rows, hidden] and table [n_tags, n_t, 6, hidden]")
    (n, c), (n_tags, n_t, _, _), dev = x.shape, table.shape, x.get_device()
    if x_out is None:
        x_out = torch.empty_like(x)
    norm_table = (next_table if branch else table) if h is not None else None
    rows, row, tab = (n, c), (n,), (n_tags, n_t, 6, c)
    _want("x", x, torch.bfloat16, rows, dev)
    _want("y", y, torch.bfloat16, rows, dev)
    _want("x_out", x_out, torch.bfloat16, rows, dev)
    _want("tag", tag, torch.int32, row, dev)
    _want("tidx", tidx, torch.int32, row, dev)
    _want("table", table, torch.float32, tab, dev)
    if norm_table is not None and norm_table is not table:
        _want("next_table", norm_table, torch.float32, tab, dev)
    if post_gain is not None:
        _want("post_gain", post_gain, torch.bfloat16, (c,), dev)
    if h is not None and h != "bf16" and h not in FORMATS:
        raise ValueError(f"h must be None, 'bf16', 'mx' or 'nv', got {h!r}")
    if rotate and h not in FORMATS:
        raise ValueError("rotate is for an h in 4 bits")
    out = fp4 = None
    if norm_table is not None:
        if h == "bf16":
            out = torch.empty_like(x)
        else:
            out = fp4 = Fp4Tensor(n, c, h, x.device)
            fp4.rotated = bool(rotate)
    if n:
        a = _pack_sandwich(n, c, n_tags, n_t, branch, post_norm, post_eps, norm_eps, branch_scale, x.data_ptr(),
                           y.data_ptr(), 0 if post_gain is None else post_gain.data_ptr(), tag.data_ptr(), tidx.data_ptr(),
                           table.data_ptr(), 0 if norm_table is None else norm_table.data_ptr(), x_out.data_ptr(),
                           0 if out is None or fp4 is not None else out.data_ptr(), 0 if fp4 is None else fp4.ref, rotate)
        _call(_sandwich, dev, a)
    return x_out, out


def _want(name, t, dtype, shape, dev):
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        raise ValueError(f"{name}: expected {dtype} {shape} contiguous on CUDA device {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
