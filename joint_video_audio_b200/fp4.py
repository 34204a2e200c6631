"""The 4-bit linear path and the sandwich norm for torch tensors (no arithmetic
here): include/h3blk.h states the formats and the formulas, csrc/fp4_torch.cpp
checks the tensors and makes the calls.

Tensors are contiguous; quantize_fp4's x and a given `out` may have a row stride that
is a multiple of 8. Outputs come from the caching
allocator without torch's dispatcher: dispatch modes do not see them, deterministic
mode does not fill them, and they carry no gradient. A kernel that gives up a wait
is reported by check_fp4 alone."""
from __future__ import annotations

from functools import lru_cache

import torch

from . import _binding as B


class _Host:
    """The calls of csrc/fp4_torch.cpp. Its module is tied to one Python and one
    torch, so that it is imported with the first 4-bit call: the rest of the package
    does without."""

    def __getattr__(self, name):
        if name.startswith("_"):
            raise AttributeError(name)
        try:
            from . import _fp4_torch as m
        except ImportError as e:
            raise ImportError("the 4-bit calls need joint_video_audio_b200/_fp4_torch, built for this Python and torch "
                              f"(python joint_video_audio_b200/build.py): {e}") from e
        m.set_error(B.H3BlkError)
        self.__dict__.update({k: f for k, f in vars(m).items() if not k.startswith("_")})
        return self.__dict__[name]


_host = _Host()
FORMATS = {"mx": B.H3BLK_FP4_MX, "nv": B.H3BLK_FP4_NV}
_IS_F32 = {torch.bfloat16: False, torch.float32: True}


def _code(fmt) -> int:
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}, got {fmt!r}")
    return FORMATS[fmt]


def _f32(dtype) -> bool:
    if dtype not in _IS_F32:
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    return _IS_F32[dtype]


@lru_cache(maxsize=1024)
def _layout(rows: int, K: int, fmt: str):
    """(byte lengths, offsets, total) of a matrix's three parts in its buffer."""
    return _host.layout(_code(fmt), rows, K)


class Fp4Tensor:
    """A [rows, K] matrix in microscaled 4-bit floats on the GPU (h3blk_fp4).

    codes      uint8 [rows, K / 2], two e2m1 codes a byte
    scales     uint8 [..., 512] atoms of 128 rows x 4 block scales
    row_scale  fp32 [rows]
    rotated    whether the values went through the Hadamard rotation
    """

    __slots__ = ("fmt", "shape", "rotated", "buffer")

    def __init__(self, rows: int, K: int, fmt: str = "nv", device="cuda"):
        total = _layout(rows, K, fmt)[2]
        self.fmt, self.shape, self.rotated = fmt, (rows, K), False
        self.buffer = torch.empty(total, dtype=torch.uint8, device=device)

    def _part(self, i):
        lens, at, _ = _layout(*self.shape, self.fmt)
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


def _matrix(fmt, shape, rotated, buffer) -> Fp4Tensor:
    q = Fp4Tensor.__new__(Fp4Tensor)
    q.fmt, q.shape, q.rotated, q.buffer = fmt, shape, rotated, buffer
    return q


def quantize_fp4(x: torch.Tensor, fmt: str = "nv", rotate: bool = False, out: Fp4Tensor | None = None) -> Fp4Tensor:
    """bf16 [rows, K] (rows may be strided) -> microscaled 4-bit floats.

    fmt "mx": blocks of 32 with power-of-two scales; "nv": blocks of 16 with
    e4m3 scales and a power-of-two scale per row. rotate: the block-128 Hadamard
    transform of the W8A8 path first (a product takes two rotated operands or
    two that are not). h3blk_quantize_fp4."""
    if out is None:
        shape, buffer = _host.quantize(x, _code(fmt), rotate, None)
        return _matrix(fmt, shape, bool(rotate), buffer)
    if out.fmt != fmt or out.shape != tuple(x.shape):
        raise ValueError(f"out: expected {fmt} {tuple(x.shape)} on {x.device}, got {out}")
    _host.quantize(x, _code(fmt), rotate, out.buffer)
    out.rotated = bool(rotate)
    return out


def dequantize_fp4(q: Fp4Tensor, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values `q` stands for, bf16 or fp32 [rows, K] (h3blk_dequantize_fp4)."""
    rows, K = q.shape
    return _host.dequantize(q.buffer, _code(q.fmt), rows, K, _f32(dtype), out)


def gemm_fp4(a: Fp4Tensor, b: Fp4Tensor, swiglu: bool = False, dtype=torch.bfloat16,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """A [M, K] B [N, K]^T of two 4-bit matrices -> bf16 or fp32 [M, N]; with
    swiglu, B holds the gate rows, then the up rows, and the result is
    silu(gate) * up [M, N / 2] (h3blk_gemm_fp4)."""
    (rows, K), (cols, Kb) = a.shape, b.shape
    if a.fmt != b.fmt or K != Kb or a.rotated != b.rotated:
        raise ValueError(f"operands do not match: {a} and {b}")
    return _host.gemm(a.buffer, rows, b.buffer, cols, _code(a.fmt), K, swiglu, _f32(dtype), out)


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
    With more than 2048 channels a rotated h takes longer than a "bf16" one with
    quantize_fp4 behind it (which rounds it to bf16 in between), an "nv" one about
    as long.
    h3blk_sandwich_norm."""
    if rotate and h not in FORMATS:
        raise ValueError("rotate is for an h in 4 bits")
    if h is not None and h != "bf16" and h not in FORMATS:
        raise ValueError(f"h must be None, 'bf16', 'mx' or 'nv', got {h!r}")
    norm_table = None if h is None else next_table if branch else table
    x_out, out = _host.sandwich(x, y, tag, tidx, table, branch, norm_table, post_norm, post_gain, post_eps, norm_eps,
                                branch_scale, -2 if h is None else FORMATS.get(h, -1), rotate, x_out)
    if out is not None and h != "bf16":
        out = _matrix(h, tuple(x.shape), bool(rotate), out)
    return x_out, out


def check_fp4(device=None) -> int:
    """Device status of the 4-bit calls and the sandwich norm on `device` (the
    current one) since the last check, behind a synchronisation with its current
    stream: H3BLK_OK, or H3BLK_ERR_TIMEOUT if a kernel gave up a wait and left its
    output incomplete. h3blk_fp4_check."""
    with torch.cuda.device(device):
        return B.h3blk_fp4_check(torch.cuda.current_stream().cuda_stream)
