"""Cases of the microscaled 4-bit linear path and of the sandwich norm that feeds it.

Four operators: quantisation of bf16 rows to 4-bit floats with block scales, its inverse, the product of two
such operands (plain and SwiGLU), and the norms after and before a block fused with its gate and residual.
`run` computes a case in elementary torch operations where `own` is false, and by the package's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
RSQRT128 = 1.0 / math.sqrt(128.0)


def _lib():
    import joint_video_audio_b200 as j
    return j


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the tiny block's rows: a call of a few microseconds, latency counts
        {"name": "round_nv_tiny", "op": "round", "fmt": "nv", "rows": 320, "k": 256, "pad": 0, "rotate": False},
        # attention output of an odd number of packed rows, read out of a wider buffer
        {"name": "round_nv_attn_out", "op": "round", "fmt": "nv", "rows": 8191, "k": 7168, "pad": 64, "rotate": False},
        # the SwiGLU output of the 32k-row sequence
        {"name": "round_mx_ffn_32k", "op": "round", "fmt": "mx", "rows": 32768, "k": 14336, "pad": 0, "rotate": False},
        # one row through the attention's output projection: the weight is all there is to read
        {"name": "linear_nv_1row", "op": "linear", "fmt": "nv", "m": 1, "n": 5376, "k": 7168, "out": "bf16", "rotate": False},
        # the text refiner's QKV projection, rotated as the int8 path is
        {"name": "linear_mx_text", "op": "linear", "fmt": "mx", "m": 512, "n": 21504, "k": 5376, "out": "bf16", "rotate": True},
        # the video head: few output columns, fp32 out, an odd number of rows
        {"name": "linear_mx_head", "op": "linear", "fmt": "mx", "m": 31247, "n": 96, "k": 5376, "out": "fp32", "rotate": False},
        # FFN down of the 32k-row sequence: the largest product with its quantisation
        {"name": "linear_nv_down_32k", "op": "linear", "fmt": "nv", "m": 32768, "n": 5376, "k": 14336, "out": "bf16", "rotate": True},
        # FFN up with SwiGLU of 8192 rows, operands already in 4 bits
        {"name": "product_nv_swiglu_8k", "op": "product", "fmt": "nv", "m": 8192, "n": 28672, "k": 5376, "out": "bf16", "swiglu": True},
        # the same product of the audio rows, in the other format, plain
        {"name": "product_mx_audio", "op": "product", "fmt": "mx", "m": 1008, "n": 28672, "k": 5376, "out": "bf16", "swiglu": False},
        # the tiny block with its 32 padding rows
        {"name": "sandwich_tiny", "op": "sandwich", "rows": 320, "c": 256, "branch": 0, "post": True, "padding": 32, "mixed": True},
        # after the FFN of the 32k-row sequence, modulated by the next layer's table
        {"name": "sandwich_32k", "op": "sandwich", "rows": 32768, "c": 5376, "branch": 1, "post": True, "padding": 168, "mixed": False},
        # after attention, straight into the FFN's SwiGLU product: h leaves the norm in 4 bits
        {"name": "chain_nv_ffn_up", "op": "chain", "fmt": "nv", "rows": 4001, "c": 5376, "f": 14336, "padding": 33, "mixed": True, "rotate": True},
    ]


def _log(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["round", "round", "linear", "product", "sandwich", "sandwich", "chain"])
    fmt = rng.choice(["mx", "nv"])
    if op == "round":
        return {"op": op, "fmt": fmt, "rows": _log(rng, 1, 32768, 1), "k": _log(rng, 32, 14336, 32), "pad": 8 * rng.randrange(0, 9),
                "rotate": False}
    if op == "sandwich":
        rows = _log(rng, 1, 32768, 1)
        return {"op": op, "rows": rows, "c": _log(rng, 128, 5376, 128), "branch": rng.randrange(2), "post": rng.random() < 0.7,
                "padding": rng.randrange(0, rows // 8 + 1), "mixed": rng.random() < 0.5}
    if op == "chain":
        rows = _log(rng, 1, 4096, 1)
        return {"op": op, "fmt": fmt, "rows": rows, "c": _log(rng, 128, 5376, 128), "f": _log(rng, 128, 14336, 128),
                "padding": rng.randrange(0, rows // 8 + 1), "mixed": rng.random() < 0.5, "rotate": rng.random() < 0.5}
    m, rotate = _log(rng, 1, 8192, 1), rng.random() < 0.4
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "linear":
        return {"op": op, "fmt": fmt, "m": m, "n": _log(rng, 8, 28672, 8), "k": _log(rng, 128, 14336, 128 if rotate else 32), "out": out,
                "rotate": rotate}
    swiglu = rng.random() < 0.5
    return {"op": op, "fmt": fmt, "m": m, "n": _log(rng, 256, 28672, 256) if swiglu else _log(rng, 8, 28672, 8),
            "k": _log(rng, 32, 14336, 32), "out": out, "swiglu": swiglu}


# ------------------------------------------------------------------ inputs

def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rows(g, n, k):
    """Activations as bf16: unit normal with a spread of row sizes and some channels ten times as large, one zero row."""
    x = _rand(g, n, k)
    x *= torch.exp(0.5 * _rand(g, n, 1))
    x[:, torch.randint(0, k, (max(1, k // 128),), generator=g, device=DEV)] *= 10.0
    if n > 4:
        x[n // 2] = 0.0
    return x.to(torch.bfloat16)


def _weight(g, n, k):
    return (_rand(g, n, k) / math.sqrt(k)).to(torch.bfloat16)


def _modulated(g, c, padding):
    """Packed rows' residual stream, the block's output, tags (tag -1: padding), timestep indices and a table.
    The sequence is packed as the model packs it: text, then audio, then video rows, padding last; "mixed" draws
    each row's timestep index by itself, as two-time conditioning does."""
    n, ch = c["rows"], c["c"]
    tag = torch.full((n,), 3, device=DEV, dtype=torch.int32)
    tag[:n // 10] = 2
    tag[:n // 16] = 0
    tidx = (tag == 2).to(torch.int32)
    if c["mixed"]:
        tidx = torch.randint(0, 2, (n,), generator=g, device=DEV, dtype=torch.int32)
    if padding:
        tag[n - padding:] = -1
    return {"x": (1.5 * _rand(g, n, ch)).to(torch.bfloat16), "y": _rows(g, n, ch), "tag": tag, "tidx": tidx,
            "table": 0.3 * _rand(g, 4, 2, 6, ch), "next": 0.3 * _rand(g, 4, 2, 6, ch),
            "gain": (1 + 0.1 * _rand(g, ch)).to(torch.bfloat16), "alpha": 0.7}


def _inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 11)
    op = c["op"]
    if op == "round":
        return {"x": _rows(g, c["rows"], c["k"] + c["pad"])[:, :c["k"]]}
    if op in ("linear", "product"):
        return {"x": _rows(g, c["m"], c["k"]), "w": _weight(g, c["n"], c["k"])}
    d = _modulated(g, c, c["padding"])
    if op == "chain":
        d["w"] = _weight(g, 2 * c["f"], c["c"])
    return d


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    # weights, and the product's operands, are quantised once, as a program that loads them does
    for k in ("w", "x") if case["op"] == "product" else ("w",):
        if k in s:
            fmt, rotate = case["fmt"], case.get("rotate", False)
            s[k] = _lib().quantize_fp4(s[k], fmt, rotate=rotate) if own else _values(s[k].float(), fmt, rotate)
    return s


# ------------------------------------------------------------------ plain forms

def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device=DEV)
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _e2m1(a):
    """Magnitudes (>= 0) to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code."""
    return 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5).float() + (a >= 3.5) + 2.0 * (a > 5.0)


def _values(x, fmt, rotate):
    """fp32 [rows, K] -> the values its 4-bit form stands for, fp32."""
    n, k = x.shape
    if rotate:
        x = (x.view(n, k // 128, 128) @ _hadamard(x.dtype)).view(n, k)
    if fmt == "mx":
        b = x.view(n, k // 32, 32)
        amax = b.abs().amax(-1, keepdim=True)
        m, e = torch.frexp(amax)
        e = (e - torch.where(m <= 0.875, 3, 2)).clamp(-126, 127)
        scale = torch.ldexp(torch.ones_like(amax), e)
        row = torch.ones_like(amax[:, :1])
    else:
        b = x.view(n, k // 16, 16)
        top = b.abs().amax((1, 2), keepdim=True)
        m, e = torch.frexp(top)
        e = (e - torch.where(m <= 0.65625, 12, 11)).clamp(-126, 127)
        row = torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, 0))
        b = b / row
        scale = (b.abs().amax(-1, keepdim=True) / 6.0).to(torch.float8_e4m3fn).float()
    q = torch.where(scale > 0, b / scale, 0.0)
    v = torch.copysign(_e2m1(q.abs()), q) * scale * row
    return v.view(n, k) * (RSQRT128 if rotate else 1.0)


def _norm(v, eps):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)


def _modulation(table, tag, tidx, i):
    m = table[tag.clamp(min=0).long(), tidx.long(), i]
    return torch.where(tag[:, None] >= 0, m, 0.0)


def _sandwich(s, branch, post):
    """(x1, h) in the precision of s's floating tensors; `post` says whether the block's output is normed."""
    p = _norm(s["y"], EPS) * s["gain"] if post else s["y"]
    x1 = s["x"] + s["alpha"] * _modulation(s["table"], s["tag"], s["tidx"], 5 if branch else 2) * p
    t, i = (s["next"], 0) if branch else (s["table"], 3)
    h = _norm(x1, EPS) * (1 + _modulation(t, s["tag"], s["tidx"], i + 1)) + _modulation(t, s["tag"], s["tidx"], i)
    return x1, h


def _out(c):
    return torch.float32 if c.get("out") == "fp32" else torch.bfloat16


def _product(a, b, swiglu):
    y = a @ b.T
    if swiglu:
        g, u = y.chunk(2, 1)
        y = g / (1 + torch.exp(-g)) * u
    return y


def _plain(s):
    c = s["case"]
    if c["op"] == "round":
        return _values(s["x"].float().contiguous(), c["fmt"], c["rotate"]).to(torch.bfloat16)
    if c["op"] == "linear":
        return _product(_values(s["x"].float(), c["fmt"], c["rotate"]), s["w"], False).to(_out(c))
    if c["op"] == "product":
        return _product(s["x"], s["w"], c["swiglu"]).to(_out(c))
    f = {k: v.float() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items() if k != "w"}
    if c["op"] == "sandwich":
        x1, h = _sandwich(f, c["branch"], c["post"])
        return {"x": x1.to(torch.bfloat16), "h": h.to(torch.bfloat16)}
    x1, h = _sandwich(f, 0, True)
    return {"x": x1.to(torch.bfloat16), "y": _product(_values(h, c["fmt"], c["rotate"]), s["w"], True).to(torch.bfloat16)}


# ------------------------------------------------------------------ one pass

def _own(s):
    j, c = _lib(), s["case"]
    if c["op"] == "round":
        return j.dequantize_fp4(j.quantize_fp4(s["x"], c["fmt"], rotate=c["rotate"]))
    if c["op"] == "linear":
        return j.gemm_fp4(j.quantize_fp4(s["x"], c["fmt"], rotate=c["rotate"]), s["w"], dtype=_out(c))
    if c["op"] == "product":
        return j.gemm_fp4(s["x"], s["w"], swiglu=c["swiglu"], dtype=_out(c))
    args = (s["x"], s["y"], s["tag"], s["tidx"], s["table"])
    if c["op"] == "sandwich":
        x1, h = j.sandwich_norm(*args, branch=c["branch"], next_table=s["next"], post_norm=c["post"],
                                post_gain=s["gain"] if c["post"] else None, post_eps=EPS, norm_eps=EPS, branch_scale=s["alpha"])
        return {"x": x1, "h": h}
    x1, h = j.sandwich_norm(*args, branch=0, post_gain=s["gain"], post_eps=EPS, norm_eps=EPS, branch_scale=s["alpha"],
                            h=c["fmt"], rotate=c["rotate"])
    return {"x": x1, "y": j.gemm_fp4(h, s["w"], swiglu=True)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def _bytes4(fmt, n, k):
    return n * k // 2 + n * k // (32 if fmt == "mx" else 16)


def work(case):
    c = case
    if c["op"] == "round":  # bf16 in, bf16 values out
        return {"bytes": 4 * c["rows"] * c["k"], "flops": 2 * c["rows"] * c["k"]}
    if c["op"] == "sandwich":
        return {"bytes": 8 * c["rows"] * c["c"], "flops": 12 * c["rows"] * c["c"]}
    if c["op"] == "chain":
        n, ch, f = c["rows"], c["c"], c["f"]
        return {"bytes": 6 * n * ch + _bytes4(c["fmt"], 2 * f, ch) + 2 * n * f, "flops": 4 * n * ch * f}
    m, n, k = c["m"], c["n"], c["k"]
    a = 2 * m * k if c["op"] == "linear" else _bytes4(c["fmt"], m, k)
    y = m * n * (4 if c["out"] == "fp32" else 2) // (2 if c.get("swiglu") else 1)
    return {"bytes": a + _bytes4(c["fmt"], n, k) + y, "flops": 2 * m * n * k}


# ------------------------------------------------------------------ in 64 bits

def _exact_values(x, fmt, rotate):
    """The definition, in 64 bits: nearest entry of the value table by searching its midpoints, scales by division."""
    n, k = x.shape
    if rotate:
        t = x.view(n, k // 128, 128)
        step = 1
        while step < 128:  # Walsh-Hadamard butterflies
            t = t.view(n, -1, 2, step)
            t = torch.stack([t[:, :, 0] + t[:, :, 1], t[:, :, 0] - t[:, :, 1]], 2)
            step *= 2
        x = t.reshape(n, k)
    size = 32 if fmt == "mx" else 16
    b = x.reshape(n, k // size, size)
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        scale = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / 7.0)).clamp(min=-126)), 1.0)
        scale = torch.where(amax <= 3.5 * scale, scale / 2, torch.where(amax > 7.0 * scale, scale * 2, scale))
    else:
        top = amax.amax(1, keepdim=True)
        e = torch.where(top > 0, torch.ceil(torch.log2(top / 2688.0)).clamp(min=-126), 0.0)
        row = torch.exp2(e)
        row = torch.where((top > 0) & (top <= 1344.0 * row), row / 2, torch.where(top > 2688.0 * row, row * 2, row))
        s = amax / row / 6.0
        ulp = torch.exp2(torch.floor(torch.log2(s.clamp(min=2.0 ** -6))) - 3)
        scale = torch.round(s / ulp) * ulp * row
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    mid = (table[1:] + table[:-1]) / 2
    q = torch.where(scale > 0, b.abs() / scale, 0.0)
    lo = torch.bucketize(q, mid)                    # ties go down ...
    hi = torch.bucketize(q, mid, right=True)        # ... or up: the even of the two
    code = torch.where(lo % 2 == 0, lo, hi)
    v = torch.sign(b) * table[code] * scale
    return v.reshape(n, k) / (math.sqrt(128.0) if rotate else 1.0)


def _exact_norm(v):
    return v / torch.sqrt(torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / v.shape[-1] + EPS)


def exact(case, seed):
    c = case
    d = _inputs(c, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in d.items()}
    if c["op"] == "round":
        return _exact_values(wide["x"].contiguous(), c["fmt"], c["rotate"])
    rot = c.get("rotate", False)
    if c["op"] in ("linear", "product"):
        x, w = _exact_values(wide["x"], c["fmt"], rot), _exact_values(wide["w"], c["fmt"], rot)
        y = torch.einsum("mk,nk->mn", x, w)
        if c.get("swiglu"):
            f = c["n"] // 2
            y = y[:, :f] * torch.sigmoid(y[:, :f]) * y[:, f:]
        return y
    valid = (wide["tag"] >= 0).double()[:, None]
    key = (wide["tag"].long() * 2 + wide["tidx"].long()).clamp(min=0)
    vec = lambda t, i: t.reshape(8, 6, -1)[:, i][key] * valid  # noqa: E731
    branch = c.get("branch", 0)
    p = _exact_norm(wide["y"]) * wide["gain"] if c.get("post", True) else wide["y"]
    x1 = wide["x"] + 0.7 * vec(wide["table"], (2, 5)[branch]) * p
    t = wide["next"] if branch else wide["table"]
    h = _exact_norm(x1) * (1.0 + vec(t, (4, 1)[branch])) + vec(t, (3, 0)[branch])
    if c["op"] == "sandwich":
        return {"x": x1, "h": h}
    w = _exact_values(wide["w"], c["fmt"], rot)
    y = torch.einsum("mk,nk->mn", _exact_values(h, c["fmt"], rot), w)
    g, u = y[:, :c["f"]], y[:, c["f"]:]
    return {"x": x1, "y": g * torch.sigmoid(g) * u}
