"""The 4-bit operators, in their plain form and as the package's calls.

A 4-bit matrix ("microscaled floating point") holds k values a row in blocks
along k, each value an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) times
its block's scale:
  "mx": blocks of 32, scale 2^(floor(log2 amax) - 2), held as e8m0;
  "nv": blocks of 16, scale s g, s = e4m3(amax / (6 g)) and g the matrix's
        power of two, the least with amax_matrix <= 2688 g.
Codes are rounded to nearest, ties to even, and saturate at 6.

Storage: codes [rows, pitch] bytes, two codes a byte (the lower k in the low
four bits), pitch = 16 ceil(k / 32), the rest of a row zero; scales one byte a
block in atoms of 512 bytes, one for 128 rows x 4 blocks, atoms in row-major
order: the byte of row r, block b is (r % 32) 16 + (r % 128 // 32) 4 + b % 4 of
atom (r // 128, b // 4); those of no row or block are zero.

Operators: quantising one matrix or a list of them, along the rows, along the
columns (the stored matrix is then the transpose) or both, and back to
values; the product A B^T of two 4-bit matrices; the product of a few bf16
rows with a 4-bit matrix; a linear layer's forward and backward pass with all
three products in 4 bits.
"""

import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token's activations before a product
        {"name": "quantize one token", "op": "quantize", "fmt": "mx", "n": 1, "rows": 1, "cols": 2048, "along": "cols",
         "dtype": "bf16"},
        # a batch of activations, for the product and for the weight's gradient; a ragged token count
        {"name": "quantize activations", "op": "quantize", "fmt": "nv", "n": 1, "rows": 8191, "cols": 4096,
         "along": "both", "dtype": "bf16"},
        # an odd fp32 matrix, transposed only
        {"name": "quantize odd transposed", "op": "quantize", "fmt": "mx", "n": 1, "rows": 1409, "cols": 2047,
         "along": "rows", "dtype": "fp32"},
        # the experts' master weights after an optimizer step, for the forward and the backward products
        {"name": "quantize experts", "op": "quantize", "fmt": "nv", "n": 24, "rows": 2048, "cols": 1408,
         "along": "both", "dtype": "fp32"},
        # the tokens routed to one expert
        {"name": "product one expert", "op": "product", "fmt": "mx", "m": 77, "n": 1408, "k": 2048, "out": "bf16",
         "add": False},
        # a weight gradient added to a gradient buffer; no size a multiple of a tile
        {"name": "product odd added", "op": "product", "fmt": "nv", "m": 2047, "n": 1409, "k": 5000, "out": "fp32",
         "add": True},
        # the largest square product of the size sweep
        {"name": "product large", "op": "product", "fmt": "nv", "m": 8192, "n": 8192, "k": 8192, "out": "bf16",
         "add": False},
        # one token through an up projection
        {"name": "rows one token", "op": "rows", "fmt": "nv", "t": 1, "n": 8192, "k": 2048, "out": "bf16"},
        # a few tokens through an odd matrix
        {"name": "rows odd", "op": "rows", "fmt": "mx", "t": 5, "n": 2047, "k": 1409, "out": "fp32"},
        # a batch of single tokens through an LM head
        {"name": "rows head", "op": "rows", "fmt": "nv", "t": 16, "n": 65536, "k": 2048, "out": "bf16"},
        # a training step of one expert on its tokens
        {"name": "linear one expert", "op": "linear", "fmt": "mx", "t": 777, "k": 2048, "n": 1408},
        # a training step of an up projection
        {"name": "linear up", "op": "linear", "fmt": "nv", "t": 8192, "k": 2048, "n": 8192},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; one in two a multiple of 16 where there is room."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.5:
        v = v // 16 * 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "product", "rows", "linear"])
    fmt = rng.choice(["mx", "nv"])
    if op == "quantize":
        rows, cols = _size(rng, 1, 16384), _size(rng, 1, 8192)
        n = min(_size(rng, 1, 24), max(1, 24 * 2048 * 1408 // (rows * cols)))
        while n * rows * cols > 24 * 2048 * 1408:
            rows = rows // 2
        return {"op": op, "fmt": fmt, "n": n, "rows": rows, "cols": cols, "along": rng.choice(["cols", "rows", "both"]),
                "dtype": rng.choice(["bf16", "fp32"])}
    if op == "product":
        out = rng.choice(["bf16", "fp32"])
        return {"op": op, "fmt": fmt, "m": _size(rng, 1, 8192), "n": _size(rng, 16, 8192), "k": _size(rng, 32, 8192),
                "out": out, "add": out == "fp32" and rng.random() < 0.5}
    if op == "rows":
        n, k = _size(rng, 16, 65536), _size(rng, 32, 8192)
        while n * k > 65536 * 2048:
            n = n // 2
        return {"op": op, "fmt": fmt, "t": _size(rng, 1, 32), "n": n, "k": k, "out": rng.choice(["bf16", "fp32"])}
    t, k, n = _size(rng, 1, 8192), _size(rng, 32, 8192), _size(rng, 32, 8192)
    while t * k * n > 8192 * 2048 * 8192:
        t = t // 2
    return {"op": op, "fmt": fmt, "t": t, "k": k, "n": n}


# ------------------------------------------------------------------ the plain form


def _blocks(x, blk):
    """x [..., k] as [..., blocks, blk], filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % blk)).unflatten(-1, (-1, blk))


def _pow2(e, dtype=torch.float32):
    """2^e from its bits (normal numbers): pow and ldexp may be off in the last place."""
    if dtype == torch.float64:
        return (e.long() + 1023 << 52).view(dtype)
    return (e.int() + 127 << 23).view(dtype)


def _round_e4m3(d):
    ulp = _pow2((torch.frexp(d).exponent - 1).clamp(min=-6) - 3)
    return torch.round(d / ulp) * ulp


def _round_e2m1(v):
    a = v.abs()
    ulp = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / ulp) * ulp).clamp(max=6).copysign(v)


def _tensor_scale(x):
    """g of each matrix of x [..., rows, cols]: the least power of two with amax <= 2688 g = 1.3125 2^11 g."""
    f, e = torch.frexp(x.abs().amax(dim=(-2, -1)))
    return _pow2(e - 12 + (f > 0.65625).int())


def _quantized(x, fmt, g):
    """(e2m1 values [..., blocks, blk], block scales [..., blocks]) of x in blocks along its last dimension."""
    b = _blocks(x, BLOCK[fmt])
    amax = b.abs().amax(-1)
    if fmt == "mx":
        scale = torch.where(amax > 0, _pow2(torch.frexp(amax).exponent - 3), 1.0)
        return _round_e2m1(b / scale[..., None]), scale
    g = g[..., None, None]
    scale = _round_e4m3(amax / (6 * g)) * g
    v = _round_e2m1(b / torch.where(scale > 0, scale, 1.0)[..., None])
    return torch.where(scale[..., None] > 0, v, 0.0), scale


def _values(x, fmt, g):
    """x rounded to 4 bits in blocks along its last dimension, as the values they stand for."""
    v, scale = _quantized(x, fmt, g)
    return (v * scale[..., None]).flatten(-2)[..., : x.shape[-1]]


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _scale_places(rows, blocks, device):
    """The place of each block's scale, [rows, blocks]."""
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(blocks, device=device)[None, :]
    return (r // 128 * -(-blocks // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def _stored(x, fmt):
    """A 4-bit matrix of x [rows, k] as a program holds it: codes, scales, (g, amax)."""
    rows, k = x.shape
    g = _tensor_scale(x)
    v, scale = _quantized(x, fmt, g)
    blocks = scale.shape[1]
    grid = torch.tensor(E2M1[:8], device=x.device)
    code = torch.searchsorted(grid, v.abs().flatten(1).contiguous()).to(torch.uint8) + 8 * (v.flatten(1) < 0).to(torch.uint8)
    code = torch.nn.functional.pad(code, (0, -(-k // 32) * 32 - code.shape[1]))
    data = (code[:, 0::2] | code[:, 1::2] << 4).contiguous()
    if fmt == "mx":
        byte = (torch.frexp(scale).exponent - 1 + 127).to(torch.uint8)
    else:
        byte = (scale / g).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.zeros(-(-rows // 128) * -(-blocks // 4) * 512, dtype=torch.uint8, device=x.device)
    scales[_scale_places(rows, blocks, x.device)] = byte
    return data, scales, torch.stack([g, x.abs().amax()])


def _decoded(stored, rows, k, fmt, dtype=torch.float32):
    """The values of a stored 4-bit matrix."""
    data, scales, ts = stored
    blk = BLOCK[fmt]
    blocks = -(-k // blk)
    code = torch.stack([data & 15, data >> 4], -1).flatten(1)[:, :k]
    v = torch.tensor(E2M1, dtype=dtype, device=data.device)[code.int()]
    byte = scales[_scale_places(rows, blocks, data.device)]
    if fmt == "mx":
        scale = _pow2(byte.int() - 127, dtype)
    else:
        scale = byte.view(torch.float8_e4m3fn).to(dtype) * ts[0].to(dtype)
    return v * scale.repeat_interleave(blk, 1)[:, :k]


# ------------------------------------------------------------------ the cases


def _normal(shape, gen, std):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _activations(rows, k, gen):
    """Normalised activations: a few channels are far larger than the rest, and tokens differ in size."""
    x = _normal((rows, k), gen, 1.0)
    x *= torch.exp(_normal((k,), gen, 0.8)) * torch.exp(_normal((rows, 1), gen, 0.3))
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "quantize":
        shape = (c["n"], c["rows"], c["cols"])
        if c["dtype"] == "fp32":  # master weights; each matrix has a size of its own
            x = _normal(shape, gen, 0.02) * torch.exp(_normal((c["n"], 1, 1), gen, 0.5))
        else:
            x = torch.stack([_activations(c["rows"], c["cols"], gen) for _ in range(c["n"])])
        c["x"] = x.to(DTYPE[c["dtype"]])
    elif c["op"] == "product":
        c["a"] = _stored(_activations(c["m"], c["k"], gen), c["fmt"])
        c["b"] = _stored(_normal((c["n"], c["k"]), gen, 0.02), c["fmt"])
        if c["add"]:
            c["c"] = _normal((c["m"], c["n"]), gen, 0.5)
    elif c["op"] == "rows":
        c["x"] = _activations(c["t"], c["k"], gen).to(torch.bfloat16)
        c["w"] = _stored(_normal((c["n"], c["k"]), gen, 0.02), c["fmt"])
    else:
        c["x"] = _activations(c["t"], c["k"], gen).to(torch.bfloat16)
        c["w"] = _normal((c["k"], c["n"]), gen, 0.02)
        c["dy"] = _normal((c["t"], c["n"]), gen, 1e-3).to(torch.bfloat16)
    return c


def _run_own(c):
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4

    if c["op"] == "quantize":
        if c["n"] == 1:
            q = fp4.fp4_quantize(c["x"][0], fmt=c["fmt"], along=c["along"])
            return [[m.dequantize(torch.bfloat16)] for m in (q if c["along"] == "both" else [q])]
        if "plan" not in c:  # what a program keeps for a list of matrices: the plan, with the memory of their 4-bit forms
            c["plan"] = fp4.Fp4Plan(c["x"].unbind(0), fmt=c["fmt"], along=c["along"], values=torch.bfloat16)
        c["plan"].run()
        return c["plan"].dequantize()
    if c["op"] == "product":
        a = fp4.Fp4Matrix(c["m"], c["k"], c["fmt"], *c["a"])
        b = fp4.Fp4Matrix(c["n"], c["k"], c["fmt"], *c["b"])
        if c["add"]:
            out = c["c"].clone()
            return fp4.fp4_product(a, b, out=out, accumulate=True)
        return fp4.fp4_product(a, b, out_dtype=DTYPE[c["out"]])
    if c["op"] == "rows":
        w = fp4.Fp4Matrix(c["n"], c["k"], c["fmt"], *c["w"])
        return fp4.fp4_rows_product(c["x"], w, out_dtype=DTYPE[c["out"]])
    y, kept = fp4.fp4_linear(c["x"], c["w"], fmt=c["fmt"])
    dx, dw = fp4.fp4_linear_backward(kept, c["dy"])
    return y, dx, dw


def run(c):
    if own:
        return _run_own(c)
    fmt = c["fmt"]
    if c["op"] == "quantize":
        x = c["x"].float()
        g = _tensor_scale(x)
        out = []
        if c["along"] in ("cols", "both"):
            out.append(list(_values(x, fmt, g).to(torch.bfloat16)))
        if c["along"] in ("rows", "both"):
            out.append(list(_values(x.transpose(1, 2), fmt, g).to(torch.bfloat16)))
        return out
    if c["op"] == "product":
        out = _decoded(c["a"], c["m"], c["k"], fmt) @ _decoded(c["b"], c["n"], c["k"], fmt).T
        return (out + c["c"] if c["add"] else out).to(DTYPE[c["out"]])
    if c["op"] == "rows":
        return (c["x"].float() @ _decoded(c["w"], c["n"], c["k"], fmt).T).to(DTYPE[c["out"]])
    x, w, dy = c["x"].float(), c["w"], c["dy"].float()
    gx, gw, gy = _tensor_scale(x), _tensor_scale(w), _tensor_scale(dy)
    y = _values(x, fmt, gx) @ _values(w.T, fmt, gw).T
    dx = _values(dy, fmt, gy) @ _values(w, fmt, gw).T
    dw = _values(x.T, fmt, gx) @ _values(dy.T, fmt, gy).T
    return y.to(torch.bfloat16), dx.to(torch.bfloat16), dw


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_values(x, fmt):
    """x [rows, k], in 64 bits, to 4 bits along k by comparing with the midpoints between the values of e2m1."""
    rows, k = x.shape
    blk = BLOCK[fmt]
    out = torch.zeros(rows, -(-k // blk) * blk, dtype=torch.float64, device=x.device)
    out[:, :k] = x
    out = out.view(rows, -1, blk)
    amax = out.abs().max(dim=2, keepdim=True).values
    if fmt == "mx":
        step = (torch.where(amax > 0, amax, 4.0).contiguous().view(torch.int64) >> 52) - 2  # the exponent's bits
        step = (step << 52).view(torch.float64)
    else:
        g = 2.0 ** math.ceil(math.log2(float(amax.max()) / 2688))
        grid = torch.arange(0, 127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
        middle = (grid[1:] + grid[:-1]) / 2
        step = amax / (6 * g)
        at = torch.searchsorted(middle, step)
        tie = (at < 126) & (middle[at.clamp(max=125)] == step) & (at % 2 == 1)
        step = grid[at + tie.long()] * g
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    got = torch.zeros_like(out)
    for i in range(1, 8):  # a tie goes to the even code: up from an odd one, down from an even one
        border = (grid[i] + grid[i - 1]) / 2 * step
        reached = out.abs() >= border if i % 2 == 0 else out.abs() > border
        got = torch.where(reached & (step > 0), grid[i] * step, got)
    return (got * out.sign()).view(rows, -1)[:, :k]


def exact(case, seed):
    c = prepare(case, seed)
    fmt = c["fmt"]
    if c["op"] == "quantize":
        out = []
        if c["along"] in ("cols", "both"):
            out.append([_exact_values(x.double(), fmt) for x in c["x"]])
        if c["along"] in ("rows", "both"):
            out.append([_exact_values(x.double().T, fmt) for x in c["x"]])
        return out
    if c["op"] == "product":
        out = torch.einsum("mk,nk->mn", _decoded(c["a"], c["m"], c["k"], fmt, torch.float64),
                           _decoded(c["b"], c["n"], c["k"], fmt, torch.float64))
        return out + c["c"].double() if c["add"] else out
    if c["op"] == "rows":
        return torch.einsum("tk,nk->tn", c["x"].double(), _decoded(c["w"], c["n"], c["k"], fmt, torch.float64))
    x, w, dy = c["x"].double(), c["w"].double(), c["dy"].double()
    y = torch.einsum("tk,nk->tn", _exact_values(x, fmt), _exact_values(w.T, fmt))
    dx = torch.einsum("tn,kn->tk", _exact_values(dy, fmt), _exact_values(w, fmt))
    dw = torch.einsum("kt,nt->kn", _exact_values(x.T, fmt), _exact_values(dy.T, fmt))
    return y, dx, dw


def _held(rows, k, fmt):
    """Bytes of a 4-bit matrix: half a byte a value and a byte a block."""
    return rows * (k / 2 + -(-k // BLOCK[fmt]))


def work(case):
    c, fmt = case, case["fmt"]
    if c["op"] == "quantize":
        n, r, k = c["n"], c["rows"], c["cols"]
        ways = [(r, k)] * (c["along"] != "rows") + [(k, r)] * (c["along"] != "cols")
        size = n * r * k * (2 if c["dtype"] == "bf16" else 4)
        # the source once; each 4-bit matrix written, read again and its values written in bf16
        return {"bytes": size + sum(n * (2 * _held(*w, fmt) + 2 * r * k) for w in ways), "flops": 0}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        out = m * n * (2 if c["out"] == "bf16" else 12 if c["add"] else 4)  # added: read, copied and added to
        return {"bytes": _held(m, k, fmt) + _held(n, k, fmt) + out, "flops": 2 * m * n * k}
    if c["op"] == "rows":
        t, n, k = c["t"], c["n"], c["k"]
        return {"bytes": _held(n, k, fmt) + 2 * t * k + t * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * t * n * k}
    t, k, n = c["t"], c["k"], c["n"]
    held = sum(_held(*s, fmt) for s in ((t, k), (k, t), (k, n), (n, k), (t, n), (n, t)))
    # the sources once, the six 4-bit matrices written and read, y and dx in bf16, dw in fp32
    return {"bytes": 2 * t * k + 4 * k * n + 2 * t * n + 2 * held + 2 * t * n + 2 * t * k + 4 * k * n, "flops": 6 * t * k * n}
