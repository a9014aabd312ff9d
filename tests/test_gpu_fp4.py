"""The 4-bit operators on the GPU against the fp64 oracle: quantisation bit
for bit with its storage, the products within bounds derived from their
arithmetic, the linear layer's step, streams, captured calls, and a run of
all of them with the optimizer step."""

import numpy as np
import pytest
import torch

import oracle.fp4_oracle as o

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
# one rounding of the output: half a step of its type
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def fp4():
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4 as m
    return m


def values(shape, seed, dtype="fp32", spread=1.0):
    """Normal values whose rows and columns differ in size, rounded to dtype (fp64 array and CUDA tensor)."""
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape) * np.exp(spread * r.standard_normal((shape[0], 1)))
    x = x * np.exp(spread * r.standard_normal((1, shape[1])))
    t = torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dtype])
    return t.double().cpu().numpy(), t


def guarded(fp4, rows, k, fmt):
    """An Fp4Matrix over storage filled with 0xAA, with guard bytes around each part."""
    m = fp4.Fp4Matrix.empty(rows, k, fmt)
    bufs = [torch.full((t.numel() + 512,), 0xAA, dtype=torch.uint8, device="cuda") for t in (m.data, m.scales)]
    ts = torch.full((4,), -7.0, device="cuda")
    g = fp4.Fp4Matrix(rows, k, fmt, *[b[256:b.numel() - 256] for b in bufs], ts[1:3])
    g.guards = bufs, ts
    return g


def check_stored(m, q, amax_known=True):
    data, scales = q.stored()
    assert np.array_equal(m.data.cpu().numpy().reshape(data.shape), data)
    assert np.array_equal(m.scales.cpu().numpy(), scales)
    if m.fmt == "nv":
        assert m.tensor_scale.cpu().tolist() == [q.g, q.amax]
    if hasattr(m, "guards"):
        for b in m.guards[0]:
            assert (b[:256] == 0xAA).all() and (b[-256:] == 0xAA).all()
        assert m.guards[1][0] == -7.0 and m.guards[1][3] == -7.0


SHAPES = [(1, 1), (1, 2048), (2048, 1), (3, 17), (31, 33), (64, 48), (128, 128), (129, 257), (200, 31), (255, 130),
          (300, 520), (1, 16), (7, 4000), (8, 2048), (8, 2049), (16385, 1)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_is_bitwise_the_oracle(fp4, shape, dtype, fmt):
    """Codes, scales, padding and tensor scale, in both directions and each alone; nothing else is written."""
    x64, x = values(shape, hash(shape) % 1000, dtype)
    for along in ("cols", "rows", "both"):
        outs = [guarded(fp4, *s, fmt) for s in ([shape] * (along != "rows") + [shape[::-1]] * (along != "cols"))]
        fp4.fp4_quantize(x, fmt=fmt, along=along, out=tuple(outs) if along == "both" else outs[0])
        want = [o.quantize(x64, fmt)] * (along != "rows") + [o.quantize(x64.T, fmt)] * (along != "cols")
        for m, q in zip(outs, want):
            check_stored(m, q)
            for dt in DT.values():
                v = m.dequantize(dt)
                assert torch.equal(v.double(), torch.from_numpy(q.values()).cuda())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_ties_borders_and_extremes(fp4, dtype, fmt):
    """Values on and next to every border: midpoints of the codes under every
    significand of a scale, amax at the borders of the scales, signed zeros,
    the smallest and largest magnitudes."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    blk = o.BLOCK[fmt]
    rows = []
    for sig in range(8, 16):  # amax / 6 with every 4-bit significand, and codes at the midpoints
        unit = sig / 8.0
        row = np.zeros(blk)
        row[0] = 6 * unit
        row[1:8] = [m * unit for m in mids]
        row[8:15] = [-np.nextafter(np.float32(m * unit), np.float32(0)) for m in mids]
        rows.append(row)
        rows.append(np.roll(row, 3) * 2.0 ** -5)
    for s in (o.E4M3[1:] + o.E4M3[:-1])[::3] / 2:  # a block maximum half way between two scales
        row = np.zeros(blk)
        row[blk - 1] = 6 * s
        row[0] = -3 * s
        rows.append(row)
        rows.append(row * (1 + 2.0 ** -7))
    ext = np.zeros(blk)
    ext[:6] = [0.0, -0.0, 1e-38, -1e-40, 2.0 ** -126, 2.0 ** -149]
    rows.append(ext)
    x = np.stack(rows)
    x[0, 0] = 2688.0  # g = 1 for the whole matrix
    big = np.zeros((2, blk))
    big[0, 0], big[1, 1] = 2.0 ** 126, -(2.0 ** 125)
    tiny = np.stack([ext, ext * 2, -ext])
    for m in (x, x * 2.0 ** -60, big, tiny, np.zeros((3, blk + 1))):
        t = torch.from_numpy(m.astype(np.float32)).cuda().to(DT[dtype])
        m64 = t.double().cpu().numpy()
        c, r = fp4.fp4_quantize(t, fmt=fmt, along="both")
        for got, want in ((c, o.quantize(m64, fmt)), (r, o.quantize(m64.T, fmt))):
            check_stored(got, want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_non_finite(fp4, dtype, fmt):
    """A NaN or an infinity makes its block NaN, in both directions, and changes no other."""
    x64, x = values((150, 200), 5, dtype)
    for i, j, v in ((0, 0, np.nan), (37, 99, np.inf), (149, 199, -np.inf), (64, 64, -np.nan)):
        x[i, j] = v
        x64[i, j] = v
    c, r = fp4.fp4_quantize(x, fmt=fmt, along="both")
    for m, q in ((c, o.quantize(x64, fmt)), (r, o.quantize(x64.T, fmt))):
        want = torch.from_numpy(q.values()).cuda()
        got = m.dequantize(torch.float32).double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
        assert torch.equal(m.scales, torch.from_numpy(q.stored()[1]).cuda())
    x[:] = float("nan")
    assert torch.isnan(fp4.fp4_quantize(x, fmt=fmt).dequantize()).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("off,ld", [(0, 320), (1, 320), (3, 317), (8, 321)])
def test_quantize_and_dequantize_strided(fp4, off, ld, dtype, fmt):
    """Sources and destinations inside larger rows, aligned and not; the rest of the destination stays."""
    _, big = values((140, ld), 6, dtype)
    x = big[:, off:off + 300]
    m = fp4.fp4_quantize(x, fmt=fmt)
    q = o.quantize(x.double().cpu().numpy(), fmt)
    check_stored(m, q)
    dst = torch.full((140, ld), 99.0, dtype=DT[dtype], device="cuda")
    m.dequantize(out=dst[:, off:off + 300])
    assert torch.equal(dst[:, off:off + 300].double(), torch.from_numpy(q.values()).cuda())
    assert (dst[:, :off] == 99).all() and (dst[:, off + 300:] == 99).all()


def test_every_code_and_scale_byte_decodes(fp4):
    """All 16 codes under all 256 scale bytes, both formats; what passes
    fp32's range (from 2 times 2^127 on) reads as infinity."""
    for fmt in ("mx", "nv"):
        blk = o.BLOCK[fmt]
        k = 256 * blk
        codes = np.tile(np.arange(blk) % 16, (1, 256))
        byte = np.arange(256)[None, :]
        q = o.Fp4(codes, byte, 0.5 if fmt == "nv" else 1.0, 0.0, fmt, k)
        data, scales = q.stored()
        m = fp4.Fp4Matrix(1, k, fmt, torch.from_numpy(data).cuda(), torch.from_numpy(scales).cuda(),
                          torch.tensor([0.5, 0.0], device="cuda"))
        with np.errstate(over="ignore"):
            want = q.values().astype(np.float32).astype(np.float64)
        got = m.dequantize(torch.float32).double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        assert np.array_equal(got[fine], want[fine])


def quantized(fp4, shape, seed, fmt, spread=0.7):
    x64, x = values(shape, seed, "fp32", spread)
    return fp4.fp4_quantize(x, fmt=fmt), o.quantize(x64, fmt).values()


def check_product(got, a, b, dtype, add=None):
    """|got - A B^T| within: the fp32 sums (at most one rounding, to within a
    step, of each partial sum of 16 products, every partial sum at most the
    sum of magnitudes S), the scaling, the added term and the output's
    rounding."""
    want = a @ b.T
    s = np.abs(a) @ np.abs(b).T
    n = -(-a.shape[1] // 16) + 2
    tol = n * 2.0 ** -23 * s
    if add is not None:
        want = want + add
        tol = tol + 2.0 ** -24 * (np.abs(want) + tol)
    tol = tol + HALF[dtype] * (np.abs(want) + tol) + 1e-38
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float(np.max(err / tol))


PRODUCTS = [(1, 1, 1), (1, 16, 32), (5, 130, 64), (128, 128, 256), (129, 127, 257), (77, 1408, 2048), (300, 200, 31),
            (256, 256, 512), (255, 513, 1000), (1, 2048, 1408), (2048, 1, 100)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("shape", PRODUCTS)
def test_product_matches_the_oracle(fp4, shape, fmt):
    m, n, k = shape
    a, a64 = quantized(fp4, (m, k), 11, fmt)
    b, b64 = quantized(fp4, (n, k), 12, fmt)
    for dt in DT.values():
        check_product(fp4.fp4_product(a, b, out_dtype=dt), a64, b64, dt)
    c64, c = values((m, n), 13)
    check_product(fp4.fp4_product(a, b, out=c, accumulate=True), a64, b64, torch.float32, c64)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("shape", [(2048, 2048, 1408), (2047, 1409, 5000), (1100, 4000, 321)])
def test_large_products_match_the_oracle(fp4, shape, fmt):
    """Sizes on the path of CTA pairs, ragged in every dimension."""
    m, n, k = shape
    a, a64 = quantized(fp4, (m, k), 14, fmt)
    b, b64 = quantized(fp4, (n, k), 15, fmt)
    for dt in DT.values():
        check_product(fp4.fp4_product(a, b, out_dtype=dt), a64, b64, dt)
    assert fp4.fp4_status() == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("ld,off", [(400, 0), (401, 0), (400, 3), (353, 1)])
@pytest.mark.parametrize("m", [200, 2400])
def test_product_into_a_strided_output(fp4, m, ld, off, fmt):
    """Row pitches and offsets that allow vector stores and that do not; what lies between the rows stays."""
    k, n = 192, 350
    a, a64 = quantized(fp4, (m, k), 16, fmt)
    b, b64 = quantized(fp4, (n, k), 17, fmt)
    for dt in DT.values():
        big = torch.full((m + 2, ld), 5.0, dtype=dt, device="cuda")
        out = big[1:m + 1, off:off + n]
        fp4.fp4_product(a, b, out=out)
        check_product(out, a64, b64, dt)
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:m + 1, off:off + n] = False
        assert (big[keep] == 5.0).all()


@pytest.mark.parametrize("m", [3000, 40000])
@pytest.mark.parametrize("n", [264, 288, 392, 416, 520])
def test_product_with_a_narrow_last_tile(fp4, m, n):
    """Last column tiles of which a warp stores one block, many tiles a CTA:
    every column as that of a product with the last columns alone."""
    a = fp4.fp4_quantize(torch.randn(m, 96, device="cuda"), fmt="mx")
    w = torch.randn(n, 96, device="cuda")
    b = fp4.fp4_quantize(w, fmt="mx")
    for dt in DT.values():
        out = fp4.fp4_product(a, b, out_dtype=dt)
        for lo in range(0, n, 128):
            part = fp4.fp4_quantize(w[lo:lo + 128], fmt="mx")
            assert torch.equal(out[:, lo:lo + 128], fp4.fp4_product(a, part, out_dtype=dt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m", [200, 2400])
def test_product_nan_scales_stay_in_their_row_and_column(fp4, m, fmt):
    n, k = 1500, 300
    a64, x = values((m, k), 18)
    b64, w = values((n, k), 19)
    x[7, 299] = float("inf")
    w[1400, 0] = float("nan")
    a, b = fp4.fp4_quantize(x, fmt=fmt), fp4.fp4_quantize(w, fmt=fmt)
    out = fp4.fp4_product(a, b, out_dtype=torch.float32)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[7] = True
    bad[:, 1400] = True
    assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("m", [100, 2500])
def test_product_with_an_arbitrary_tensor_scale(fp4, m):
    """g of a checkpoint that is no power of two."""
    a, a64 = quantized(fp4, (m, 128), 20, "nv")
    b, b64 = quantized(fp4, (1300, 128), 21, "nv")
    ga, gb = a.tensor_scale[0].item(), b.tensor_scale[0].item()
    a.tensor_scale[0], b.tensor_scale[0] = 0.0123, 3.7
    fa, fb = a.tensor_scale[0].item() / ga, b.tensor_scale[0].item() / gb
    check_product(fp4.fp4_product(a, b, out_dtype=torch.float32), a64 * fa, b64 * fb, torch.float32)
    x64, x = values((3, 128), 22, "bf16")
    check_rows(fp4.fp4_rows_product(x, b, out_dtype=torch.float32), x64, b64 * fb, torch.float32)


@pytest.mark.parametrize("m", [40, 2500])
@pytest.mark.parametrize("ea,eb", [(110, -95), (-95, 110), (-60, -50), (60, 50)])
def test_product_of_operands_far_apart(fp4, m, ea, eb):
    """Tensor scales at the ends of fp32's range whose product is within it."""
    a64, x = values((m, 96), 43, "fp32", 0.0)
    b64, w = values((1400, 96), 44, "fp32", 0.0)
    x.mul_(2.0 ** ea)
    w.mul_(2.0 ** eb)
    for fmt in ("mx", "nv"):
        qv = lambda t: o.quantize(t.double().cpu().numpy(), fmt).values()  # noqa: E731
        got = fp4.fp4_product(fp4.fp4_quantize(x, fmt=fmt), fp4.fp4_quantize(w, fmt=fmt), out_dtype=torch.float32)
        check_product(got, qv(x), qv(w), torch.float32)


def test_products_of_nothing(fp4):
    """No rows, no columns, no k."""
    for fmt in ("mx", "nv"):
        e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        b = fp4.fp4_quantize(e(7, 40), fmt=fmt)
        none = fp4.fp4_quantize(e(0, 40), fmt=fmt)
        assert none.dequantize().shape == (0, 40)
        assert fp4.fp4_product(none, b).shape == (0, 7) and fp4.fp4_product(b, none).shape == (7, 0)
        flat = fp4.fp4_quantize(e(7, 0), fmt=fmt)
        out = torch.full((7, 9), 3.0, device="cuda")
        fp4.fp4_product(flat, fp4.fp4_quantize(e(5, 0), fmt=fmt), out=out[:, 2:7])
        assert (out[:, 2:7] == 0).all() and (out[:, :2] == 3).all() and (out[:, 7:] == 3).all()
        fp4.fp4_product(flat, fp4.fp4_quantize(e(9, 0), fmt=fmt), out=out.fill_(2.0), accumulate=True)
        assert (out == 2).all()
        assert fp4.fp4_rows_product(e(0, 40).bfloat16(), b).shape == (0, 7)
        assert (fp4.fp4_rows_product(e(3, 0).bfloat16(), flat) == 0).all()
        y, kept = fp4.fp4_linear(e(0, 40), e(40, 7), fmt=fmt)
        dx, dw = fp4.fp4_linear_backward(kept, e(0, 7))
        assert y.shape == (0, 7) and dx.shape == (0, 40) and (dw == 0).all() and dw.shape == (40, 7)
    torch.cuda.synchronize()


def check_rows(got, x, w, dtype):
    """fp32 sums of products: at most k roundings of partial sums, each at
    most the sum of magnitudes S, and two a product for its scales; bf16 rows
    are taken exactly, up to 2^-24 of S."""
    want = x @ w.T
    s = np.abs(x) @ np.abs(w).T
    tol = (x.shape[1] + 4) * 2.0 ** -24 * s
    tol = tol + HALF[dtype] * (np.abs(want) + tol) + 1e-38
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 2048, 2048), (2, 17, 31), (5, 2047, 1409), (8, 130, 64), (9, 300, 4096),
                                   (16, 1000, 257), (17, 64, 1000), (31, 129, 96), (32, 4096, 512), (1, 70000, 48)])
def test_rows_product_matches_the_oracle(fp4, t, n, k, fmt):
    x64, x = values((t, k), 23, "bf16")
    w, w64 = quantized(fp4, (n, k), 24, fmt)
    for dt in DT.values():
        check_rows(fp4.fp4_rows_product(x, w, out_dtype=dt), x64, w64, dt)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("t,n,k", [(1, 40, 10240), (3, 50, 10241), (20, 33, 20600), (32, 200, 10239)])
def test_rows_product_long_k(fp4, t, n, k, fmt):
    """k at, next to and past what shared memory holds of X at a time; a row
    alone gives the bits that it gives among others."""
    x64, x = values((t, k), 40, "bf16", 1.0)
    w, w64 = quantized(fp4, (n, k), 41, fmt)
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    check_rows(got, x64, w64, torch.float32)
    assert torch.equal(fp4.fp4_rows_product(x[t - 1:], w, out_dtype=torch.float32), got[t - 1:])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_product_extreme_rows(fp4, fmt):
    """Rows of zeros, of subnormals, near bf16's largest values, and of values
    2^40 apart: each keeps its own precision."""
    k, n = 256, 48
    x = torch.randn(6, k, device="cuda").bfloat16()
    x[1] = 0
    x[2] = (torch.randn(k, device="cuda") * 2.0 ** -128).bfloat16()
    x[3] = (torch.randn(k, device="cuda").clamp(-1, 1) * 2.0 ** 118).bfloat16()
    x[4, ::2] *= 2.0 ** 20
    x[4, 1::2] *= 2.0 ** -20
    x[5] = 2.0 ** -133
    w, w64 = quantized(fp4, (n, k), 42, fmt, 0.0)
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    check_rows(got, x.double().cpu().numpy(), w64, torch.float32)
    assert (got[1] == 0).all()


def test_offsets_past_32_bits(fp4):
    """Codes, sources and outputs of more than 2^31 bytes and 2^31 elements:
    the last rows are those of the last rows alone."""
    x = torch.empty(70000, 65536, dtype=torch.bfloat16, device="cuda")
    for i in range(0, 70000, 5000):
        x[i:i + 5000] = torch.randn(5000, 65536, device="cuda")
    m = fp4.fp4_quantize(x, fmt="mx")
    tail = fp4.fp4_quantize(x[-130:], fmt="mx")
    assert m.data.numel() > 2 ** 31
    assert torch.equal(m.data.view(70000, -1)[-130:], tail.data.view(130, -1))
    v = torch.empty_like(x)
    m.dequantize(out=v)
    assert torch.equal(v[-130:], tail.dequantize())
    del v
    tok = x[:2, :].contiguous()
    assert torch.equal(fp4.fp4_rows_product(tok, m)[:, -130:], fp4.fp4_rows_product(tok, tail))
    del x, m
    a = fp4.fp4_quantize(torch.randn(70000, 64, device="cuda"), fmt="mx")
    b = fp4.fp4_quantize(torch.randn(32768, 64, device="cuda"), fmt="mx")
    out = fp4.fp4_product(a, b)
    assert out.numel() > 2 ** 31
    last = fp4.fp4_quantize(a.dequantize()[-112:], fmt="mx")
    assert torch.equal(out[-112:], fp4.fp4_product(last, b))
    assert fp4.fp4_status() == 0


@pytest.mark.parametrize("along", ["cols", "rows"])
def test_more_tile_rows_than_a_grid_dimension(fp4, along):
    """Rows past 32768 tiles of 64."""
    rows = 32768 * 64 + 100
    x = torch.randn(rows, 33, device="cuda").bfloat16()
    m = fp4.fp4_quantize(x, fmt="mx", along=along)
    v = m.dequantize()
    cut = 32768 * 64 - 64
    tail = fp4.fp4_quantize(x[cut:], fmt="mx", along=along).dequantize()
    assert torch.equal(v[cut:] if along == "cols" else v[:, cut:], tail)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_product_strides_and_independence(fp4, fmt):
    """Strided rows and outputs, values of very different size, rows alone and
    together; NaN and infinity stay in their row."""
    t, n, k = 11, 333, 500
    _, big = values((t, k + 9), 25, "bf16", spread=3.0)
    w, w64 = quantized(fp4, (n, k), 26, fmt)
    for off in (0, 1, 8):
        x = big[:, off:off + k]
        out = torch.full((t, n + 5), 4.0, device="cuda")
        fp4.fp4_rows_product(x, w, out=out[:, 2:n + 2])
        check_rows(out[:, 2:n + 2], x.double().cpu().numpy(), w64, torch.float32)
        assert (out[:, :2] == 4).all() and (out[:, n + 2:] == 4).all()
    x = big[:, :k].contiguous()
    whole = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    for i in (0, 3, 10):
        assert torch.equal(fp4.fp4_rows_product(x[i:i + 1], w, out_dtype=torch.float32), whole[i:i + 1])
    x[4, 17] = float("inf")
    x[9, 499] = float("nan")
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    fine = [i for i in range(t) if i not in (4, 9)]
    assert torch.equal(got[fine], whole[fine])
    assert torch.isnan(got[9]).all() and not torch.isfinite(got[4]).any()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_product_nan_scale(fp4, fmt):
    w64, w = values((200, 96), 27)
    w[150, 95] = float("nan")
    q = fp4.fp4_quantize(w, fmt=fmt)
    _, x = values((3, 96), 28, "bf16")
    out = fp4.fp4_rows_product(x, q)
    assert torch.isnan(out[:, 150]).all() and torch.isfinite(out[:, :150]).all() and torch.isfinite(out[:, 151:]).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("t,k,n", [(1, 32, 16), (5, 100, 33), (130, 256, 140), (777, 512, 384)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_step_matches_the_oracle(fp4, t, k, n, dtype, fmt):
    x64, x = values((t, k), 29, dtype)
    w64, w = values((k, n), 30, "fp32")
    g64, dy = values((t, n), 31, dtype)
    qv = lambda m: o.quantize(m, fmt).values()  # noqa: E731
    y, kept = fp4.fp4_linear(x, w, fmt=fmt)
    dx, dw = fp4.fp4_linear_backward(kept, dy)
    check_product(y, qv(x64), qv(w64.T), torch.bfloat16)
    check_product(dx, qv(g64), qv(w64), torch.bfloat16)
    check_product(dw, qv(x64.T), qv(g64.T), torch.float32)
    # a pair of stored forms gives the same, and gradients accumulate
    y2, kept2 = fp4.fp4_linear(x, fp4.fp4_quantize(w, fmt=fmt, along="both"))
    assert torch.equal(y, y2)
    twice = dw.clone()
    fp4.fp4_linear_backward(kept2, dy, dw=twice, accumulate=True)
    check_product(twice, qv(x64.T), qv(g64.T), torch.float32, dw.double().cpu().numpy())
    g16 = torch.empty(k, n, dtype=torch.bfloat16, device="cuda")
    fp4.fp4_linear_backward(kept2, dy, dw=g16)
    check_product(g16, qv(x64.T), qv(g64.T), torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_gradients_against_differences(fp4, fmt):
    """On operands that 4 bits hold exactly (a 6 in every block) the layer is
    bilinear: a central difference of sum(y * dy) equals the gradient."""
    r = np.random.default_rng(32)
    pick = lambda *s: o.E2M1[r.integers(0, 8, s)] * r.choice([-1.0, 1.0], s)  # noqa: E731
    x, w, dy = pick(48, 64), pick(64, 40), pick(48, 40)
    for m in (x, w, dy):
        m[:, ::8] = 6.0
        m[::8, :] = 6.0
    x[5, 9], w[9, 13] = 1.0, 1.0
    cu = lambda m: torch.from_numpy(m.astype(np.float32)).cuda()  # noqa: E731

    def loss(x, w):
        return float((fp4.fp4_linear(cu(x), cu(w), fmt=fmt, out_dtype=torch.float32)[0].double() * cu(dy).double()).sum())

    _, kept = fp4.fp4_linear(cu(x), cu(w), fmt=fmt)
    dx, dw = fp4.fp4_linear_backward(kept, cu(dy), dx_dtype=torch.float32)
    step = np.zeros_like(x)
    step[5, 9] = 0.5
    assert loss(x + step, w) - loss(x - step, w) == float(dx[5, 9])
    step = np.zeros_like(w)
    step[9, 13] = 0.5
    assert loss(x, w + step) - loss(x, w - step) == float(dw[9, 13])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("along", ["cols", "rows", "both"])
def test_plan_equals_single_calls(fp4, along, fmt):
    """A list with ragged, tiny and empty matrices; run again after the tensors changed."""
    shapes = [(200, 96), (1, 1), (0, 8), (129, 300), (64, 2048), (257, 33), (5, 0)]
    xs = [values(s, 33 + i)[1] if 0 not in s else torch.zeros(*s, device="cuda") for i, s in enumerate(shapes)]
    plan = fp4.Fp4Plan(xs, fmt=fmt, along=along, values=torch.float32)
    for _ in range(2):
        plan.run()
        vals = plan.dequantize()
        for i, x in enumerate(xs):
            want = fp4.fp4_quantize(x, fmt=fmt, along=along)
            pairs = zip(plan.matrices[i], want) if along == "both" else [(plan.matrices[i], want)]
            for f, (m, q) in enumerate(pairs):
                assert torch.equal(m.data, q.data) and torch.equal(m.scales, q.scales)
                if fmt == "nv" and x.numel():
                    assert torch.equal(m.tensor_scale, q.tensor_scale)
                assert torch.equal(vals[f][i], q.dequantize(torch.float32))
        for x in xs:
            x.mul_(0.3).add_(0.01)
    plan.close()


def test_plan_refusals(fp4):
    x = torch.zeros(4, 32, device="cuda")
    with pytest.raises(ValueError):
        fp4.Fp4Plan([x, x.bfloat16()])
    with pytest.raises(TypeError):
        fp4.Fp4Plan([x], values=torch.float16)
    plan = fp4.Fp4Plan([x])
    with pytest.raises(Exception):
        plan.dequantize()


def test_front_end_refusals(fp4):
    x = torch.zeros(64, 64, device="cuda")
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, fmt="fp8")
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, along="diagonal")
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x.T[:32])
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x[0].expand(3, 64))
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x[0])
    with pytest.raises(TypeError):
        fp4.fp4_quantize(x.half())
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, out=fp4.Fp4Matrix.empty(64, 32, "nv"))
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, out=fp4.Fp4Matrix.empty(64, 64, "mx"))
    with pytest.raises(TypeError):
        fp4.fp4_quantize(x, along="both", out=fp4.Fp4Matrix.empty(64, 64, "nv"))
    a, b = fp4.fp4_quantize(x), fp4.fp4_quantize(x[:, :32])
    with pytest.raises(ValueError):
        fp4.fp4_product(a, b)
    with pytest.raises(ValueError):
        fp4.fp4_product(a, fp4.fp4_quantize(x, fmt="mx"))
    with pytest.raises(ValueError):
        fp4.fp4_product(a, a, accumulate=True)
    with pytest.raises(ValueError):
        fp4.fp4_product(a, a, out=torch.empty(64, 64, dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(ValueError):
        fp4.fp4_product(a, a, out=torch.empty(63, 64, device="cuda"))
    with pytest.raises(TypeError):
        fp4.fp4_product(a, a, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fp4.fp4_product(a, a, out=torch.empty(64, device="cuda").expand(64, 64))
    with pytest.raises(ValueError):
        fp4.fp4_rows_product(torch.zeros(33, 64, dtype=torch.bfloat16, device="cuda"), a)
    with pytest.raises(TypeError):
        fp4.fp4_rows_product(x[:3], a)
    with pytest.raises(ValueError):
        fp4.fp4_rows_product(x[:3, :32].bfloat16(), a)
    with pytest.raises(ValueError):
        fp4.fp4_linear(x, torch.zeros(32, 8, device="cuda"))
    with pytest.raises(ValueError):
        fp4.fp4_linear(x, (a, a), fmt="mx")
    y, kept = fp4.fp4_linear(x, x)
    with pytest.raises(ValueError):
        fp4.fp4_linear_backward(kept, x[:32])
    with pytest.raises(ValueError):
        fp4.fp4_linear_backward(kept, x, accumulate=True)
    with pytest.raises(ValueError):
        fp4.fp4_linear_backward(kept, x, dw=torch.empty(64, 64, dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(ValueError):
        fp4.fp4_linear_backward(kept, x, dw=torch.empty(64, 63, device="cuda"))
    with pytest.raises(TypeError):
        fp4.fp4_linear_backward(kept, x, dx_dtype=torch.float16)
    with pytest.raises(TypeError):
        fp4.fp4_linear(x, x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fp4.fp4_linear(x, x, fmt="int4")
    from matrix_orthogonalizing_optimizer_muon_b200 import _lib as L
    with pytest.raises(L.MuonError):  # the output over an operand
        short = fp4.fp4_quantize(x[:4])
        fp4.fp4_product(short, short, out=short.data[:64].view(torch.float32).view(4, 4))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_other_streams_and_repeats(fp4, fmt):
    """Calls on two streams at once, many times: bitwise the results of one alone."""
    _, x = values((700, 512), 34, "bf16")
    _, w = values((600, 512), 35)
    _, tok = values((4, 512), 36, "bf16")
    q, wq = fp4.fp4_quantize(x, fmt=fmt), fp4.fp4_quantize(w, fmt=fmt)
    want = fp4.fp4_product(q, wq), fp4.fp4_rows_product(tok, wq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[] for _ in streams]
    for _ in range(10):
        for s, g in zip(streams, got):
            qs = fp4.fp4_quantize(x, fmt=fmt, stream=s)
            ws = fp4.fp4_quantize(w, fmt=fmt, stream=s)
            g.append((qs, ws, fp4.fp4_product(qs, ws, stream=s), fp4.fp4_rows_product(tok, ws, stream=s)))
    torch.cuda.synchronize()
    for g in got:
        for qs, ws, y, r in g:
            assert torch.equal(qs.data, q.data) and torch.equal(ws.scales, wq.scales)
            assert torch.equal(y, want[0]) and torch.equal(r, want[1])
    assert fp4.fp4_status(streams[0]) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_captured_step_replays_on_new_inputs(fp4, fmt):
    """Forward, backward and few-row calls in one CUDA graph, a second graph
    beside it: replays on new inputs equal eager calls."""
    t, k, n = 300, 256, 200
    graphs = []
    for s in range(2):
        x, w, dy = (values(sh, 37 + s, d)[1] for sh, d in (((t, k), "bf16"), ((k, n), "fp32"), ((t, n), "bf16")))
        dw = torch.zeros(k, n, device="cuda")

        def step(x=x, w=w, dy=dy, dw=dw):
            y, kept = fp4.fp4_linear(x, w, fmt=fmt)
            dx, _ = fp4.fp4_linear_backward(kept, dy, dw=dw)
            return y, dx, fp4.fp4_rows_product(x[:3], fp4.fp4_quantize(w, fmt=fmt, along="rows"))

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, step, outs, (x, w, dy), dw))
    for seed in (50, 51):
        for graph, step, outs, ins, dw in graphs:
            for i, v in enumerate(ins):
                v.copy_(values(tuple(v.shape), seed + i)[1])
            graph.replay()
        graphs[0][0].replay()
        torch.cuda.synchronize()
        for graph, step, outs, ins, dw in graphs:
            got = [v.clone() for v in outs] + [dw.clone()]
            want = list(step()) + [dw]
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_training_run_with_the_optimizer_step(fp4):
    """Three steps of a two-layer model on 4-bit products: forward and
    backward read the plan's 4-bit weights, HybridStep (Muon on the matrices,
    AdamW on a gain) takes the gradients and refreshes them.  Every step's
    outputs against the oracle from the GPU's own weights, and the refreshed
    copies bitwise."""
    import oracle.muon_oracle as orc
    from _gpu import ABC32, LR, MU, WD, check_step
    from matrix_orthogonalizing_optimizer_muon_b200.api import HybridStep
    shapes = [(96, 160), (160, 64)]
    ws = [values(s, 60 + i, "fp32", 0.0)[1].mul_(0.05) for i, s in enumerate(shapes)]
    ms = [torch.zeros_like(w) for w in ws]
    gain, gm, gv = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    plan = fp4.Fp4Plan(ws, fmt="nv", along="both")
    opt = HybridStep(shapes, [64], momenta=ms, adam_states=[(gm, gv)], vector_g_dtypes=[torch.float32], fp4=plan)
    plan.run()
    h64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    qv = lambda m: o.quantize(m, "nv").values()  # noqa: E731
    rms = torch.zeros(2, device="cuda")
    for step in range(1, 4):
        x64, x = values((200, 96), 70 + step, "bf16", 0.3)
        h, kept0 = fp4.fp4_linear(x, plan.matrices[0])
        a = torch.relu(h)
        y, kept1 = fp4.fp4_linear(a, plan.matrices[1])
        check_product(h, qv(x64), qv(h64(ws[0]).T), torch.bfloat16)
        check_product(y, qv(h64(a)), qv(h64(ws[1]).T), torch.bfloat16)
        dout = ((y.float() * gain - x[:, :64].float()) / 200)
        dgain = (dout * y.float()).sum(0)
        dy = (dout * gain).to(torch.bfloat16)
        da, dw1 = fp4.fp4_linear_backward(kept1, dy)
        dh = torch.where(h > 0, da, 0)
        _, dw0 = fp4.fp4_linear_backward(kept0, dh)
        check_product(dw1, qv(h64(a).T), qv(h64(dy).T), torch.float32)
        check_product(dw0, qv(x64.T), qv(h64(dh).T), torch.float32)
        before = [h64(w) for w in ws], [h64(m) for m in ms]
        opt.step(list(zip(ws, (dw0, dw1), ms)), [(gain, dgain, gm, gv)], t=step, lr=LR, weight_decay=WD, momentum=MU,
                 coeffs=ABC32, update_rms=rms)
        for i, g in enumerate((dw0, dw1)):
            check_step(before[0][i], before[1][i], h64(g), h64(ws[i]), h64(ms[i]), float(rms[i]), lr=LR, wd=WD, mu=MU)
            for m, q in zip(plan.matrices[i], (o.quantize(h64(ws[i]), "nv"), o.quantize(h64(ws[i]).T, "nv"))):
                check_stored(m, q)
    assert opt.status() == 0 and fp4.fp4_status() == 0
    tok = x[:1]
    check_rows(fp4.fp4_rows_product(tok, plan.matrices[0][1]), h64(tok), qv(h64(ws[0]).T), torch.bfloat16)
    opt.close()
    plan.close()
