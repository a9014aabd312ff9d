"""The 4-bit operators at the ends of their ranges: few-row products whose
rows and scales spread over all of bf16 and e8m0."""

import numpy as np
import pytest
import torch

import oracle.fp4_oracle as o
from test_gpu_fp4 import check_product, check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4():
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4 as m
    return m


def matrix(fp4, codes, byte, fmt, g=1.0):
    """(Fp4Matrix, its values in fp64) of given codes [rows, k] and scale bytes [rows, blocks]."""
    q = o.Fp4(codes, byte, g, 0.0, fmt, codes.shape[1])
    data, scales = q.stored()
    ts = torch.tensor([g, 0.0], device="cuda") if fmt == "nv" else None
    m = fp4.Fp4Matrix(*codes.shape, fmt, torch.from_numpy(data).cuda(), torch.from_numpy(scales).cuda(), ts)
    return m, q.values()


def ones(rows, k, fmt):
    """Scale bytes of 1."""
    return np.full((rows, -(-k // o.BLOCK[fmt])), 127 if fmt == "mx" else 0x38)


def bf16(x):
    t = torch.from_numpy(x.astype(np.float32)).cuda().to(torch.bfloat16)
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_product_keeps_a_value_far_below_the_largest(fp4, fmt):
    """2^30 meets a zero code: what is left of the row is the result, to the bit."""
    codes = np.array([[0, 2, 0, 2]])  # 0 and 1
    w, w64 = matrix(fp4, codes, ones(1, 4, fmt), fmt)
    x, x64 = bf16(np.array([[2.0 ** 30, 2.0 ** -10, -(2.0 ** 90), 0.0],
                            [-(2.0 ** 127), 2.0 ** -133, 0.0, 0.0],
                            [2.0 ** 22, 3 * 2.0 ** -20, 1.0, 2.0 ** -18]]))
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32).double().cpu().numpy()
    assert np.array_equal(got, x64 @ w64.T)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("t,n,k", [(1, 40, 96), (3, 300, 2048), (7, 33, 1409), (12, 100, 512), (32, 70, 200), (5, 48, 10500), (20, 50, 6000)])
def test_rows_product_of_rows_that_spread_over_the_whole_range(fp4, t, n, k, fmt):
    """Every row's values lie in groups down to 2^-250 of its largest, and each
    row of W is zero under all groups above one of its own: each output within
    the fp32 bound of the products that it is made of, and a row alone gives
    the bits that it gives among others."""
    r = np.random.default_rng(t * 1000 + k)
    groups = np.array([100, 60, 31, 1, -1, -30, -35, -70, -100])
    at = r.integers(0, len(groups), k)
    x64 = r.standard_normal((t, k)) * 2.0 ** groups[at]
    x64[0] = r.standard_normal(k)              # an ordinary row among them
    if t > 2:
        x64[1] *= 2.0 ** -20
        x64[2, at < 4] = 0.0
    x, x64 = bf16(x64)
    codes = r.integers(0, 16, (n, k))
    codes[at[None, :] < r.integers(0, len(groups), n)[:, None]] = 0
    byte = r.integers(110, 140, (n, -(-k // 32))) if fmt == "mx" else r.integers(1, 127, (n, -(-k // 16)))
    w, w64 = matrix(fp4, codes, byte, fmt, 2.0 ** -6)
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    check_rows(got, x64, w64, torch.float32)
    for i in {0, 1 % t, t - 1}:
        assert torch.equal(fp4.fp4_rows_product(x[i:i + 1], w, out_dtype=torch.float32), got[i:i + 1])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_product_spread_rows_with_nan_and_infinity(fp4, fmt):
    """A NaN or an infinity in a row of several parts stays in its row, and a NaN scale in its column."""
    r = np.random.default_rng(5)
    x, x64 = bf16(r.standard_normal((4, 256)) * 2.0 ** r.integers(-100, 100, 256))
    codes = r.integers(1, 8, (40, 256))
    byte = ones(40, 256, fmt)
    w, w64 = matrix(fp4, codes, byte, fmt)
    whole = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    check_rows(whole, x64, w64, torch.float32)
    x[1, 100], x[3, 0] = float("nan"), float("inf")
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    assert torch.equal(got[0::2], whole[0::2])
    assert torch.isnan(got[1]).all() and (got[3] == float("inf")).all()
    byte[7, 3] = 255 if fmt == "mx" else 127
    w, _ = matrix(fp4, codes, byte, fmt)
    got = fp4.fp4_rows_product(x[::2].contiguous(), w, out_dtype=torch.float32)
    assert torch.isnan(got[:, 7]).all()
    keep = [j for j in range(40) if j != 7]
    assert torch.equal(got[:, keep], whole[0::2][:, keep])


@pytest.mark.parametrize("t,n,k", [(3, 200, 64), (9, 100, 4096), (32, 33, 500), (2, 40, 10400)])
@pytest.mark.parametrize("spread", [0, 60])
def test_rows_product_mx_over_the_whole_range_of_scales(fp4, t, n, k, spread):
    """MX scales from 2^-127 to 2^127 with rows of X of any size (and, with
    spread, of many sizes within): whatever is within fp32's range is within
    the bound of its sum, and repeated calls give the same bits."""
    r = np.random.default_rng(n + k)
    nb = -(-k // 32)
    centre = r.integers(0, 255, n)             # every row of W around a size of its own
    centre[:4] = (0, 1, 253, 254)
    byte = np.clip(centre[:, None] + r.integers(-6, 7, (n, nb)), 0, 254)
    byte[4:n // 2] = r.integers(0, 255, (n // 2 - 4, nb)) # or all sizes in one row
    codes = r.integers(0, 16, (n, k))
    w, w64 = matrix(fp4, codes, byte, "mx")
    e = np.linspace(-120, 120, t)[:, None] + r.integers(-spread, spread + 1, k)
    x, x64 = bf16(np.clip(r.standard_normal((t, k)), -2, 2) * 2.0 ** np.clip(e, -130, 126))
    got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    s = np.abs(x64) @ np.abs(w64).T
    fits = s < 2.0 ** 127
    assert fits.any() and (s[fits] > 2.0 ** 100).any()
    g64 = got.double().cpu().numpy()
    tol = (k + 4) * 2.0 ** -24 * s + 2.0 ** -24 * np.abs(x64 @ w64.T) + (nb + 20) * 2.0 ** -149
    err = np.abs(g64 - x64 @ w64.T)
    assert (err <= tol)[fits].all(), float(np.max((err / tol)[fits]))
    again = fp4.fp4_rows_product(x, w, out_dtype=torch.float32)
    assert torch.equal(again.view(torch.int32), got.view(torch.int32))


def test_rows_product_mx_tiny_rows_and_large_scales(fp4):
    """A row of 2^-60 against scales of 2^115 to 2^125 over a long k, and the
    same with a zero block of the largest scale beside blocks of the least."""
    r = np.random.default_rng(8)
    codes = r.integers(0, 16, (64, 8192))
    w, w64 = matrix(fp4, codes, r.integers(242, 253, (64, 256)), "mx")
    x, x64 = bf16(r.standard_normal((2, 8192)) * 2.0 ** -60)
    check_rows(fp4.fp4_rows_product(x, w, out_dtype=torch.float32), x64, w64, torch.float32)
    byte = np.zeros((64, 256), dtype=np.int64)
    byte[:, ::7] = 254
    codes.reshape(64, 256, 32)[:, ::7] = 0
    w, w64 = matrix(fp4, codes, byte, "mx")
    x, x64 = bf16(r.standard_normal((2, 8192)) * 2.0 ** 120)
    check_rows(fp4.fp4_rows_product(x, w, out_dtype=torch.float32), x64, w64, torch.float32)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_new_plan_holds_its_tensors(fp4, fmt):
    """The documented order, a layer on a plan that was only made: the bits of the weights' own quantisation."""
    junk = torch.full((1 << 24,), 0x77, dtype=torch.uint8, device="cuda")
    del junk  # what the plan's storage may hold before
    r = np.random.default_rng(3)
    ws = [torch.from_numpy(r.standard_normal(s).astype(np.float32)).cuda() for s in ((300, 200), (64, 96))]
    x = torch.from_numpy(r.standard_normal((40, 300)).astype(np.float32)).cuda()
    plan = fp4.Fp4Plan(ws, fmt=fmt, along="both", values=torch.bfloat16)
    y, _ = fp4.fp4_linear(x, plan.matrices[0])
    assert torch.equal(y, fp4.fp4_linear(x, ws[0], fmt=fmt)[0])
    for i, w in enumerate(ws):
        for m, q in zip(plan.matrices[i], fp4.fp4_quantize(w, fmt=fmt, along="both")):
            assert torch.equal(m.data, q.data) and torch.equal(m.scales, q.scales)
    plan.close()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_codes_past_k_are_zero_beside_a_value_that_is_not_finite(fp4, bad, dtype, fmt):
    """The last, partial block of a row and of a column holds a NaN or an infinity; the storage past it is 0."""
    for rows, k in ((150, 200), (3, 17), (70, 33), (1, 1)):
        x = torch.randn(rows, k, device="cuda").to(dtype)
        x[rows - 1, k - 1] = bad
        for m in fp4.fp4_quantize(x, fmt=fmt, along="both"):
            data = m.data.view(m.rows, -1)
            codes = torch.stack([data & 15, data >> 4], -1).flatten(1)
            assert codes.shape[1] >= m.k and (codes[:, m.k:] == 0).all()
            assert torch.isnan(m.dequantize()[-1, -1])


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_nv_midpoints_near_the_largest_values(fp4, dtype, rows):
    """Midpoints of the codes and their fp32 neighbours under every scale of
    the matrix scales 2^112 to 2^117: bitwise the oracle, as a small matrix and
    behind a pass of its own."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    top = float(np.finfo(np.float32).max)
    for e in (112, 115, 116, 117):
        blocks = []
        for s in o.E4M3[1:]:
            d = s * 2.0 ** e
            if 6 * d * (1 + 2.0 ** -4) > top:
                continue
            v = (mids * d).astype(np.float32)
            for near in (v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))):
                row = np.zeros(16, dtype=np.float32)
                row[0], row[1:8], row[8:15] = 6 * d, near, -near
                blocks.append(row)
        x = np.stack(blocks).reshape(1, -1)
        x[0, 0] = min(2688.0 * 2.0 ** e, top)  # the matrix's largest: g = 2^e
        t = torch.from_numpy(np.repeat(x, rows, 0)).cuda().to(dtype)
        m64 = t.double().cpu().numpy()
        want = o.quantize(m64, "nv")
        assert want.g == 2.0 ** e
        got = fp4.fp4_quantize(t, fmt="nv")
        data, scales = want.stored()
        fine = np.repeat(want.scale_bytes != 127, 8, axis=1)  # as bf16 the largest fp32 is an infinity: its block has no codes
        assert np.array_equal(got.data.cpu().numpy().reshape(data.shape)[:, :fine.shape[1]][fine], data[:, :fine.shape[1]][fine])
        assert np.array_equal(got.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("ga,gb", [(1.37 * 2.0 ** -140, 1.7 * 2.0 ** 122), (2.0 ** 120, -(2.0 ** -149)),
                                   (1.9 * 2.0 ** -120, 1.1 * 2.0 ** 60), (2.0 ** -100, 2.0 ** -20), (2.0 ** 127, 2.0 ** -127)])
@pytest.mark.parametrize("m", [40, 2500])
def test_products_with_tensor_scales_at_the_ends_of_fp32(fp4, m, ga, gb):
    """Tensor scales of a checkpoint, subnormal ones too: fp32 sums times both
    scales, and rows of X as large or small as the scale is small or large."""
    r = np.random.default_rng(9)
    n, k = 1300, 200
    both = []
    for rows, g in ((m, ga), (n, gb)):
        g = float(np.float32(g))
        both.append(matrix(fp4, r.integers(0, 16, (rows, k)), r.integers(1, 127, (rows, -(-k // 16))), "nv", g))
    (a, a64), (b, b64) = both
    check_product(fp4.fp4_product(a, b, out_dtype=torch.float32), a64, b64, torch.float32)
    up = float(np.clip(-np.round(np.log2(abs(gb))), -105, 105))
    x, x64 = bf16(r.standard_normal((5, k)) * 2.0 ** up)
    check_rows(fp4.fp4_rows_product(x, b, out_dtype=torch.float32), x64, b64, torch.float32)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_product_counts_subnormals_once(fp4, fmt):
    """Rows whose parts end at the subnormals beside a row with more parts,
    for every exponent of the largest value: a subnormal is in one part."""
    w, w64 = matrix(fp4, np.array([[0, 2, 2, 2]]), ones(1, 4, fmt), fmt)
    for e0 in range(-126, 128, 31):
        x = np.zeros((32, 4))
        for i in range(31):
            x[i] = 2.0 ** min(e0 + i, 127), 3 * 2.0 ** -133, 2.0 ** -126, 2.0 ** -132
        x[31] = 2.0 ** 127, 2.0 ** -133, 0.0, 0.0
        x, x64 = bf16(x)
        got = fp4.fp4_rows_product(x, w, out_dtype=torch.float32).double().cpu().numpy()
        assert np.array_equal(got, x64 @ w64.T)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_rows_product_of_spread_rows_strided_captured_and_side_by_side(fp4, off, fmt):
    """Rows of several parts inside larger rows, aligned and not, into strided
    bf16 and fp32 outputs; a graph that was captured on ordinary rows replayed
    on them; two streams at once."""
    r = np.random.default_rng(12 + off)
    t, n, k = 11, 333, 500
    big = torch.zeros(t, k + 12, dtype=torch.bfloat16, device="cuda")
    x = big[:, off:off + k]
    x.copy_(torch.from_numpy(r.standard_normal((t, k)).astype(np.float32)))
    codes = r.integers(0, 16, (n, k))
    codes[::3, :k // 2] = 0
    byte = r.integers(0, 255, (n, -(-k // 32))) // 4 + 95 if fmt == "mx" else r.integers(1, 127, (n, -(-k // 16)))
    w, w64 = matrix(fp4, codes, byte, fmt)
    outs = {dt: torch.full((t, n + 5), 4.0, dtype=dt, device="cuda") for dt in (torch.float32, torch.bfloat16)}

    def run():
        for out in outs.values():
            fp4.fp4_rows_product(x, w, out=out[:, 2:n + 2])

    def check():
        for dt, out in outs.items():
            check_rows(out[:, 2:n + 2], x.double().cpu().numpy(), w64, dt)
            assert (out[:, :2] == 4).all() and (out[:, n + 2:] == 4).all()

    run()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    x[:, :k // 2] *= 2.0 ** 60
    x[3] *= 2.0 ** -50
    graph.replay()
    torch.cuda.synchronize()
    check()
    want = outs[torch.float32][:, 2:n + 2].clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fp4.fp4_rows_product(x, w, out_dtype=torch.float32, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
