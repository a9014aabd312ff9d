"""Pins of the 4-bit oracle: against library roundings, closed forms and
properties; planted mistakes fail them.  CPU only."""

import numpy as np
import pytest
import torch

import oracle.fp4_oracle as o


def rng(seed=0):
    return np.random.default_rng(seed)


def f32(x):
    return np.asarray(x, dtype=np.float32).astype(np.float64)


def test_e4m3_table_is_torchs():
    b = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(b, o.E4M3)
    assert o.E4M3[-1] == 448.0


def test_e4m3_rounding_is_torchs():
    x = np.concatenate([f32(rng(1).uniform(0, 448, 4000)), f32(2.0 ** rng(2).uniform(-12, 8.8, 4000)), o.E4M3,
                        (o.E4M3[1:] + o.E4M3[:-1]) / 2])
    got = o.E4M3[o.nearest_even(x, o.E4M3, 1.0)]
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, want)


def test_e2m1_ties_and_saturation():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 7.0, 100.0, 0.0])
    got = o.E2M1[o.nearest_even(x, o.E2M1, 1.0)]
    assert list(got) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0, 0.0]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_representable_values_come_back(fmt):
    """Blocks that hold a 6 (mx: any binade of its scale; nv: the matrix's
    largest and block scales that e4m3 holds) are kept exactly."""
    r = rng(3)
    v = o.E2M1[r.integers(0, 8, (9, 96))] * r.choice([-1.0, 1.0], (9, 96))
    v[:, :: o.BLOCK[fmt]] = 6.0
    scale = 2.0 ** r.integers(-3, 4, (9, 96 // o.BLOCK[fmt]))
    x = v * np.repeat(scale, o.BLOCK[fmt], axis=1)
    assert np.array_equal(o.quantize(x, fmt).values(), x)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 17), (5, 100), (130, 64)])
def test_error_is_at_most_half_a_step(fmt, shape):
    x = f32(rng(4).standard_normal(shape) * np.exp(rng(5).standard_normal(shape)))
    q = o.quantize(x, fmt)
    unit = np.repeat(q.scales(), o.BLOCK[fmt], axis=1)[:, : shape[1]]
    a = np.abs(x)
    step = np.where(a < 2 * unit, 0.5, np.where(a < 4 * unit, 1.0, 2.0)) * unit
    # saturated values are off by what is past 6 scales: mx scales leave up to
    # 8, an nv scale rounded down (by at most 1/16) up to 6.4
    over = np.maximum(0.0, a - 6 * unit)
    assert np.all(np.abs(q.values() - x) <= step / 2 + over)
    assert np.all(over <= (2.0 if fmt == "mx" else 0.4) * unit + 1e-300)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_power_of_two_scaling(fmt):
    x = f32(rng(6).standard_normal((4, 70)))
    a, b = o.quantize(x, fmt), o.quantize(x * 2.0 ** 9, fmt)
    assert np.array_equal(a.codes, b.codes) and np.array_equal(a.values() * 2.0 ** 9, b.values())


def test_tensor_scale_is_the_least_power_of_two():
    for amax in (2688.0, np.nextafter(np.float32(2688.0), np.float32(3000)), 1.0, 0.0137, 3.4e38, 1e-30, 0.0):
        g, a = o.tensor_scale(np.array([[float(amax), 0.0]]))
        assert o.is_power_of_two(g) and a <= 2688 * g and (g == 2.0 ** -100 or a > 2688 * g / 2)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_non_finite_blocks(fmt):
    x = f32(rng(7).standard_normal((2, 96)))
    clean = o.quantize(x, fmt).values()
    x[0, 40] = np.inf
    x[1, 3] = np.nan
    v = o.quantize(x, fmt).values()
    blk = o.BLOCK[fmt]
    bad = np.zeros((2, 96), dtype=bool)
    bad[0, 40 // blk * blk: 40 // blk * blk + blk] = True
    bad[1, :blk] = True
    assert np.isnan(v[bad]).all()
    if fmt == "mx":  # nv: the largest magnitude may have been in a bad block
        assert np.array_equal(v[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_storage_round_trip(fmt):
    """The stored bytes read back by the documented formula, byte by byte."""
    x = f32(rng(8).standard_normal((150, 77)))
    q = o.quantize(x, fmt)
    data, scales = q.stored()
    blk = o.BLOCK[fmt]
    nb = -(-77 // blk)
    assert data.shape == (150, 48) and scales.size == 2 * -(-nb // 4) * 512
    val = q.values()
    for r in (0, 31, 32, 127, 128, 149):
        for k in (0, 1, 15, 16, 63, 76):
            code = (data[r, k // 2] >> (4 * (k % 2))) & 15
            b = k // blk
            byte = scales[(r // 128 * -(-nb // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]
            s = 2.0 ** (float(byte) - 127) if fmt == "mx" else o.E4M3[byte] * q.g
            assert (-1.0 if code & 8 else 1.0) * o.E2M1[code & 7] * s == val[r, k]


def test_linear_equals_the_exact_layer_on_representable_operands():
    """With every operand representable in 4 bits the layer is linear, and its
    gradients are those of sum(y * dy): checked against central differences,
    which are exact for a bilinear function up to rounding."""
    r = rng(9)
    pick = lambda *s: o.E2M1[r.integers(0, 8, s)] * r.choice([-1.0, 1.0], s)  # noqa: E731
    x, w, dy = pick(8, 40), pick(40, 12), pick(8, 12)
    for m in (x, w, dy):  # a 6 in every block of either direction fixes the block scales at 1
        m[:, ::8] = 6.0
        m[::8, :] = 6.0
    for fmt in ("mx", "nv"):
        y, dx, dw = o.linear(x, w, dy, fmt)
        assert np.array_equal(y, x @ w) and np.array_equal(dx, dy @ w.T) and np.array_equal(dw, x.T @ dy)
    loss = lambda x, w: float(np.sum((x @ w) * dy))  # noqa: E731
    for i, j in ((0, 0), (3, 17), (7, 39)):
        d = np.zeros_like(x)
        d[i, j] = 0.5
        assert abs((loss(x + d, w) - loss(x - d, w)) - dx[i, j]) < 1e-9
    for i, j in ((0, 0), (21, 5), (39, 11)):
        d = np.zeros_like(w)
        d[i, j] = 0.5
        assert abs((loss(x, w + d) - loss(x, w - d)) - dw[i, j]) < 1e-9


def test_planted_mistakes_are_caught(monkeypatch):
    def ties_away(x, grid, unit):
        idx = np.zeros(x.shape, dtype=np.int64)
        for i in range(1, len(grid)):
            idx += x >= (grid[i] + grid[i - 1]) / 2 * unit
        return idx

    with monkeypatch.context() as m:
        m.setattr(o, "nearest_even", ties_away)
        with pytest.raises(AssertionError):
            test_e2m1_ties_and_saturation()
    with monkeypatch.context() as m:
        m.setattr(o, "tensor_scale", lambda x: (float(np.abs(x).max()) / 2688, float(np.abs(x).max())))
        with pytest.raises(AssertionError):
            test_tensor_scale_is_the_least_power_of_two()
    right = o.Fp4.stored

    def swapped(self):
        data, scales = right(self)
        return (data << 4) | (data >> 4), scales

    with monkeypatch.context() as m:
        m.setattr(o.Fp4, "stored", swapped)
        with pytest.raises(AssertionError):
            test_storage_round_trip("mx")
