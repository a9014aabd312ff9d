"""Plain fp64 oracle of the microscaled 4-bit matrices (numpy only).

Every rounding is decided by comparing exact fp64 quantities: block scales
and codes are found among all their candidate values, with the midpoints'
products as borders (a source value has at most 24 significant bits, a
midpoint times a scale at most 7, times a power of two).  Shares no code with
the GPU path.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = {"mx": 32, "nv": 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3: byte -> value (sign bit clear); 0x7f is NaN
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])


def nearest_even(x: np.ndarray, grid: np.ndarray, unit) -> np.ndarray:
    """Index of the value of `grid` (times `unit`) nearest to x >= 0; ties go
    to the even index, values past the end to the last."""
    idx = np.zeros(x.shape, dtype=np.int64)
    for i in range(1, len(grid)):
        border = (grid[i] + grid[i - 1]) / 2 * unit
        idx += (x > border) | ((x == border) & (i % 2 == 0))
    return idx


def tensor_scale(x: np.ndarray):
    """(g, amax): the least power of two >= 2^-100 with amax <= 2688 g, amax
    the largest finite magnitude."""
    a = np.abs(x[np.isfinite(x)])
    amax = float(a.max()) if a.size else 0.0
    e = -100
    while amax > 2688.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e, amax


class Fp4:
    """codes [rows, k] (0..15), scale bytes [rows, blocks], g, amax."""

    def __init__(self, codes, scale_bytes, g, amax, fmt, k):
        self.codes, self.scale_bytes, self.g, self.amax, self.fmt, self.k = codes, scale_bytes, g, amax, fmt, k

    def scales(self) -> np.ndarray:
        if self.fmt == "mx":
            s = 2.0 ** (self.scale_bytes.astype(np.float64) - 127)
            return np.where(self.scale_bytes == 255, np.nan, s)
        s = np.append(E4M3, np.nan)[self.scale_bytes & 127]
        return np.where(self.scale_bytes & 128, -s, s) * self.g

    def values(self) -> np.ndarray:
        v = E2M1[self.codes & 7] * np.where(self.codes & 8, -1.0, 1.0)
        return v * np.repeat(self.scales(), BLOCK[self.fmt], axis=1)[:, : self.k]

    def stored(self):
        """(codes as bytes [rows, pitch], scale bytes in atoms), padding zero."""
        rows = self.codes.shape[0]
        pitch = 16 * -(-self.k // 32)
        data = np.zeros((rows, pitch), dtype=np.uint8)
        for half in (0, 1):
            c = self.codes[:, half::2].astype(np.uint8)
            data[:, : c.shape[1]] |= c << (4 * half)
        nb = self.scale_bytes.shape[1]
        atoms = -(-nb // 4)
        out = np.zeros((-(-rows // 128), atoms, 32, 4, 4), dtype=np.uint8)  # row block, atom, r % 32, r / 32, b % 4
        for b in range(nb):
            for r0 in range(0, rows, 32):
                n = min(32, rows - r0)
                out[r0 // 128, b // 4, :n, r0 % 128 // 32, b % 4] = self.scale_bytes[r0:r0 + n, b]
        return data, out.reshape(-1)


def quantize(x: np.ndarray, fmt: str) -> Fp4:
    """x [rows, k] in blocks along k.  Codes of a block whose scale is NaN are 0 here."""
    rows, k = x.shape
    blk = BLOCK[fmt]
    nb = -(-k // blk)
    xp = np.zeros((rows, nb * blk))
    xp[:, :k] = x
    xb = xp.reshape(rows, nb, blk)
    bad = ~np.isfinite(xb).all(axis=2)
    xb = np.where(bad[:, :, None], 0.0, xb)
    amax_b = np.abs(xb).max(axis=2) if k else np.zeros((rows, 0))
    g, amax = tensor_scale(x)
    if fmt == "mx":
        # floor(log2 amax) from frexp, which is exact; the exponent byte is at least 0
        e = np.where(amax_b > 0, np.frexp(amax_b)[1] - 1 - 2, -127)
        byte = np.clip(e + 127, 0, 254)
        unit = 2.0 ** (byte.astype(np.float64) - 127)
        byte = np.where(bad, 255, byte)
    else:
        byte = nearest_even(amax_b, E4M3, 6 * g)
        unit = E4M3[byte] * g
        byte = np.where(bad, 127, byte)
    idx = nearest_even(np.abs(xb), E2M1, unit[:, :, None])
    idx = np.where((unit > 0)[:, :, None], idx, 0)
    codes = np.where(np.signbit(xb), idx + 8, idx).reshape(rows, -1)[:, :k]
    return Fp4(codes, byte.astype(np.int64), g, amax, fmt, k)


def product(a: Fp4, b: Fp4) -> np.ndarray:
    return a.values() @ b.values().T


def linear(x, w, dy, fmt):
    """(y, dx, dw) of a linear layer whose three products round their
    operands to 4 bits along the summed dimension; w is [K, N]."""
    y = product(quantize(x, fmt), quantize(w.T, fmt))
    dx = product(quantize(dy, fmt), quantize(w, fmt))
    dw = product(quantize(x.T, fmt), quantize(dy.T, fmt))
    return y, dx, dw


def is_power_of_two(v: float) -> bool:
    return v > 0 and math.frexp(v)[0] == 0.5
