"""Paths of the 4-bit operators that need larger sizes: accumulation by CTA
pairs, and NV sources of more than 2^31 elements."""

import pytest
import torch

import oracle.fp4_oracle as o
from test_gpu_fp4 import check_product, quantized, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4():
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4 as m
    return m


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(200, 350, 192), (2400, 1350, 320), (2048, 1408, 777), (2300, 1301, 100)])
@pytest.mark.parametrize("ld,off", [(None, 0), (1500, 0), (1500, 4), (1501, 0), (1500, 3)])
def test_accumulation_into_strided_outputs(fp4, m, n, k, ld, off, fmt):
    """Few tiles (single CTAs) and many (pairs), rows that the TMA reduction
    takes and rows that it does not: the sum within its bound, twice the same
    bits, and what lies between the rows stays."""
    a, a64 = quantized(fp4, (m, k), 16, fmt)
    b, b64 = quantized(fp4, (n, k), 17, fmt)
    c64, c = values((m, n), 18)
    runs = []
    for _ in range(2):
        big = torch.full((m + 2, ld or n), 5.0, device="cuda")
        out = big[1:m + 1, off:off + n]
        out.copy_(c)
        fp4.fp4_product(a, b, out=out, accumulate=True)
        check_product(out, a64, b64, torch.float32, c64)
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:m + 1, off:off + n] = False
        assert (big[keep] == 5.0).all()
        runs.append(out.clone())
    assert torch.equal(*runs)
    assert fp4.fp4_status() == 0


@pytest.mark.parametrize("along", ["cols", "rows"])
def test_nv_sources_past_32_bits(fp4, along):
    """The largest magnitude lies in the last row, past 2^31 elements: the
    last rows' codes and scales are those of the last rows alone."""
    x = torch.empty(70000, 32768, dtype=torch.bfloat16, device="cuda")
    for i in range(0, 70000, 5000):
        x[i:i + 5000] = torch.randn(5000, 32768, device="cuda")
    x[-1, -1] = 300.0
    assert x.numel() > 2 ** 31
    cut = 70000 // 128 * 128 - 128  # a whole scale atom before the end
    m = fp4.fp4_quantize(x, fmt="nv", along=along)
    tail = fp4.fp4_quantize(x[cut:], fmt="nv", along=along)
    assert m.tensor_scale[1] == 300.0 and torch.equal(m.tensor_scale, tail.tensor_scale)
    if along == "cols":
        assert torch.equal(m.data.view(70000, -1)[cut:], tail.data.view(70000 - cut, -1))
        n = tail.scales.numel()
        assert torch.equal(m.scales[-n:], tail.scales)
    else:
        pitch, tp = 16 * -(-70000 // 32), 16 * -(-(70000 - cut) // 32)
        assert torch.equal(m.data.view(32768, pitch)[:, cut // 2:], tail.data.view(32768, tp))
        v = m.dequantize()
        assert torch.equal(v[:, cut:], tail.dequantize())
