"""A 4-bit product whose device-side wait runs out, without a fault: the wait
is on a barrier that nothing arrives at, with a limit of microseconds, before
any load or tensor-core instruction.  It is reported once, and the next
product is right."""

import pytest
import torch

from matrix_orthogonalizing_optimizer_muon_b200 import _lib as L
from test_gpu_fp4 import check_product, quantized

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wait_ns", [2000, 50000])
@pytest.mark.parametrize("m", [100, 2400])
def test_timed_out_product_is_reported_and_the_next_one_is_right(m, wait_ns):
    """Single CTAs and CTA pairs."""
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4
    a, a64 = quantized(fp4, (m, 512), 1, "nv")
    b, b64 = quantized(fp4, (1500, 512), 2, "nv")
    out = torch.full((m, 1500), 7.0, device="cuda")
    assert fp4.fp4_status() == L.MUON_OK
    L.muon_fp4_inject_wait_timeout(wait_ns)
    fp4.fp4_product(a, b, out=out)
    assert fp4.fp4_status() == L.MUON_ERR_TIMEOUT
    assert fp4.fp4_status() == L.MUON_OK  # read-and-clear
    assert (out == 7.0).all()
    check_product(fp4.fp4_product(a, b, out=out), a64, b64, torch.float32)
    assert fp4.fp4_status() == L.MUON_OK
    out.fill_(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fp4.fp4_product(a, b, out=out, stream=side)
    assert fp4.fp4_status(side) == L.MUON_OK  # synchronises it
    check_product(out, a64, b64, torch.float32)


def test_injection_arguments_are_checked():
    for bad in (0, 1000000001):
        with pytest.raises(L.MuonError) as e:
            L.muon_fp4_inject_wait_timeout(bad)
        assert e.value.status == L.MUON_ERR_INVALID_ARG
