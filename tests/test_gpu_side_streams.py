"""Plans whose first use is on another stream than the one that they were made
on, right after they were made."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_fp4_plan_runs_at_once_on_a_side_stream(fmt):
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [torch.randn(r, c, generator=g, device="cuda") for r, c in ((2048, 1408), (129, 300), (5, 7)) * 20]
    want = [fp4.fp4_quantize(x, fmt=fmt, along="both") for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        side = torch.cuda.Stream()
        plan = fp4.Fp4Plan(xs, fmt=fmt, along="both", values=torch.float32)
        plan.run(stream=side)
        cols, rows = plan.dequantize(stream=side)
        side.synchronize()
        for i, pair in enumerate(want):
            for m, q, v in zip(plan.matrices[i], pair, (cols[i], rows[i])):
                assert torch.equal(m.data, q.data) and torch.equal(m.scales, q.scales)
                assert torch.equal(v, q.dequantize(torch.float32))
        plan.close()
