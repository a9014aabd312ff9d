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


def test_optimizer_and_pack_plans_run_at_once_on_a_side_stream():
    """Muon, AdamW, entropy and pack plans: the bits of a plan used where it was made."""
    from matrix_orthogonalizing_optimizer_muon_b200.api import AdamWPlan, EntropyPlan, MuonPlan, PackPlan
    g = torch.Generator(device="cuda").manual_seed(2)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    shapes = [(64, 96), (130, 70), (256, 256)] * 30
    ws, gs, ms = ([new(*s) for s in shapes] for _ in range(3))
    vs = [(new(n), new(n), new(n), new(n).abs()) for n in (1000, 7, 70000)]
    dsts = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes]

    def run(stream):
        """Everything from the same values on `stream`; the results."""
        w, m = [t.clone() for t in ws], [t.clone() for t in ms]
        v = [tuple(t.clone() for t in q) for q in vs]
        h = torch.empty(len(shapes), device="cuda")
        for d in dsts:
            d.zero_()
        torch.cuda.synchronize()
        plan = MuonPlan(shapes)
        plan.step(list(zip(w, gs, m)), lr=0.02, weight_decay=0.1, stream=stream)
        adam = AdamWPlan([q[0].numel() for q in v], g_dtypes=[torch.float32] * len(v))
        adam.step(v, step=3, lr=0.01, weight_decay=0.1, stream=stream)
        ent = EntropyPlan(shapes)
        ent.compute(ws, h, stream=stream)
        pack = PackPlan(list(zip(ws, dsts)))
        pack.run(stream=stream)
        torch.cuda.synchronize()
        assert plan.status() == 0
        for p in (plan, adam, ent, pack):
            p.close()
        return w + m + [t for q in v for t in q] + [h] + [d.clone() for d in dsts]

    want = run(None)
    for _ in range(3):
        for a, b in zip(run(torch.cuda.Stream()), want):
            assert torch.equal(a, b)
