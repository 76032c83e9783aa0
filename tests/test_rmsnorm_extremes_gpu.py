"""The root-mean-square norm where numbers end (infinities, NaN, squares and products beyond fp32), beside
the borders between two 8-bit codes, in every layout to and from 8 bits, and with many rows a CTA.

Tolerances are those of the operators' tests: 1e-5 max|y| per element, 1e-4 max|y| for sums, plus 2^-8 |y|
for a rounding to bf16; what is held in 8 bits is compared bit by bit."""
import numpy as np
import pytest

import oracle.gated as og
from gated_cases import rms_inputs, rounded
from test_gated_gpu import EL, SUM, act, built, check, cuda, held_bits, wide  # noqa: F401 (built: the fixture)

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_rows_in_many_turns(dtype):
    """More rows of more than 8192 columns than the GPU holds CTAs for, the sum in the residual's place."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    rows, n = 1501, 8203
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *a: torch.randn(*a, generator=g, device="cuda").to(act(dtype))  # noqa: E731
    x, res, dy, ds = r(rows, n), r(rows, n), r(rows, n), r(rows, n)
    w = torch.rand(n, generator=g, device="cuda") + 0.5
    st = trunk.RMSNormStep(rows, n, act(dtype), keep8=True).bind(x, w, res, dy, ds)
    st.run()
    s = (x.float() + res.float()).to(act(dtype))
    assert torch.equal(st.s, s)
    s = s.double()
    scale = torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5)
    check(st.y, (s * scale * w).cpu().numpy(), EL, "y")
    held = trunk.Unpack8Step(rows, n).bind(st.s8).run().double()
    assert ((held - s).abs() <= 2.0 ** -4 * s.abs() + 2.0 ** -9).all()
    hat, gr = held * scale, dy.double() * w
    dx = scale * (gr - hat * (gr * hat).mean(1, keepdim=True)) + ds.double()
    check(st.dx, dx.cpu().numpy(), SUM, "dx")
    check(st.dw, (dy.double() * hat).sum(0).cpu().numpy(), SUM, "dw")
    check(st.y_again, (hat * w).cpu().numpy(), EL, "y_again")


@pytest.mark.parametrize("backward", [False, True])
def test_long_rows_go_side_by_side(backward):
    """64 rows of more than 8192 columns take about as long as one of them, each on an SM of its own: with
    eight rows to a CTA they would take eight times as long."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    def us(rows):
        r = lambda *a: torch.randn(*a, device="cuda")  # noqa: E731
        st = trunk.RMSNormStep(rows, 65536).bind(r(rows, 65536), r(65536), dy=r(rows, 65536))
        run, times = st.backward if backward else st.forward, []
        st.run()
        for _ in range(40):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            run()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[20]

    one, many = us(1), us(64)
    assert many < 4 * one, f"{one} and {many} ms"
