"""What the selective scan's long recurrences keep of fp32's precision, in the 2-norm."""
import pytest
import torch

import trunk_plain64 as p64
from trunk_draws import Draw, doubles, scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from recurrent_cfc_cell_gb300 import build

    build.build()


@pytest.mark.parametrize("K,B,D,N,G", [(512, 8, 1024, 16, 2), (509, 13, 464, 32, 1)])
def test_scan_errors_do_not_add_up(K, B, D, N, G):
    """A step rounds a state's factor and its sum, each by 3e-8 rms and in random direction: over 500
    steps sqrt(2 x 500) 3e-8 = 9.5e-7 for a state that forgets nothing, the more so less for what is
    summed over channels, steps or sequences.  Errors in one direction would add up to 500 times
    their size instead: a factor 2e-8 too small to 1e-5.  1e-6, and half as much again for dh0, where
    nothing is averaged."""
    from recurrent_cfc_cell_gb300 import trunk

    i = scan_inputs(K, B, D, N, G, "f32", K)
    i["dh_last"].zero_()  # sums over steps alone
    want = p64.scan(doubles(i), torch.full((B,), K, device="cuda"))
    i["D"] = i.pop("skip")
    st = trunk.ScanStep(K, B, D, N, G, train=True).bind(**i)
    st.run()
    out = st.outputs()
    for k, v in want.items():
        err = ((out[k].double() - v).norm() / v.norm()).item()
        assert err <= (1.5e-6 if k == "dh0" else 1e-6), (k, err)


def test_steps_past_the_end_leave_the_state_alone_exactly():
    """The factor of such a step is exactly 1: a sequence ends with the state it has there."""
    from recurrent_cfc_cell_gb300 import trunk

    K, B, D, N = 40, 3, 40, 16
    i = scan_inputs(K, B, D, N, 1, "f32", 5)
    i = {k: i[k] for k in ("x", "dt", "A", "Bm", "Cm", "dt_bias", "h0")}
    ends = [0, 3, 17]
    st = trunk.ScanStep(K, B, D, N).bind(
        **i, lengths=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    st.run()
    assert torch.equal(st.h[0], i["h0"][0])
    for b in (1, 2):
        one = {k: v[:ends[b], b:b + 1] if k in ("x", "dt", "Bm", "Cm") else v for k, v in i.items()}
        one["h0"] = i["h0"][b:b + 1].clone()
        alone = trunk.ScanStep(ends[b], 1, D, N).bind(**one)
        alone.run()
        assert torch.equal(alone.h[0], st.h[b])
