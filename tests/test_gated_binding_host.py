"""Outputs that a step is given from outside, on the host."""
import pytest
import torch

from recurrent_cfc_cell_gb300 import build, trunk


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_outputs_from_outside():
    y, dx = torch.zeros(4, 8), torch.zeros(4, 8)
    st = trunk.RMSNormStep(4, 8, device="cpu", into=dict(y=y, dx=dx))
    st._alloc_grads()
    assert st.y is y and st.dx is dx and st.dw.shape == (8,)
    own = trunk.RMSNormStep(4, 8, device="cpu")
    assert own.y is not y and own.y.shape == (4, 8)
    t = {k: torch.zeros(5, 2, 8) for k in ("y", "dx", "df", "dz")}
    st = trunk.GatedStep(5, 2, 8, train=True, device="cpu", into=t)
    assert st.y is t["y"] and st.dx is t["dx"] and st.df is t["df"]


def test_other_names_are_refused():
    for make in (lambda into: trunk.RMSNormStep(4, 8, device="cpu", into=into),
                 lambda into: trunk.GatedStep(5, 2, 8, train=True, device="cpu", into=into)):
        for name in ("dX", "states", "rstd"):
            with pytest.raises(ValueError, match="into"):
                make({name: torch.zeros(4, 8)})
