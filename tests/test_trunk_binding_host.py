"""Steps of the trunk operators that nothing is bound to, on the host: they say so instead of leaving
their outputs as they were."""
import pytest
import torch

from recurrent_cfc_cell_gb300 import build, trunk


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def steps():
    return [trunk.LayerNormStep(4, 8, device="cpu"), trunk.DropoutNormStep(4, 8, 0.5, device="cpu"),
            trunk.ConvStep(5, 2, 8, 4, device="cpu"), trunk.ScanStep(5, 2, 8, 4, device="cpu"),
            trunk.ScanStep(5, 2, 8, 4, device="cpu", train=True)]


@pytest.mark.parametrize("k", range(5))
def test_unbound_steps_do_not_run(k):
    st = steps()[k]
    for call in (st.forward, st.backward, st.run):
        with pytest.raises(ValueError, match="bound"):
            call()


def bad_bind(st):
    x = torch.zeros(4, 8)  # not on a GPU: refused
    if isinstance(st, trunk.LayerNormStep):
        return st.bind(x, x[0], x[0], x)
    if isinstance(st, trunk.DropoutNormStep):
        return st.bind(x, None, torch.zeros(2, dtype=torch.int64), x[0], x[0], x)
    x = torch.zeros(5, 2, 8)
    if isinstance(st, trunk.ConvStep):
        return st.bind(x, torch.zeros(8, 4), dy=x)
    bc = torch.zeros(5, 2, 1, 4)
    return st.bind(x, x, torch.zeros(8, 4), bc, bc)


@pytest.mark.parametrize("k", range(5))
def test_a_refused_bind_leaves_nothing_bound(k):
    """Not the calls on the tensors that were bound before."""
    st, ran = steps()[k], []
    st._forward, st._backward = (ran.append,), (ran.append,)  # as if bound
    with pytest.raises(ValueError):
        bad_bind(st)
    for call in (st.forward, st.backward, st.run):
        with pytest.raises(ValueError, match="bound"):
            call()
    assert not ran


def test_a_refused_bind_of_a_token_keeps_the_state_of_its_call():
    x, state = torch.zeros(2, 8), torch.zeros(2, 3, 8)
    tok = trunk.ConvToken(2, 8, 4, device="cpu")
    tok.state, tok._call = "old", "old"
    with pytest.raises(ValueError):
        tok.bind(x, torch.zeros(8, 4), state)
    assert tok.state == tok._call == "old"
    tok = trunk.ScanToken(2, 8, 4, device="cpu")
    tok.state, tok._call = "old", "old"
    bc = torch.zeros(2, 1, 4)
    with pytest.raises(ValueError):
        tok.bind(x, x, torch.zeros(8, 4), bc, bc, torch.zeros(2, 8, 4))
    assert tok.state == tok._call == "old"
