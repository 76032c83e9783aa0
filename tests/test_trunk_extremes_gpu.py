"""Inputs at the edge of what fp32 holds."""
import pytest
import torch

import trunk_plain64 as p64
from test_trunk_gpu import EL, SUM
from trunk_draws import Draw, check, doubles, scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from recurrent_cfc_cell_gb300 import build

    build.build()


@pytest.mark.parametrize("K,N", [(20, 16), (300, 16), (9, 5)])
def test_rates_that_forget_at_once(K, N):
    """Decay rates so large that A log2 e leaves fp32's range, in sequences that end inside a chunk:
    such a state is what its last step put in."""
    from recurrent_cfc_cell_gb300 import trunk

    B, D, G = 4, 40, 1
    i = scan_inputs(K, B, D, N, G, "f32", K)
    i["A"][::3, 1] = -3e38
    i["A"][5] = -2.5e38
    ends = Draw(1).lengths(B, K, K, 5, 0, K - 1)
    want = p64.scan(doubles(i), ends.long())
    assert all(torch.isfinite(v).all() for v in want.values())
    i["D"] = i.pop("skip")
    st = trunk.ScanStep(K, B, D, N, G, train=True).bind(**i, lengths=ends)
    st.run()
    out = st.outputs()
    for k, v in want.items():
        check(out[k], v, EL if k in ("y", "h") else SUM, k)
    # No state at all is left of before where the rate is infinite.
    i["A"][5] = float("-inf")
    st.forward()
    check(st.h, want["h"], EL, "h")
    check(st.y, want["y"], EL, "y")
    # Token by token.
    tok = trunk.ScanToken(B, D, N, G)
    state = i["h0"].clone()
    for t in range(4):
        tok.bind(*(i[k][t] if k != "A" else i[k] for k in ("x", "dt", "A", "Bm", "Cm")), state,
                 i["D"], i["dt_bias"], i["z"][t]).run()
    i["skip"] = i.pop("D")
    i["A"][5] = -3e38
    first = {k: v[:4] if k in ("x", "dt", "z", "dy", "Bm", "Cm") else v for k, v in doubles(i).items()}
    check(state, p64.scan(first, torch.full((B,), 4, device="cuda"), backward=False)["h"], EL, "h")


@pytest.mark.parametrize("n", [1, 8, 37, 256])
def test_one_row_of_any_stride(n):
    """A single row's stride means nothing, whatever torch says it is: a column turned on its side
    is contiguous, and as good an output as any."""
    from recurrent_cfc_cell_gb300 import _lib
    from test_trunk_gpu import rng_tensor

    d = Draw(n)
    x, w, b = d.normal(1, n), d.f32(n), d.f32(n)
    rng, stats = rng_tensor(1, 2), torch.empty(1, 2, device="cuda")

    def row():
        t = torch.full((n, 1), float("nan"), device="cuda").T
        assert t.shape == (1, n) and t.is_contiguous()
        return t

    y, want, g, dx = row(), torch.empty_like(x), row(), row()
    _lib.cfc_layernorm_forward(x, w, b, want, stats)
    _lib.cfc_layernorm_forward(x, w, b, y, stats)
    assert torch.equal(y, want)
    _lib.cfc_dropout_forward(x, None, rng, 0.5, want)
    _lib.cfc_dropout_forward(x, None, rng, 0.5, y)
    assert torch.equal(y, want)
    g.copy_(x)
    dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    _lib.cfc_layernorm_backward(g, x, w, stats, dx, dw, db)
    _lib.cfc_layernorm_backward(x, x, w, stats, want, dw, db)
    assert torch.equal(dx, want) and torch.equal(db, x[0])


def test_a_refused_gradient_leaves_nothing_bound():
    """Not the forward pass alone, with the gradients of a step before."""
    from recurrent_cfc_cell_gb300 import trunk

    d = Draw(1)
    x, w, dy = d.normal(4, 8), d.f32(8), d.normal(4, 7)
    st = trunk.LayerNormStep(4, 8).bind(x, w, w, x)
    with pytest.raises(ValueError):
        st.bind(x, w, w, dy)
    with pytest.raises(ValueError, match="bound"):
        st.run()
    x, dt = d.normal(4, 2, 8), d.normal(4, 2, 8)
    bc, A = d.normal(4, 2, 1, 4), -torch.ones(8, 4, device="cuda")
    st = trunk.ScanStep(4, 2, 8, 4)
    with pytest.raises(ValueError):
        st.bind(x, dt, A, bc, bc, dy=x)  # made without train
    with pytest.raises(ValueError, match="bound"):
        st.run()
