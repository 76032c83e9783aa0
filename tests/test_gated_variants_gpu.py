"""Variants of the gated block's operators that only some sizes reach, and values that are not numbers
in the recurrence's gradients and among 4-bit weights.

Tolerances are those of the operators' tests (1e-5 max|y| per element, 1e-4 max|y| for sums over steps, a
product's K terms each off by 2^-24 of the sum of magnitudes)."""
import numpy as np
import pytest

import oracle.gated as og
from gated_cases import gated_inputs, weights4_inputs
from test_gated_gpu import SUM, act, built, check, cuda, gated_check, gated_step  # noqa: F401 (built: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [6, 8])
def test_bias_gradient_of_many_sequences(D):
    """More partial sums than one CTA's merge takes, with and without four columns at a time."""
    K, B = 9, 2100
    ends = np.random.default_rng(D).integers(0, K + 1, size=B)
    i = gated_inputs(K, B, D, "f32", D, ends)
    st = gated_step(i, K, B, D, "f32", dh_last=True)
    gated_check(st, i, dh_last=True)
    first = st.dbias.clone()
    st.dbias.fill_(float("nan"))
    st.run()
    assert (st.dbias == first).all()


@pytest.mark.parametrize("M,N,K,group,dtype", [(1, 40, 12000, 128, "f32"), (2, 40, 12000, 64, "f32"),
                                               (1, 40, 40000, 128, "bf16"), (2, 40, 17000, 32, "bf16"),
                                               (1, 16000, 11000, 128, "f32"), (1, 40000, 11000, 128, "f32")])
def test_matvec4_in_several_chunks_of_one_row(M, N, K, group, dtype):
    """x beyond what shared memory holds, for tiles of rows that eight, four and two warps go along."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = weights4_inputs(M, N, K, group, dtype, N + K)
    codes, scales = torch.from_numpy(i["codes"]).cuda(), cuda(i["scales"], "bf16")
    st = trunk.MatvecStep(M, trunk.Weights4(codes, scales, K, group), act(dtype)).bind(cuda(i["x"], dtype))
    st.run()
    c = torch.stack([codes & 15, codes >> 4], -1).view(N, -1)[:, :K].double() - 8
    W = c * scales.double().repeat_interleave(group, 1)[:, :K]
    x = st.inputs["x"].double()
    want = x @ W.T
    bound = (K + 8) * 2.0 ** -24 * (x.abs() @ W.abs().T) * (1 + 2.0 ** -7)
    if dtype == "bf16":
        bound += 2.0 ** -8 * want.abs()
    assert ((st.y.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("K,D", [(45, 64), (45, 33), (45, 50), (900, 64), (900, 33)])
@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gradients_behind_a_length_are_0_whatever_comes_back(bad, keep8, K, D):
    """An infinite gradient of the last state reaches a sequence's steps, and none behind them."""
    i = gated_inputs(K, 3, D, "f32", K + D, [K - 2, 13, 0])
    i["dh_last"][1, D // 2] = bad
    st = gated_step(i, K, 3, D, "f32", keep8=keep8, dh_last=True)
    for b, e in enumerate(i["ends"]):
        for v in (st.y, st.dx, st.df, st.dz):
            assert not v[e:, b].any()
    i["dh_last"][1, D // 2] = 0
    fine = gated_step(i, K, 3, D, "f32", keep8=keep8, dh_last=True)
    import torch

    for name in ("dx", "df", "dz"):
        a, b = getattr(st, name).clone(), getattr(fine, name).clone()
        if name != "dz":
            assert not torch.isfinite(a[12, 1, D // 2])
            a[:, 1, D // 2] = b[:, 1, D // 2] = 0
        assert torch.equal(a, b)


def test_groups_with_an_infinity_are_not_numbers():
    """As a block in 8 bits: a group of weights with an infinity or a NaN is NaN throughout, and others are
    as they were."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    W = torch.randn(5, 130, device="cuda")
    clean = trunk.Weights4.quantized(W, 64)
    W[1, 70], W[2, 3], W[3, 129] = float("inf"), -float("inf"), float("nan")
    codes, scales = trunk.Weights4.quantized(W, 64)
    bad = torch.zeros(5, 3, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 0] = bad[3, 2] = True
    assert torch.equal(torch.isnan(scales), bad)
    assert torch.equal(scales[~bad], clean[1][~bad])
    rows = [0, 4]
    assert torch.equal(codes[rows], clean[0][rows])
    x = torch.ones(1, 130, device="cuda")
    st = trunk.MatvecStep(1, trunk.Weights4(codes, scales, 130, 64)).bind(x)
    st.run()
    assert torch.equal(torch.isnan(st.y[0]), torch.tensor([0, 1, 1, 1, 0], device="cuda").bool())


def test_nothing_bound_is_refused():
    """Tokens and conversions as the other steps; a bind that is refused leaves the call before it."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib, trunk

    z = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
    held = trunk.Pack8Step(4, 8).bind(z(4, 8)).run()
    for step, good, bad in (
            (trunk.Pack8Step(4, 8), (z(4, 8),), (z(4, 9),)),
            (trunk.Unpack8Step(4, 8), (held,), (_lib.Held8((4, 9)),)),
            (trunk.GatedToken(4, 8), (z(4, 8), z(4, 8), z(4, 8)), (z(4, 8), z(4, 9), z(4, 8))),
            (trunk.ConvToken(4, 8, 3), (z(4, 8), z(8, 3), z(4, 2, 8)), (z(4, 8), z(8, 3), z(4, 2, 9))),
            (trunk.ScanToken(4, 8, 4), (z(4, 8), z(4, 8), z(8, 4), z(4, 1, 4), z(4, 1, 4), z(4, 8, 4)),
             (z(4, 8), z(4, 9), z(8, 4), z(4, 1, 4), z(4, 1, 4), z(4, 8, 4)))):
        with pytest.raises(ValueError, match="bound"):
            step.run()
        step.bind(*good).run()
        call = step._call
        with pytest.raises(ValueError):
            step.bind(*bad)
        assert step._call is call
