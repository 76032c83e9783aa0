"""Serving on 4-bit weights at the ends of what a call allows: prompts of more rows than one call of the
products takes, shapes that only have as many elements as the right ones, a capture that fails.

Tolerances are those of the operators' tests (1e-5 max|y| for a product's fp32 sums, 1e-4 for a trunk
of several operators)."""
import numpy as np
import pytest

import oracle.gated as og
from gated_cases import rounded
from test_gated_gpu import EL, built, check, cuda  # noqa: F401 (built: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_products_of_more_rows_than_one_call_takes(dtype):
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    M, N, K = 2 ** 19 + 7, 5, 40
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    r = np.random.default_rng(4)
    W = cuda(r.normal(size=(N, K)))
    codes, scales = trunk.Weights4.quantized(W, 32)
    x = rounded(r.normal(size=(M, K)), dtype)
    st = trunk.MatvecStep(M, trunk.Weights4(codes, scales, K, 32), act).bind(cuda(x, dtype))
    st.run()
    check(st.y, x @ og.weights4(codes.cpu().numpy(), scales.double().cpu().numpy(), K, 32).T, EL, "y")
    first = st.y.clone()
    g = st.capture()
    st.y.zero_()
    g.replay()
    assert torch.equal(st.y, first)


def test_a_prompt_of_any_length():
    """More than 2^19 rows at a time, against the same prompt in parts."""
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedServe, make_gated_params

    P = make_gated_params(1, 8, 8, 32, seed=3)
    for K, B, cut in ((2 ** 19 + 9, 1, 2 ** 18), (131073, 5, 70000)):
        s = torch.randn(K, B, 8, device="cuda")
        one, two = GatedServe(B, P, group=32), GatedServe(B, P, group=32)
        whole = one.prompt(s)
        parts = torch.cat([two.prompt(s[:cut]), two.prompt(s[cut:])])
        assert (whole - parts).abs().max() <= 1e-4 * parts.abs().max()
        a, b = one.states[0], two.states[0]
        assert (a - b).abs().max() <= 1e-4 * b.abs().max()


def test_shapes_of_as_many_elements_are_refused():
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedServe, GatedTrunk, make_gated_params

    K, B, D, C = 6, 4, 32, 32
    P = make_gated_params(1, D, 64, C)
    z = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
    serve, trunk = GatedServe(B, P, group=32), GatedTrunk(K, B, P)
    for shape in ((K, D, B), (K, B * D), (K * B, D), (K, 2 * B, D // 2)):
        with pytest.raises(ValueError):
            serve.prompt(z(*shape))
        with pytest.raises(ValueError):
            trunk.forward(z(*shape), z(B, C), z(K, B))
    with pytest.raises(ValueError):
        trunk.forward(z(B, K, D), z(B, C), z(K, B))
    with pytest.raises(ValueError):
        serve.prompt(z(K, B, D).bfloat16())
    assert serve.prompt(z(K, B, D)).shape == (K, B, D)


def test_a_token_whose_capture_fails_leaves_the_states(monkeypatch):
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedServe, make_gated_params

    P = make_gated_params(2, 32, 64, 32)
    s = torch.randn(5, 3, 32, device="cuda")
    serve, other = GatedServe(3, P, group=32), GatedServe(3, P, group=32)
    serve.prompt(s[:4])
    other.prompt(s[:4])

    def fails(*a, **k):
        raise RuntimeError("no capture")

    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "graph", fails)
        with pytest.raises(RuntimeError):
            serve.token(s[4])
    assert all(torch.equal(a, b) for a, b in zip(serve.states, other.states))
    assert torch.equal(serve.token(s[4]), other.token(s[4]))
