"""The trunk block (the trunk operators and the cell together): its gradients against float64
autograd of the same block, and serving token by token against the prompt."""
import numpy as np
import pytest

import oracle.trunk as ot

pytestmark = pytest.mark.gpu

# Six operators and four products in a row, each within 1e-5 of its exact result in fp32 (the
# single operators' tests), with sums over K * B rows behind the parameters' gradients: 1e-4 each
# way, as the single operators' gradients, for the outputs' tolerance twice that of one operator.
OUT_TOL, GRAD_TOL = 2e-5, 2e-4


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch

    from recurrent_cfc_cell_gb300 import build

    build.build()
    torch.backends.cuda.matmul.allow_tf32 = False


def reference(P, s, h0, ts, keep, scale, G):
    """The block in float64 torch operations, for autograd."""
    import torch

    K, B, D = s.shape
    E, N = P["A"].shape
    norm = lambda v, w, b: torch.nn.functional.layer_norm(v, (D,), w, b, 1e-5)  # noqa: E731
    xz = norm(s, P["w1"], P["b1"]) @ P["W_in"].T
    W = P["conv_w"].shape[1]
    line = torch.cat([torch.zeros(W - 1, B, E, dtype=s.dtype), xz[..., :E]])
    u = torch.nn.functional.silu(sum(line[j:j + K] * P["conv_w"][:, j] for j in range(W)) + P["conv_b"])
    p = u @ P["W_p"].T
    dt = torch.nn.functional.softplus(p[..., :E] + P["dt_bias"])
    bc = p[..., E:].unflatten(-1, (2, G, N)).repeat_interleave(E // G, 3)
    h, ys = torch.zeros(B, E, N, dtype=s.dtype), []
    for t in range(K):
        h = torch.exp(dt[t][..., None] * P["A"]) * h + (dt[t] * u[t])[..., None] * bc[t, :, 0]
        ys.append((h * bc[t, :, 1]).sum(-1) + P["D"] * u[t])
    y = torch.stack(ys) * torch.nn.functional.silu(xz[..., E:])
    n2 = norm(s + keep * (y @ P["W_out"].T) * scale, P["w2"], P["b2"])
    h, H = h0, []
    for t in range(K):
        pre = torch.einsum("gcn,bn->gbc", P["cell_W"], torch.cat([n2[t], h], -1)) + P["cell_b"][:, None]
        gate = torch.sigmoid(pre[2] * ts[t][:, None] + pre[3])
        h = torch.tanh(pre[0]) * (1 - gate) + gate * torch.tanh(pre[1])
        H.append(h)
    return torch.stack(H)


def test_block_gradients():
    import torch

    from recurrent_cfc_cell_gb300.block import TrunkBlock, make_params

    K, B, D, E, N, C, G = 12, 3, 24, 32, 8, 32, 2
    P = make_params(D, E, N, C, G=G, seed=1)
    g = torch.Generator().manual_seed(2)
    s, h0, dH = (torch.randn(*d, generator=g) for d in ((K, B, D), (B, C), (K, B, C)))
    ts = torch.rand(K, B, generator=g) + 0.5
    rng = torch.tensor([11, 12], dtype=torch.int64, device="cuda")
    block = TrunkBlock(K, B, P, p_drop=0.25, G=G)
    H = block.forward(s.cuda(), h0.cuda(), ts.cuda(), rng)
    grads = block.backward(dH.cuda())
    keep, scale = ot.dropout_mask(K * B, D, 0.25, 11, 12)
    ref = {k: v.double().cpu().requires_grad_() for k, v in P.items()}
    s64, h64 = s.double().requires_grad_(), h0.double().requires_grad_()
    want = reference(ref, s64, h64, ts.double(), torch.from_numpy(keep.reshape(K, B, D)), scale, G)
    (want * dH.double()).sum().backward()
    ref = {**{k: v.grad for k, v in ref.items()}, "ds": s64.grad, "dh0": h64.grad}
    assert (H.double().cpu() - want).abs().max() <= OUT_TOL * want.abs().max()
    for k, v in ref.items():
        err = (grads[k].double().cpu() - v).abs().max() / v.abs().max()
        assert err <= GRAD_TOL, (k, float(err))


def test_serving_tokens_follow_the_prompt():
    """A prompt in one piece, against its first part as a prompt and the rest token by token."""
    import torch

    from recurrent_cfc_cell_gb300.block import TrunkServe, make_params

    K, B, D, E, N = 10, 4, 40, 64, 16
    P = make_params(D, E, N, 16, seed=3)
    s = torch.randn(K, B, D, generator=torch.Generator().manual_seed(4)).cuda()
    whole = TrunkServe(B, P).prompt(s)
    serve = TrunkServe(B, P)
    parts = [serve.prompt(s[:4])]
    parts += [serve.token(s[t]).clone()[None] for t in range(4, K)]
    got = torch.cat(parts)
    assert (got - whole).abs().max() <= OUT_TOL * whole.abs().max()
    # A second prompt continues from the carried states.
    serve = TrunkServe(B, P)
    got = torch.cat([serve.prompt(s[:7]), serve.prompt(s[7:])])
    assert (got - whole).abs().max() <= OUT_TOL * whole.abs().max()
