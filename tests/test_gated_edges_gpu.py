"""The gated block's operators at the ends of what a call allows: tensors of more than 2^31 elements,
inputs that repeat in memory, streams other than the default one, values that are not numbers.

Tolerances are those of the operators' other tests (1e-5 max|y| for what is computed per element, 1e-4
for sums over steps, 2^-8 |y| for a rounding to bf16)."""
import numpy as np
import pytest

import oracle.gated as og
from gated_cases import gated_inputs, rounded
from test_gated_gpu import EL, SUM, built, check, cuda  # noqa: F401 (built: the fixture)

pytestmark = pytest.mark.gpu


def tail(rows, n, last, seed):
    """bf16 [rows, n]: zeros, and random numbers in the last rows, which are also given in float64."""
    import torch

    v = rounded(np.random.default_rng(seed).normal(size=(last, n)), "bf16")
    t = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    t[-last:] = cuda(v, "bf16")
    return t, v


@pytest.mark.parametrize("n", [512, 513])
def test_rmsnorm_beyond_31_bits(n):
    """Rows whose first element lies beyond 2^31; dw is the last rows' alone, since dy is 0 elsewhere."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    rows, last = 2 ** 31 // n + 40, 30
    x, x64 = tail(rows, n, last, n)
    dy, dy64 = tail(rows, n, last, n + 1)
    w = rounded(np.random.default_rng(2).normal(1.0, 0.2, size=n), "f32")
    st = trunk.RMSNormStep(rows, n, dtype=torch.bfloat16, keep8=True).bind(x, cuda(w), dy=dy)
    st.run()
    y64 = og.rmsnorm(x64, w, 1e-5)
    check(st.y[-last:], y64, EL, "y")
    s8 = og.held8(x64)
    up = trunk.Unpack8Step(rows, n, dtype=torch.bfloat16).bind(st.s8).run()
    assert np.array_equal(up[-last:].double().cpu().numpy(), s8)
    dx, dw, again = og.rmsnorm_backward(dy64, x64, w, 1e-5, s8)
    check(st.dx[-last:], dx, SUM, "dx")
    check(st.dw, dw, SUM, "dw")
    check(st.y_again[-last:], again, EL, "y_again")
    assert not st.y[:-last].any() and not st.dx[:-last].any()
    packed = trunk.Pack8Step(rows, n, dtype=torch.bfloat16).bind(x).run()
    assert torch.equal(packed.codes, st.s8.codes) and torch.equal(packed.scales, st.s8.scales)


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("K,B,D", [(1030, 64, 32600), (2 ** 24, 1, 130)])
def test_gated_beyond_31_bits(K, B, D, keep8):
    """The last channels of the last sequence, and the last steps of those, by rounds and by segments.
    Where there is nothing before, x is 0 and the state stays 0."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    assert K * B * D > 2 ** 31
    bf, T, C = torch.bfloat16, 160, 32  # T: not a multiple of a segment
    i = gated_inputs(T, 1, C, "bf16", D)
    i["h0"][:] = 0

    def place(k):
        t = torch.zeros(K, B, D, dtype=bf, device="cuda")
        t[-T:, -1, -C:] = cuda(i[k][:, 0], "bf16")
        return t

    bias = torch.zeros(D, device="cuda")
    bias[-C:] = cuda(i["bias"])
    st = trunk.GatedStep(K, B, D, bf, train=True, keep8=keep8).bind(
        place("x"), place("f"), bias, place("z"), dy=place("dy"))
    st.run()
    # 8 bits have a scale for 32 channels from the tensor's first one on, and h is formed again from
    # every eighth step's state on: the oracle has the zeros before the last channels and steps too,
    # from the borders of a block and of a period on.
    channels, steps = (D - C) % 32, (K - T) % 8
    for k, v in i.items():
        if k != "ends":
            i[k] = np.pad(v, ([(steps, 0)] if v.ndim == 3 else []) + [(0, 0)] * (v.ndim > 1)
                          + [(channels, 0)])
    C, T = C + channels, T + steps
    i["ends"][:] = T
    y, h, _ = og.gated(i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"])
    check(st.y[-T:, -1:, -C:], y, EL, "y")
    check(st.h[-1:, -C:], h, EL, "h")
    want, again = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"],
                                    None, keep8)
    for name in ("dx", "dz"):
        check(getattr(st, name)[-T:, -1:, -C:], want[name], SUM, name)
    check(st.df[-T:, -1:, -C:], want["df"], SUM, "df")
    if keep8:
        check(st.y_again[-T:, -1:, -C:], again, EL, "y_again")
    assert not st.y[:-T].any() and not st.y[:, :-1].any()


def test_weights4_beyond_32_bits():
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    N, K, group = 2 ** 20 + 5, 8200, 128
    r = np.random.default_rng(1)
    row = rounded(r.normal(size=K), "bf16")
    codes, scales = trunk.Weights4.quantized(cuda(row, "bf16")[None].expand(N, K), group)
    assert codes.numel() > 2 ** 32
    assert torch.equal(codes[-1], codes[0]) and torch.equal(scales[-1], scales[0])
    tail8 = torch.from_numpy(r.integers(0, 256, size=(8, codes.shape[1]), dtype=np.uint8)).cuda()
    codes[-8:] = tail8
    weights = trunk.Weights4(codes, scales, K, group)
    x = rounded(r.normal(size=(2, K)), "bf16")
    st = trunk.MatvecStep(2, weights, dtype=torch.bfloat16).bind(cuda(x, "bf16"))
    st.run()
    W = og.weights4(codes[-20:].cpu().numpy(), scales[-20:].double().cpu().numpy(), K, group)
    check(st.y[:, -20:], x @ W.T, SUM, "y")


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("K,B,D", [(40, 3, 64), (41, 3, 50), (600, 2, 40), (40, 3, 33)])
def test_gated_inputs_that_repeat(K, B, D, keep8):
    """One step for all steps, one sequence for all sequences, one row for both."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = gated_inputs(K, B, D, "f32", K + D)
    i["x"][:] = i["x"][:1]
    i["f"][:] = i["f"][:, :1]
    i["z"][:] = i["z"][:1, :1]
    i["dy"][:] = i["dy"][:1, :1]
    full = [cuda(i[k]) for k in ("x", "f", "z", "dy")]
    less = [full[0][:1].clone(), full[1][:, :1].clone(), full[2][:1, :1].clone(),
            full[3][:1, :1].clone()]
    outs = []
    for x, f, z, dy in (full, [t.expand(K, B, D) for t in less]):
        st = trunk.GatedStep(K, B, D, train=True, keep8=keep8).bind(
            x, f, cuda(i["bias"]), z, cuda(i["h0"]), dy=dy)
        st.run()
        outs.append(st.outputs())
    assert all(torch.equal(outs[0][k], outs[1][k]) for k in outs[0])
    y, _, _ = og.gated(i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"])
    check(outs[1]["y"], y, EL, "y")


def test_another_stream():
    """What a stream has written before a call is what the call reads, and two graphs of one step's
    passes, replayed in turn, share its workspace."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    K, B, D = 800, 1, 96
    i = gated_inputs(K, B, D, "f32", 1)
    x, f, dy = (torch.zeros(K, B, D, device="cuda") for _ in range(3))
    st = trunk.GatedStep(K, B, D, train=True).bind(x, f, cuda(i["bias"]), dy=dy)
    src = {k: cuda(i[k]) for k in ("x", "f", "dy")}
    want = trunk.GatedStep(K, B, D, train=True).bind(src["x"], src["f"], cuda(i["bias"]),
                                                     dy=src["dy"])
    want.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000)
        for t, k in ((x, "x"), (f, "f"), (dy, "dy")):
            t.copy_(src[k])
        st.run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(st.outputs().values(), want.outputs().values()))
    graphs = []
    for part in (st.forward, st.backward):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            part()
        graphs.append(g)
    for _ in range(2):
        for v in st.outputs().values():
            v.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(st.outputs().values(), want.outputs().values()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(1, 19500, 300, 128), (1, 40000, 130, 32), (3, 2450, 1100, 64),
                                         (8, 5000, 2050, 128), (12, 9000, 1000, 64),
                                         (30, 2500, 2100, 128), (33, 5000, 700, 32), (70, 20, 260, 64)])
def test_matvec4_spreads(M, N, K, group, dtype):
    """Every way in which a product's warps are spread over rows and columns of W, with odd ends."""
    from recurrent_cfc_cell_gb300 import trunk
    from gated_cases import weights4_inputs
    from test_gated_gpu import act
    import torch

    i = weights4_inputs(M, N, K, group, dtype, N + K)
    weights = trunk.Weights4(torch.from_numpy(i["codes"]).cuda(), cuda(i["scales"], "bf16"), K, group)
    st = trunk.MatvecStep(M, weights, dtype=act(dtype)).bind(cuda(i["x"], dtype))
    st.run()
    check(st.y, i["x"] @ og.weights4(i["codes"], i["scales"], K, group).T, EL, "y")


def test_matvec4_of_every_nan():
    """A NaN whose upper 16 bits are an infinity's."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    weights = trunk.Weights4.of(torch.randn(40, 64, device="cuda"), 32)
    x = torch.randn(2, 64, device="cuda")
    x.view(torch.int32)[1, 5] = 0x7F800001
    st = trunk.MatvecStep(2, weights).bind(x)
    st.run()
    y = st.y
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1]).all()


def test_serving_refuses_another_batch():
    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedServe, make_gated_params

    serve = GatedServe(3, make_gated_params(1, 32, 64, 128), group=32)
    for shape in ((1, 32), (32,), (4, 32)):
        with pytest.raises(ValueError):
            serve.token(torch.zeros(shape, device="cuda"))
    with pytest.raises(ValueError):
        serve.token(torch.zeros(3, 32, device="cuda", dtype=torch.bfloat16))
    assert serve.token(torch.zeros(3, 32, device="cuda")).shape == (3, 32)
