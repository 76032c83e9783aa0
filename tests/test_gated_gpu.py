"""The gated block's operators on the GPU against their fp64 oracle.

Tolerances, per tensor, against y in fp64: fp32 results |x - y| <= tol max|y| with tol = 1e-5 for
what a pass computes per element and 1e-4 for sums over rows or steps (the trunk operators'
tolerances); bf16 results the same plus the rounding's bound, 2^-8 |y|.  What is packed in 8 bits is
compared bit by bit where the values are given, and against half a step of the form (2^-4 |y|, or
2^-10 of the scale) where they are computed."""
import numpy as np
import pytest

import oracle.gated as og
import oracle.trunk as ot
from gated_cases import gated_inputs, rms_inputs, weights4_inputs

pytestmark = pytest.mark.gpu

EL, SUM = 1e-5, 1e-4
DTYPES = ["f32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from recurrent_cfc_cell_gb300 import build

    build.build()


def cuda(v, dtype="f32"):
    import torch

    t = torch.float32 if dtype == "f32" else torch.bfloat16
    return torch.from_numpy(np.ascontiguousarray(v)).to(t).cuda()


def act(dtype):
    import torch

    return torch.float32 if dtype == "f32" else torch.bfloat16


def check(got, want, tol, name="", floor=0.0):
    """Every element within tol max|y| (bf16: plus 2^-8 |y|; plus `floor`)."""
    import torch

    x = got.double().cpu().numpy()
    assert x.shape == want.shape, name
    bound = tol * np.max(np.abs(want)) + floor if want.size else 0.0
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(want)
    err = np.abs(x - want)
    assert np.all(err <= bound), f"{name}: worst error {np.nanmax(err):.3g}, " \
                                 f"max|y| {np.max(np.abs(want)):.3g}"


def wide(t, pad, fill=float("nan")):
    """The same values as a view whose rows lie `pad` elements further apart and start one late."""
    import torch

    big = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device=t.device)
    v = big[..., 1:1 + t.shape[-1]] if pad else big
    v.copy_(t)
    return v


# ---- values in 8 bits ----

def held_bits(held):
    return held.codes.cpu().numpy(), held.scales.cpu().numpy()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,pad", [(1, 1, 0), (3, 8, 0), (5, 31, 0), (4, 32, 0), (4, 40, 0),
                                        (7, 96, 3), (9, 100, 0), (3, 257, 5), (33, 64, 8)])
def test_pack8_is_the_oracles_bit_by_bit(rows, n, pad, dtype):
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    r = np.random.default_rng(rows * 1000 + n)
    v = r.normal(size=(rows, n)) * 2.0 ** r.integers(-20, 20, size=(rows, 1))
    v[0, 0] = 0.0
    v[-1, n // 2] *= 1e-4  # small against its block
    x = wide(cuda(v, dtype), pad)
    v = x.double().cpu().numpy()
    held = trunk.Pack8Step(rows, n, act(dtype)).bind(x).run()
    want = [og.pack8(row) for row in v]
    codes, scales = held_bits(held)
    assert np.array_equal(scales, np.stack([s for _, s in want]))
    assert np.array_equal(codes, np.stack([c for c, _ in want]))
    for back in DTYPES:
        y = trunk.Unpack8Step(rows, n, act(back)).bind(held).run()
        assert np.array_equal(y.double().cpu().numpy(), og.held8(v))
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("n", [64, 67])
def test_pack8_ties_and_extremes(n):
    """Halfway values, magnitudes on both sides of a scale's border, the largest and the smallest of
    fp32, signed zeros; a block with an infinity or a NaN is NaN and leaves its neighbours alone."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    ties = (og.E4M3[1:] + og.E4M3[:-1]) / 2
    v = np.zeros((8, n))
    v[0, :n] = ties[-n:]
    v[0, 0] = 448.0
    v[1, :n] = -ties[:n]
    v[1, 1] = 448.0
    v[2, 0], v[2, 32] = 449.0, np.float32(np.nextafter(np.float32(448), np.float32(1000)))
    v[3, 0], v[3, 1] = 3.4028234663852886e38, 1e30
    v[4, 0], v[4, 1] = 1e-45, -1.2e-38
    v[5, 0] = -0.0
    v[6, 40], v[6, 3] = np.inf, 5.0
    v[7, 1], v[7, 40] = np.nan, -2.0
    held = trunk.Pack8Step(8, n).bind(cuda(v)).run()
    want = [og.pack8(row) for row in v.astype(np.float32).astype(np.float64)]
    codes, scales = held_bits(held)
    assert np.array_equal(scales, np.stack([s for _, s in want]))
    finite = np.repeat(scales < 255, 32, axis=1)[:, :n]
    assert np.array_equal(codes[finite], np.stack([c for c, _ in want])[finite])
    y = trunk.Unpack8Step(8, n).bind(held).run()
    assert (torch.isnan(y).cpu().numpy() == ~finite).all()


def test_unpack8_of_every_code():
    """All codes at the smallest, an ordinary and the largest scale, and the scales that packing
    never writes: 0 (2^-127) and 255 (NaN)."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib, trunk

    codes = torch.arange(256, dtype=torch.uint8).repeat(5, 1).cuda()
    scales = torch.tensor([1, 119, 246, 0, 255], dtype=torch.uint8)[:, None].repeat(1, 8).cuda()
    held = _lib.Held8((5, 256), codes=codes, scales=scales)
    y = trunk.Unpack8Step(5, 256).bind(held).run().cpu().double().numpy()
    for r, k in enumerate((1, 119, 246, 0)):
        want = np.array([og.e4m3_value(c) for c in range(256)]) * 2.0 ** (k - 127)
        assert np.array_equal(y[r], want, equal_nan=True)
    assert np.isnan(y[4]).all()


# ---- root-mean-square norm ----

# Widths below and at each team's edge, one column, odd ones, and beyond what registers hold.
WIDTHS = [(1, 1), (3, 7), (5, 8), (70, 32), (33, 33), (130, 64), (17, 127), (40, 128), (300, 256),
          (9, 257), (20, 500), (11, 512), (11, 1000), (3, 1024), (7, 1500), (6, 2048), (5, 2501),
          (4, 4096), (3, 5000), (2, 8192), (3, 8193), (2, 20000), (70, 8200)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", WIDTHS)
def test_rmsnorm(rows, n, dtype):
    from recurrent_cfc_cell_gb300 import trunk

    i = rms_inputs(rows, n, dtype, rows * 31 + n)
    st = trunk.RMSNormStep(rows, n, act(dtype)).bind(
        cuda(i["x"], dtype), cuda(i["w"]), cuda(i["residual"], dtype), cuda(i["dy"], dtype),
        cuda(i["ds"], dtype))
    st.run()
    out = st.outputs()
    assert np.array_equal(out["s"].double().cpu().numpy(), i["s"])
    check(out["y"], og.rmsnorm(i["s"], i["w"], 1e-5), EL, "y")
    dx, dw, _ = og.rmsnorm_backward(i["dy"], i["s"], i["w"], 1e-5, ds=i["ds"])
    check(out["dx"], dx, SUM, "dx")
    check(out["dw"], dw, SUM, "dw")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (5, 8), (70, 32), (33, 33), (40, 72), (17, 127),
                                    (130, 256), (9, 260), (11, 1000), (5, 2501), (4, 4096),
                                    (2, 8192), (3, 8193)])
def test_rmsnorm_in_8_bits(rows, n, dtype):
    """y to 8 bits in the forward pass, the backward pass from the stream in 8 bits."""
    from recurrent_cfc_cell_gb300 import trunk

    i = rms_inputs(rows, n, dtype, rows * 37 + n)
    st = trunk.RMSNormStep(rows, n, act(dtype), out8=True, keep8=True).bind(
        cuda(i["x"], dtype), cuda(i["w"]), cuda(i["residual"], dtype), cuda(i["dy"], dtype),
        cuda(i["ds"], dtype))
    st.run()
    want = [og.pack8(row) for row in i["s"]]
    codes, scales = held_bits(st.s8)
    assert np.array_equal(scales, np.stack([s for _, s in want]))
    assert np.array_equal(codes, np.stack([c for c, _ in want]))
    y = og.rmsnorm(i["s"], i["w"], 1e-5)
    got = trunk.Unpack8Step(rows, n).bind(st.y8).run().double().cpu().numpy()
    top = np.stack([np.abs(y[:, c:c + 32]).max(axis=1) for c in range(0, n, 32)], axis=1)
    scale = np.repeat(2.0 ** np.ceil(np.log2(np.maximum(top, 1e-30) / 448 * (1 + 1e-5))), 32,
                      axis=1)[:, :n]
    assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * scale)
                  + EL * np.abs(y).max())
    dx, dw, again = og.rmsnorm_backward(i["dy"], i["s"], i["w"], 1e-5, og.held8(i["s"]), i["ds"])
    out = st.outputs()
    check(out["dx"], dx, SUM, "dx")
    check(out["dw"], dw, SUM, "dw")
    check(out["y_again"], again, EL, "y_again")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(20000, 96), (6000, 1024), (3000, 777), (700, 5000), (300, 9000)])
def test_rmsnorm_8_bits_beside_borders(rows, n, dtype):
    """Codes are the ones of the exact y, also beside the borders between two codes: fp32 alone would
    take the other one about once in a million values, and these are several million."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    g = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *a: torch.randn(*a, generator=g, device="cuda")  # noqa: E731
    x, res, w = r(rows, n).to(act(dtype)), r(rows, n).to(act(dtype)), r(n) * 0.2 + 1.0
    st = trunk.RMSNormStep(rows, n, act(dtype), out8=True).bind(x, w, res)
    st.run()
    s = st.s.double()
    eps = float(np.float32(1e-5))
    y = s * w.double() / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    got = trunk.Unpack8Step(rows, n).bind(st.y8).run().double()
    for c in range(0, n, 32):
        v = y[:, c:c + 32]
        top = v.abs().amax(1, keepdim=True)
        m, e = torch.frexp(top)  # 448 = 0.875 * 2^9
        k = torch.where(m > 0.875, e - 8, e - 9).double()
        u = v * torch.exp2(-k)
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(u.abs().clamp(min=1e-30))), min=-6.0) - 3.0)
        assert torch.equal(got[:, c:c + 32], torch.round(u / step) * step * torch.exp2(k)), c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [64, 300, 8200])
def test_rmsnorm_alone_strided_in_place(n, dtype):
    """No residual and no stream gradient, rows further apart than they are long, the results in
    their inputs' memory."""
    from recurrent_cfc_cell_gb300 import _lib

    i = rms_inputs(9, n, dtype, n)
    w = cuda(i["w"])
    for pad in (0, 3, 8):
        x, dy = wide(cuda(i["x"], dtype), pad), wide(cuda(i["dy"], dtype), pad)
        y, rstd = wide(cuda(i["x"], dtype), pad), cuda(np.zeros(9))
        _lib.cfc_rmsnorm_forward(y, w, None, None, y, None, None, rstd)
        check(y, og.rmsnorm(i["x"], i["w"], 1e-5), EL, "y")
        dw = cuda(np.zeros(n))
        import torch

        ws = torch.empty(max(_lib.rmsnorm_workspace_bytes(9, n), 16), dtype=torch.uint8,
                         device="cuda")
        _lib.cfc_rmsnorm_backward(dy, x, w, rstd, dy, dw, None, None, ws)
        dx, want, _ = og.rmsnorm_backward(i["dy"], i["x"], i["w"], 1e-5)
        check(dy, dx, SUM, "dx")
        check(dw, want, SUM, "dw")
        # The sum in the residual's place, and the rest of the residual's rows as it was.
        x, res = wide(cuda(i["x"], dtype), pad), wide(cuda(i["residual"], dtype), pad, 7.0)
        _lib.cfc_rmsnorm_forward(x, w, res, res, None, None, None, None)
        assert np.array_equal(res.double().cpu().numpy(), i["s"])
        if pad:
            assert (res._base[..., 0] == 7.0).all() and (res._base[..., 1 + n:] == 7.0).all()


@pytest.mark.parametrize("n", [256, 301, 9001])
def test_rmsnorm_broadcast_rows(n):
    """A residual and an upstream gradient that are the same row throughout (stride 0)."""
    from recurrent_cfc_cell_gb300 import trunk

    i = rms_inputs(21, n, "f32", n)
    res, dy = cuda(i["residual"][:1]).expand(21, n), cuda(i["dy"][:1]).expand(21, n)
    st = trunk.RMSNormStep(21, n).bind(cuda(i["x"]), cuda(i["w"]), res, dy)
    st.run()
    s = (i["x"] + i["residual"][:1]).astype(np.float32).astype(np.float64)
    dx, dw, _ = og.rmsnorm_backward(np.repeat(i["dy"][:1], 21, 0), s, i["w"], 1e-5)
    check(st.y, og.rmsnorm(s, i["w"], 1e-5), EL, "y")
    check(st.dx, dx, SUM, "dx")
    check(st.dw, dw, SUM, "dw")


def test_rmsnorm_many_rows_and_reproducible():
    """More rows than CTAs have teams, so that teams take several; the same bits every time."""
    from recurrent_cfc_cell_gb300 import trunk

    for rows, n in ((20011, 64), (3001, 300), (2003, 1024), (1300, 2501)):
        i = rms_inputs(rows, n, "bf16", n)
        st = trunk.RMSNormStep(rows, n, act("bf16"), keep8=True).bind(
            cuda(i["x"], "bf16"), cuda(i["w"]), cuda(i["residual"], "bf16"), cuda(i["dy"], "bf16"),
            cuda(i["ds"], "bf16"))
        st.run()
        first = {k: v.clone() for k, v in st.outputs().items()}
        check(first["y"], og.rmsnorm(i["s"], i["w"], 1e-5), EL, "y")
        st.dw.fill_(float("nan"))
        st.run()
        assert all((first[k] == v).all() for k, v in st.outputs().items())
        import torch

        s8 = trunk.Unpack8Step(rows, n).bind(st.s8).run().double().cpu().numpy()
        dx, dw, _ = og.rmsnorm_backward(i["dy"], i["s"], i["w"], 1e-5, s8, i["ds"])
        check(first["dx"], dx, SUM, "dx")
        check(first["dw"], dw, SUM, "dw")
        assert torch.isfinite(first["dw"]).all()


# ---- gated linear recurrence ----

def gated_step(i, K, B, D, dtype, gate=True, ends=True, bias=True, h0=True, keep8=False, pad=0,
               dh_last=False):
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    lengths = torch.tensor(i["ends"], dtype=torch.int32).cuda() if ends else None
    def stop(v):  # what lies behind a sequence's end is not read
        v = v.copy()
        for b, e in enumerate(i["ends"]):
            v[e:, b] = np.nan
        return wide(cuda(v, dtype), pad)

    st = trunk.GatedStep(K, B, D, act(dtype), train=True, keep8=keep8).bind(
        stop(i["x"]), stop(i["f"]), cuda(i["bias"]) if bias else None,
        stop(i["z"]) if gate else None, cuda(i["h0"]) if h0 else None, lengths, stop(i["dy"]),
        cuda(i["dh_last"]) if dh_last else None)
    st.run()
    return st


def gated_check(st, i, gate=True, bias=True, h0=True, kept=False, dh_last=False):
    z = i["z"] if gate else None
    b = i["bias"] if bias else np.zeros_like(i["bias"])
    s = i["h0"] if h0 else np.zeros_like(i["h0"])
    y, h, _ = og.gated(i["x"], i["f"], b, z, s, i["ends"])
    out = st.outputs()
    check(out["y"], y, EL, "y")
    check(out["h"], h, EL, "h")
    want, again = og.gated_backward(i["dy"], i["x"], i["f"], b, z, s, i["ends"],
                                    i["dh_last"] if dh_last else None, kept)
    if kept:
        check(out["y_again"], again, EL, "y_again")
    for name in ("dx", "df") + (("dz",) if gate else ()):
        check(out[name], want[name], SUM, name)
    if bias:
        check(out["dbias"], want["dbias"], SUM, "dbias")
    check(out["dh0"], want["dh0"], SUM, "dh0")


GATED = [(1, 1, 1), (1, 3, 64), (7, 2, 33), (8, 1, 32), (9, 2, 65), (64, 3, 40), (127, 2, 6),
         (128, 1, 66), (129, 2, 31), (300, 2, 70), (1025, 1, 34)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,B,D", GATED)
def test_gated(K, B, D, dtype):
    i = gated_inputs(K, B, D, dtype, K * 7 + D)
    gated_check(gated_step(i, K, B, D, dtype, ends=False), i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,B,D", GATED)
def test_gated_kept_in_8_bits(K, B, D, dtype):
    ends = np.random.default_rng(K).integers(0, K + 1, size=B)
    i = gated_inputs(K, B, D, dtype, K * 7 + D, ends)
    st = gated_step(i, K, B, D, dtype, keep8=True, dh_last=True)
    gated_check(st, i, kept=True, dh_last=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate,bias,h0", [(False, True, True), (True, False, True),
                                          (True, True, False), (False, False, False)])
@pytest.mark.parametrize("keep8", [False, True])
def test_gated_without(gate, bias, h0, keep8, dtype):
    i = gated_inputs(37, 3, 50, dtype, 11, [37, 20, 3])
    st = gated_step(i, 37, 3, 50, dtype, gate, True, bias, h0, keep8)
    gated_check(st, i, gate, bias, h0, keep8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [1, 2, 8])
@pytest.mark.parametrize("D", [32, 45, 64])
def test_gated_ragged_strided(D, pad, dtype):
    """Lengths of zero, one, inside a run, at a run's and a round's border, and past K (clamped);
    views that start one element late; nothing behind a length is read, and results there are 0."""
    ends = [0, 1, 5, 8, 9, 128, 140, 200]
    i = gated_inputs(200, 8, D, dtype, D + pad, ends)
    st = gated_step(i, 200, 8, D, dtype, pad=pad, dh_last=True)
    gated_check(st, i, dh_last=True)
    for b, e in enumerate(ends):
        for v in (st.y, st.dx, st.df, st.dz):
            assert not v[e:, b].any()
    import torch

    st.inputs["lengths"].copy_(torch.tensor([-3, 1, 5, 8, 9, 128, 140, 999]))
    st.run()
    gated_check(st, i, dh_last=True)


# Few channels and many steps, which go in segments of the steps: channels in sixteens of bytes, in
# pairs and singly, segments that end inside a run's 8 steps and ones that there are not.
SEGMENTS = [(448, 1, 64), (1500, 2, 72), (1001, 3, 50), (2047, 1, 33), (5000, 1, 8), (777, 2, 130)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("K,B,D", SEGMENTS)
def test_gated_segments(K, B, D, keep8, dtype):
    ends = [K, K // 3, 0][:B]
    i = gated_inputs(K, B, D, dtype, K + D, ends)
    st = gated_step(i, K, B, D, dtype, keep8=keep8, dh_last=True, gate=D != 50)
    gated_check(st, i, kept=keep8, dh_last=True, gate=D != 50)
    first = {k: v.clone() for k, v in st.outputs().items()}
    g = st.capture()
    for v in st.outputs().values():
        v.fill_(float("nan"))
    g.replay()
    assert all((first[k] == v).all() for k, v in st.outputs().items())


@pytest.mark.parametrize("K", [40, 900])
def test_gated_state_in_its_own_place(K):
    """The last state over the initial one, in rounds and in segments."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    B, D = 2, 96
    i = gated_inputs(K, B, D, "f32", K, [K, 17])
    x, f, h = cuda(i["x"]), cuda(i["f"]), cuda(i["h0"])
    y, le = torch.empty_like(x), torch.tensor(i["ends"], dtype=torch.int32).cuda()
    ws = torch.empty(max(_lib.gated_workspace_bytes(K, B, D, False), 16), dtype=torch.uint8,
                     device="cuda")
    _lib.cfc_gated_forward(x, f, y, cuda(i["bias"]), h0=h, lengths=le, h_last=h, ws=ws)
    want, last, _ = og.gated(i["x"], i["f"], i["bias"], None, i["h0"], i["ends"])
    check(y, want, EL, "y")
    check(h, last, EL, "h")


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_batch_first_memory(dtype):
    """Sequences stored one after another, the outputs written the same way."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    K, B, D = 70, 5, 64
    i = gated_inputs(K, B, D, dtype, 3)
    x, f = (cuda(i[k].transpose(1, 0, 2), dtype).transpose(0, 1) for k in ("x", "f"))
    y = torch.full((B, K, D), 5.0, dtype=act(dtype), device="cuda")
    h = cuda(i["h0"])
    _lib.cfc_gated_forward(x, f, y.transpose(0, 1), cuda(i["bias"]), h0=h, h_last=h)
    want, last, _ = og.gated(i["x"], i["f"], i["bias"], None, i["h0"], i["ends"])
    check(y.transpose(0, 1), want, EL, "y")
    check(h, last, EL, "h")  # in its initial state's place


@pytest.mark.parametrize("K,D", [(20, 64), (700, 50)])
def test_gated_backward_forms_y_again(K, D):
    """y formed again from inputs that are kept as they are, without the gradients that are not
    wanted; z's gate strided apart from the others."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    B = 2
    i = gated_inputs(K, B, D, "f32", D)
    t = {k: cuda(i[k]) for k in ("x", "f", "dy", "bias", "h0")}
    z = wide(cuda(i["z"]), 5)
    y, again, states = torch.empty_like(t["x"]), torch.empty_like(t["x"]), torch.empty(
        -(-K // _lib.GATED_PERIOD), B, D, device="cuda")
    ws = torch.empty(max(_lib.gated_workspace_bytes(K, B, D, b) for b in (False, True)) + 16,
                     dtype=torch.uint8, device="cuda")
    _lib.cfc_gated_forward(t["x"], t["f"], y, t["bias"], z, t["h0"], states=states, ws=ws)
    dx, df, dz = (torch.empty_like(y) for _ in range(3))
    _lib.cfc_gated_backward(t["dy"], t["x"], t["f"], states, dx, df, t["bias"], z, dz=dz, y=again,
                            ws=ws)
    want, y64 = og.gated_backward(i["dy"], i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"])
    check(again, y64, EL, "y")
    check(y, y64, EL, "y")
    for name, got in (("dx", dx), ("df", df), ("dz", dz)):
        check(got, want[name], SUM, name)


def test_gated_continues():
    """A sequence in three calls, and tokens that go on from there."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    K, B, D = 96, 3, 40
    i = gated_inputs(K, B, D, "f32", 9)
    x, f, z, bias = cuda(i["x"]), cuda(i["f"]), cuda(i["z"]), cuda(i["bias"])
    y, h, _ = og.gated(i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"])
    state, parts = cuda(i["h0"]), []
    for lo, hi in ((0, 33), (33, 34), (34, 90)):
        st = trunk.GatedStep(hi - lo, B, D).bind(x[lo:hi], f[lo:hi], bias, z[lo:hi], state)
        st.run()
        parts.append(st.y)
        state = st.h
    token = trunk.GatedToken(B, D)
    for t in range(90, K):
        out, state = token.bind(x[t], f[t], state, bias, z[t]).run()
        parts.append(out.clone()[None])
    check(torch.cat(parts), y, EL, "y")
    check(state, h, EL, "h")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,pad", [(1, 1, 0), (3, 33, 0), (5, 64, 0), (4, 50, 2), (300, 128, 8)])
def test_gated_token(B, D, pad, dtype):
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = gated_inputs(1, B, D, dtype, B + D)
    y, h, _ = og.gated(i["x"], i["f"], i["bias"], i["z"], i["h0"], i["ends"])
    state = cuda(i["h0"])
    args = [wide(cuda(i[k][0], dtype), pad) for k in ("x", "f", "z")]
    st = trunk.GatedToken(B, D, act(dtype)).bind(args[0], args[1], state, cuda(i["bias"]), args[2],
                                                 torch.empty_like(state))
    got, new = st.run()
    check(got, y[0], EL, "y")
    check(new, h, EL, "h")
    assert np.array_equal(state.double().cpu().numpy(), i["h0"])  # not in its place
    got, same = trunk.GatedToken(B, D, act(dtype)).bind(args[0], args[1], state).run()
    y, h, _ = og.gated(i["x"], i["f"], 0 * i["bias"], None, i["h0"], i["ends"])
    check(got, y[0], EL, "y")
    check(same, h, EL, "h")
    assert same is state


def test_gated_extreme_gates():
    """Logits that shut or open the gate entirely, and infinite ones: states are held or replaced
    exactly; a NaN stays in its channel."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    K, B, D = 40, 1, 8
    x = torch.randn(K, B, D, device="cuda")
    f = torch.zeros(K, B, D, device="cuda")
    for d, v in enumerate((300.0, -300.0, float("inf"), -float("inf"))):
        f[..., d] = v
    x[3, 0, 6] = float("nan")
    h0 = torch.randn(B, D, device="cuda")
    st = trunk.GatedStep(K, B, D, train=True).bind(x, f, h0=h0, dy=torch.ones_like(x))
    st.run()
    assert torch.equal(st.y[..., 0], h0[:, 0].expand(K, B)) and torch.equal(st.y[..., 2], h0[:, 2].expand(K, B))
    assert torch.equal(st.y[..., 1], x[..., 1]) and torch.equal(st.y[..., 3], x[..., 3])
    assert torch.isfinite(st.y[..., [0, 1, 2, 3, 4, 5, 7]]).all() and torch.isnan(st.y[3:, :, 6]).all()
    assert torch.isfinite(st.y[:3]).all() and torch.isfinite(st.dx[..., :4]).all()
    assert torch.equal(st.dx[..., 1], torch.ones(K, B, device="cuda")) and not st.dx[..., 0].any()


def test_gated_reproducible_and_captured():
    """Two captured graphs and an eager run on another stream give the same bits; a graph reads its
    inputs when it runs."""
    import torch

    K, B, D = 150, 4, 96
    i = gated_inputs(K, B, D, "bf16", 4, [150, 9, 77, 128])
    st = gated_step(i, K, B, D, "bf16", keep8=True)
    first = {k: v.clone() for k, v in st.outputs().items()}
    g = st.capture()
    other = gated_step(i, K, B, D, "bf16", keep8=True)
    h = other.capture()
    for _ in range(2):
        for v in list(st.outputs().values()) + list(other.outputs().values()):
            v.fill_(float("nan"))
        h.replay()
        g.replay()
        torch.cuda.synchronize()
        for a in (st, other):
            assert all(torch.equal(first[k], v) for k, v in a.outputs().items())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    st.run(s)
    s.synchronize()
    assert all(torch.equal(first[k], v) for k, v in st.outputs().items())
    st.inputs["dy"].zero_()
    g.replay()
    assert not st.dx[:9].any() and not st.dbias.any()


# ---- 4-bit weights ----

W4 = [(1, 1, 1, 32), (1, 16, 128, 128), (2, 17, 129, 64), (3, 100, 31, 32), (8, 64, 256, 128),
      (9, 33, 300, 64), (16, 48, 1000, 32), (1, 500, 1025, 128), (33, 40, 96, 32), (5, 130, 2300, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,group", W4)
def test_matvec4(M, N, K, group, dtype):
    """fp32 sums of exact products: K terms, each off by 2^-24 of the sum of magnitudes at most."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = weights4_inputs(M, N, K, group, dtype, M * N + K)
    W = og.weights4(i["codes"], i["scales"], K, group)
    weights = trunk.Weights4(torch.from_numpy(i["codes"]).cuda(), cuda(i["scales"], "bf16"), K, group)
    bound = (K + 8) * 2.0 ** -24 * (np.abs(i["x"]) @ np.abs(W).T)
    want = i["x"] @ W.T
    for pad in (0, 1, 8):
        x = wide(cuda(i["x"], dtype), pad)
        st = trunk.MatvecStep(M, weights, act(dtype)).bind(x)
        st.run()
        got = st.y.double().cpu().numpy()
        rounding = 2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0.0
        assert np.all(np.abs(got - want) <= bound * (1 + 2.0 ** -7) + rounding)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (5, 33, 32), (40, 200, 64), (17, 256, 128)])
def test_weights4_quantized(N, K, group, dtype):
    """Scales are a seventh of the group's largest magnitude, to bf16; every weight is within half a
    step (and the scale's rounding, 7 steps of 2^-8)."""
    from recurrent_cfc_cell_gb300 import trunk

    r = np.random.default_rng(N * K)
    W = cuda(r.normal(size=(N, K)) * 2.0 ** r.integers(-5, 5, size=(N, 1)), dtype)
    W[0, : min(K, group)] = 0.0
    codes, scales = trunk.Weights4.quantized(wide(W, 3), group)
    v = W.double().cpu().numpy()
    s = scales.double().cpu().numpy()
    for g in range(s.shape[1]):
        top = np.abs(v[:, g * group:(g + 1) * group]).max(axis=1)
        want = ot.bf16((top.astype(np.float32) / np.float32(7)).astype(np.float64))
        assert np.array_equal(s[:, g], want)
    back = og.weights4(codes.cpu().numpy(), s, K, group)
    step = np.repeat(s, group, axis=1)[:, :K]
    assert np.all(np.abs(back - v) <= step * (0.5 + 7 * 2.0 ** -8))
    assert not back[0, : min(K, group)].any()
    if K % 2:
        assert np.all(codes.cpu().numpy()[:, -1] >> 4 == 8)


def test_matvec4_one_row_of_infinities():
    """A row of x with an infinity or a NaN does not reach the other rows."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = weights4_inputs(4, 64, 200, 64, "f32", 1)
    weights = trunk.Weights4(torch.from_numpy(i["codes"]).cuda(), cuda(i["scales"], "bf16"), 200, 64)
    x = cuda(i["x"])
    clean = trunk.MatvecStep(4, weights).bind(x)
    clean.run()
    bad = x.clone()
    bad[1, 7], bad[2, 150] = float("nan"), float("inf")
    st = trunk.MatvecStep(4, weights).bind(bad)
    st.run()
    assert torch.equal(st.y[0], clean.y[0]) and torch.equal(st.y[3], clean.y[3])
    assert torch.isnan(st.y[1]).all() and not torch.isfinite(st.y[2]).any()


def test_matvec4_of_a_file_matches_quantized_weights():
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    W = torch.randn(96, 333, device="cuda")
    x = torch.randn(2, 333, device="cuda")
    a = trunk.MatvecStep(2, trunk.Weights4.of(W, 64)).bind(x)
    a.run()
    codes, scales = trunk.Weights4.quantized(W, 64)
    b = trunk.MatvecStep(2, trunk.Weights4(codes, scales, 333, 64)).bind(x)
    b.run()
    assert torch.equal(a.y, b.y)
    assert (a.y - x @ W.T).norm() < 0.2 * (x @ W.T).norm()  # 7 steps of a normal row's 3 sigma
