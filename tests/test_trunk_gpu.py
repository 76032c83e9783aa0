"""The trunk operators on the GPU against their fp64 oracle.

Tolerances, per tensor, against y in fp64: fp32 results |x - y| <= tol max|y| with tol = 1e-5 for
what a pass computes per element and 1e-4 for sums over rows or steps (the four-gate cell's
tolerances); bf16 results the same plus 2^-8 |y|, twice the rounding's own bound."""
import numpy as np
import pytest

import oracle.trunk as ot
from trunk_cases import conv_inputs, norm_inputs, scan_inputs

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


def check(got, want, tol, name=""):
    """Every element within tol max|y| (bf16: plus 2^-8 |y|)."""
    import torch

    x = got.double().cpu().numpy()
    assert x.shape == want.shape, name
    bound = tol * np.max(np.abs(want)) if want.size else 0.0
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(want)
    err = np.abs(x - want)
    assert np.all(err <= bound), f"{name}: {np.nanmax(err - bound):.3g} over the bound, " \
                                 f"worst error {np.nanmax(err):.3g}, max|y| {np.max(np.abs(want)):.3g}"


def wide(t, pad, fill=float("nan")):
    """The same values as a view whose rows lie `pad` elements further apart, and start one
    element late: the innermost dimension contiguous, nothing aligned."""
    import torch

    big = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device=t.device)
    v = big[..., 1:1 + t.shape[-1]] if pad else big
    v.copy_(t)
    return v


# ---- layer norm and dropout ----

# Widths below and at each team's edge, one column, odd ones, and beyond what registers hold.
WIDTHS = [(1, 1), (3, 7), (5, 8), (70, 32), (33, 33), (130, 64), (17, 127), (40, 128), (300, 256),
          (9, 257), (20, 500), (11, 1000), (3, 1024), (7, 1500), (6, 2048), (5, 2501), (4, 4096),
          (3, 5000), (2, 8192), (3, 8193), (2, 20000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", WIDTHS)
def test_layernorm(rows, n, dtype):
    from recurrent_cfc_cell_gb300 import trunk

    i = norm_inputs(rows, n, dtype, rows * 31 + n)
    st = trunk.LayerNormStep(rows, n, act(dtype)).bind(
        cuda(i["x"], dtype), cuda(i["w"]), cuda(i["b"]), cuda(i["dy"], dtype))
    st.run()
    out = st.outputs()
    check(out["y"], ot.layernorm(i["x"], i["w"], i["b"], 1e-5), EL, "y")
    dx, dw, db = ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)
    if n > 1:  # one column: everything but db is zero
        check(out["dx"], dx, SUM, "dx")
        check(out["dw"], dw, SUM, "dw")
    else:
        assert not out["dx"].any() and not out["dw"].any()
    check(out["db"], db, SUM, "db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(12, 24), (40, 96), (9, 250), (6, 1030)])
def test_layernorm_strided_rows(rows, n, dtype):
    """Rows further apart than they are long, starting off alignment, NaN between them; outputs
    into views too, and nothing written beside them."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    i = norm_inputs(rows, n, dtype, 5)
    x, dy = wide(cuda(i["x"], dtype), 5), wide(cuda(i["dy"], dtype), 3)
    y, dx = (wide(torch.zeros(rows, n, dtype=act(dtype), device="cuda"), 4, 77.0) for _ in range(2))
    w, b, stats = cuda(i["w"]), cuda(i["b"]), torch.empty(rows, 2, device="cuda")
    dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    need = _lib.layernorm_workspace_bytes(rows, n)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    _lib.cfc_layernorm_forward(x, w, b, y, stats)
    _lib.cfc_layernorm_backward(dy, x, w, stats, dx, dw, db, ws)
    check(y, ot.layernorm(i["x"], i["w"], i["b"], 1e-5), EL, "y")
    for got, want in zip((dx, dw, db), ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)):
        check(got, want, SUM)
    for v in (y, dx):
        beside = v.as_strided((rows - 1, 4), (n + 4, 1), v.storage_offset() + n)
        assert (beside == 77.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,offset", [(1, 3, 5), (2, 3, 5), (3, 1, 7), (9, 5, 3), (20, 13, 1),
                                           (5, 255, 6), (3, 2043, 2), (2, 4099, 7)])
def test_layernorm_packed_rows_from_anywhere(rows, n, offset, dtype):
    """Rows one after another from any element on, so that a group of eight spans several rows or
    starts before the first: NaN around the tensor, and the results of the same rows aligned."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    i = norm_inputs(rows, n, dtype, offset)

    def packed(v, fill):
        buf = torch.full((rows * n + 16,), fill, dtype=act(dtype), device="cuda")
        view = buf[offset:offset + rows * n].view(rows, n)
        view.copy_(v)
        return buf, view

    nan = float("nan")
    (_, x), (_, dy) = packed(cuda(i["x"], dtype), nan), packed(cuda(i["dy"], dtype), nan)
    (yb, y), (db_, dx) = (packed(torch.zeros(rows, n, device="cuda"), 77.0) for _ in range(2))
    w, b, stats = cuda(i["w"]), cuda(i["b"]), torch.empty(rows, 2, device="cuda")
    dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(max(16, _lib.layernorm_workspace_bytes(rows, n)), dtype=torch.uint8, device="cuda")
    _lib.cfc_layernorm_forward(x, w, b, y, stats)
    _lib.cfc_layernorm_backward(dy, x, w, stats, dx, dw, db, ws)
    check(y, ot.layernorm(i["x"], i["w"], i["b"], 1e-5), EL, "y")
    for got, want in zip((dx, dw, db), ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)):
        if n > 1 or want is not None and np.any(want):
            check(got, want, SUM)
    for buf in (yb, db_):
        assert (buf[:offset] == 77.0).all() and (buf[offset + rows * n:] == 77.0).all()


def test_layernorm_many_rows_is_reproducible():
    """More rows than the backward's CTAs take in one turn; bitwise the same twice and in a graph."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = norm_inputs(9001, 48, "f32", 3)
    st = trunk.LayerNormStep(9001, 48).bind(cuda(i["x"]), cuda(i["w"]), cuda(i["b"]), cuda(i["dy"]))
    st.run()
    first = {k: v.clone() for k, v in st.outputs().items()}
    for got, want in zip((first["dx"], first["dw"], first["db"]),
                         ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)):
        check(got, want, SUM)
    st.run()
    assert all(torch.equal(first[k], v) for k, v in st.outputs().items())
    st.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], v) for k, v in st.outputs().items())


def test_layernorm_far_mean_and_constant_rows():
    """A mean a thousand standard deviations away costs what the rounding of the mean costs: at
    most about ten additions of 2^-24 * 1000 each.  A constant row gives b."""
    from recurrent_cfc_cell_gb300 import trunk

    i = norm_inputs(6, 512, "f32", 4, mean=1500.0)
    st = trunk.LayerNormStep(6, 512).bind(cuda(i["x"]), cuda(i["w"]), cuda(i["b"]))
    st.run()
    check(st.y, ot.layernorm(i["x"], i["w"], i["b"], 1e-5), 10 * 1000 * 2.0 ** -24)
    i["x"][:] = 3.0
    st = trunk.LayerNormStep(6, 512).bind(cuda(i["x"]), cuda(i["w"]), cuda(i["b"]))
    st.run()
    check(st.y, np.broadcast_to(i["b"], (6, 512)), EL)


def rng_tensor(seed, offset):
    import torch

    signed = [v - (1 << 64) if v >= 1 << 63 else v for v in (seed, offset)]
    return torch.tensor(signed, dtype=torch.int64, device="cuda")


SEED, OFFSET = 0xFEDCBA9876543210, 0x8000000500000003


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,p,residual", [
    (1, 1, 0.5, False), (5, 8, 0.1, True), (7, 31, 0.3, True), (40, 64, 0.25, False),
    (3, 257, 0.1, True), (2, 1003, 0.7, True), (6, 40, 0.0, True), (6, 40, 1.0, True)])
def test_dropout(rows, n, p, residual, dtype):
    """Exactly the oracle's mask and, fp32 product and sum rounded apart, exactly its values; the
    backward pass is the same mask on the gradient.  What is dropped may hold anything."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    i = norm_inputs(rows, n, dtype, 8)
    keep, scale = ot.dropout_mask(rows, n, p, SEED, OFFSET)
    x, res, rng = cuda(i["x"], dtype), cuda(i["residual"], dtype), rng_tensor(SEED, OFFSET)
    x[torch.from_numpy(~keep).cuda()] = float("nan")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    _lib.cfc_dropout_forward(x, res if residual else None, rng, p, y)
    kept = np.where(keep, i["x"], 0.0).astype(np.float32) * np.float32(scale)
    want = kept + i["residual"].astype(np.float32) if residual else kept
    want = torch.from_numpy(want).to(y.dtype)
    assert torch.equal(y.cpu(), want)
    _lib.cfc_dropout_backward(cuda(i["dy"], dtype), rng, p, dx)
    want = torch.from_numpy(np.where(keep, i["dy"], 0.0).astype(np.float32) * np.float32(scale))
    assert torch.equal(dx.cpu(), want.to(dx.dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,with_res,with_ds", [
    (1, 8, True, True), (50, 32, True, True), (21, 45, True, True), (35, 128, False, True),
    (19, 250, True, False), (8, 600, True, True), (5, 1001, True, True), (4, 2500, True, True),
    (3, 5001, True, True), (2, 8193, True, True)])
def test_dropout_layernorm(rows, n, with_res, with_ds, dtype):
    from recurrent_cfc_cell_gb300 import trunk

    p = 0.2
    i = norm_inputs(rows, n, dtype, rows + n)
    rng = rng_tensor(SEED, OFFSET)
    st = trunk.DropoutNormStep(rows, n, p, act(dtype)).bind(
        cuda(i["x"], dtype), cuda(i["residual"], dtype) if with_res else None, rng, cuda(i["w"]),
        cuda(i["b"]), cuda(i["dy"], dtype), cuda(i["ds"], dtype) if with_ds else None)
    st.run()
    out = st.outputs()
    keep, scale = ot.dropout_mask(rows, n, p, SEED, OFFSET)
    s = (i["residual"] if with_res else 0.0) + keep * i["x"] * scale
    check(out["s"], s, EL, "s")
    s = out["s"].double().cpu().numpy()  # the norm reads the stream as it is stored
    check(out["y"], ot.layernorm(s, i["w"], i["b"], 1e-5), EL, "y")
    d, dw, db = ot.layernorm_backward(i["dy"], s, i["w"], 1e-5)
    dres = d + (i["ds"] if with_ds else 0.0)
    check(out["dres"], dres, SUM, "dres")
    check(out["dx"], keep * dres * scale, SUM, "dx")
    check(out["dw"], dw, SUM, "dw")
    check(out["db"], db, SUM, "db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(6200, 1030), (6200, 1040), (1900, 5001), (1900, 4104)])
def test_wide_rows_in_many_turns(rows, n, dtype):
    """Whole-CTA rows, several to a CTA (four and more in every kernel), aligned and not, so that
    the places where rows wait are used again.  The parameters' sums of N rows: N terms of random
    sign leave about sqrt(N) 2^-24 sum|t| / max|sum| < 1e-5."""
    from recurrent_cfc_cell_gb300 import trunk

    p = 0.2
    i = norm_inputs(rows, n, dtype, rows + n)
    x, w, b = cuda(i["x"], dtype), cuda(i["w"]), cuda(i["b"])
    dy = cuda(i["dy"], dtype)
    st = trunk.LayerNormStep(rows, n, act(dtype)).bind(x, w, b, dy)
    st.run()
    out = st.outputs()
    check(out["y"], ot.layernorm(i["x"], i["w"], i["b"], 1e-5), EL, "y")
    for name, want in zip(("dx", "dw", "db"), ot.layernorm_backward(i["dy"], i["x"], i["w"], 1e-5)):
        check(out[name], want, SUM, name)
    st = trunk.DropoutNormStep(rows, n, p, act(dtype)).bind(
        x, cuda(i["residual"], dtype), rng_tensor(SEED, OFFSET), w, b, dy, cuda(i["ds"], dtype))
    st.run()
    out = st.outputs()
    keep, scale = ot.dropout_mask(rows, n, p, SEED, OFFSET)
    check(out["s"], i["residual"] + keep * i["x"] * scale, EL, "s")
    s = out["s"].double().cpu().numpy()
    check(out["y"], ot.layernorm(s, i["w"], i["b"], 1e-5), EL, "y")
    d, dw, db = ot.layernorm_backward(i["dy"], s, i["w"], 1e-5)
    check(out["dres"], d + i["ds"], SUM, "dres")
    check(out["dx"], keep * (d + i["ds"]) * scale, SUM, "dx")
    check(out["dw"], dw, SUM, "dw")
    check(out["db"], db, SUM, "db")


def test_dropout_offset_advances_in_a_graph():
    """The generator's state is read when the kernel runs: a replayed graph draws a new mask once
    the caller has moved the offset."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = norm_inputs(16, 64, "f32", 2)
    rng = rng_tensor(3, 4)
    st = trunk.DropoutNormStep(16, 64, 0.5).bind(cuda(i["x"]), None, rng, cuda(i["w"]), cuda(i["b"]))
    st.capture()
    for offset in (4, 5):
        rng[1] = offset
        st.replay()
        torch.cuda.synchronize()
        keep, _ = ot.dropout_mask(16, 64, 0.5, 3, offset)
        assert np.array_equal(st.s.cpu().numpy() != 0, keep)


# ---- causal convolution ----

def ends_of(lengths, K, B):
    return np.full(B, K) if lengths is None else np.clip(lengths, 0, K)


def lengths_tensor(lengths):
    import torch

    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


# Lengths below zero and beyond K are clamped.
CONVS = [(1, 1, 1, 2, None), (1, 3, 8, 4, None), (2, 2, 16, 4, [0, 1]), (5, 3, 7, 3, None),
         (40, 2, 64, 4, None), (67, 4, 40, 4, [67, 0, 3, 30]), (130, 3, 33, 2, [5, 129, 130]),
         (300, 2, 128, 3, [-4, 999]), (9, 70, 24, 4, None)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,B,D,W,lengths", CONVS)
def test_conv(K, B, D, W, lengths, dtype):
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    i = conv_inputs(K, B, D, W, dtype, K + D)
    ends = ends_of(lengths, K, B)
    x, du = cuda(i["x"], dtype), cuda(i["du"], dtype)
    for b in range(B):  # what lies beyond a sequence's end is not read
        x[ends[b]:, b] = float("nan")
        du[ends[b]:, b] = float("nan")
    st = trunk.ConvStep(K, B, D, W, act(dtype)).bind(
        x, cuda(i["w"]), cuda(i["bias"]), cuda(i["x0"], dtype), lengths_tensor(lengths), du)
    for t in (st.u, st.last, st.dx, st.dx0):
        t.fill_(float("nan"))
    st.run()
    out = st.outputs()
    u, last = ot.conv(i["x"], i["w"], i["bias"], i["x0"], ends)
    check(out["u"], u, EL, "u")
    assert torch.equal(out["last"].double().cpu(), torch.from_numpy(last))
    for got, want, name in zip((out["dx"], out["dx0"], out["dw"], out["dbias"]),
                               ot.conv_backward(i["du"], i["x"], i["w"], i["bias"], i["x0"], ends),
                               ("dx", "dx0", "dw", "dbias")):
        check(got, want, SUM, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("silu", [True, False])
def test_conv_batch_first_views_and_no_options(silu, dtype):
    """Batch-first memory, a channel slice that starts off alignment, no bias and no history."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    K, B, D, W = 20, 3, 32, 4
    i = conv_inputs(K, B, D, W, dtype, 6)
    x = wide(cuda(i["x"].transpose(1, 0, 2), dtype), 6).transpose(0, 1)
    du = wide(cuda(i["du"], dtype), 3)
    u = torch.empty(B, K, D, dtype=act(dtype), device="cuda").transpose(0, 1)
    dx = torch.empty_like(u)
    dw, db = torch.empty(D, W, device="cuda"), torch.empty(D, device="cuda")
    code = _lib.CFC_F32 if dtype == "f32" else _lib.CFC_BF16
    ws = torch.empty(_lib.conv_workspace_bytes(B, K, D, W, code), dtype=torch.uint8, device="cuda")
    _lib.cfc_conv_forward(x, cuda(i["w"]), u, silu=silu)
    _lib.cfc_conv_backward(du, x, cuda(i["w"]), dx, dw, db, ws=ws, silu=silu)
    none, zero = np.zeros((B, W - 1, D)), np.zeros(D)
    check(u, ot.conv(i["x"], i["w"], zero, none, [K] * B, silu)[0], EL, "u")
    want = ot.conv_backward(i["du"], i["x"], i["w"], zero, none, [K] * B, silu)
    check(dx, want[0], SUM, "dx")
    check(dw, want[2], SUM, "dw")
    check(db, want[3], SUM, "dbias")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,W", [(1, 1, 2), (3, 40, 4), (5, 33, 3), (2, 1024, 4)])
def test_conv_tokens_are_the_prompt(B, D, W, dtype):
    """Token by token, the state updated in place: the prompt's outputs and its last inputs."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    K = 6
    i = conv_inputs(K, B, D, W, dtype, 12)
    x, w, bias, state = cuda(i["x"], dtype), cuda(i["w"]), cuda(i["bias"]), cuda(i["x0"], dtype)
    want = trunk.ConvStep(K, B, D, W, act(dtype)).bind(x, w, bias, state.clone())
    want.run()
    tok = trunk.ConvToken(B, D, W, act(dtype))
    for t in range(K):
        u, state = tok.bind(x[t], w, state, bias).run()
        assert torch.equal(u, want.u[t])
    assert torch.equal(state, want.last)


# ---- selective scan ----

GRADS = (("dx", EL * 10), ("ddt", SUM), ("dz", SUM), ("dA", SUM), ("dB", SUM), ("dC", SUM),
         ("dD", SUM), ("ddt_bias", SUM), ("dh0", SUM))

# (K, B, D, N, G, lengths): single steps, chunk edges, ragged channels and states, groups, lengths
# of zero, one and beyond; the last two split the steps over CTAs.
SCANS = [(1, 1, 1, 1, 1, None), (1, 3, 40, 16, 1, None), (7, 2, 33, 4, 1, None),
         (8, 2, 64, 16, 2, [8, 0]), (9, 2, 130, 16, 1, [1, 9]), (17, 3, 48, 5, 3, [17, 16, 8]),
         (12, 2, 36, 24, 2, None), (20, 1, 70, 32, 1, [11]), (10, 2, 34, 40, 1, [0, 0]),
         (11, 1, 40, 64, 2, None), (9, 2, 33, 100, 1, [9, 4]), (6, 1, 16, 128, 1, [-2]),
         (700, 1, 40, 8, 1, None), (1030, 2, 24, 16, 2, [1030, 517])]


def bind_scan(i, K, B, D, N, G, dtype, lengths=None, **over):
    from recurrent_cfc_cell_gb300 import trunk

    ends = ends_of(lengths, K, B)
    t = {k: cuda(i[k], dtype) for k in ("x", "dt", "z", "Bm", "Cm", "dy")}
    for v in t.values():
        for b in range(B):
            v[ends[b]:, b] = float("nan")
    st = trunk.ScanStep(K, B, D, N, G, act(dtype), train=True)
    for v in vars(st).values():
        if hasattr(v, "fill_") and v.is_floating_point():
            v.fill_(float("nan"))
    args = dict(A=cuda(i["A"]), D=cuda(i["skip"]), dt_bias=cuda(i["dt_bias"]), h0=cuda(i["h0"]),
                dh_last=cuda(i["dh_last"]), lengths=lengths_tensor(lengths), **t)
    args.update(over)
    return st.bind(**args)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,B,D,N,G,lengths", SCANS)
def test_scan(K, B, D, N, G, lengths, dtype):
    i = scan_inputs(K, B, D, N, G, dtype, K + N)
    ends = ends_of(lengths, K, B)
    st = bind_scan(i, K, B, D, N, G, dtype, lengths)
    st.run()
    out = st.outputs()
    y, h, _ = ot.scan(i, ends)
    check(out["y"], y, EL, "y")
    check(out["h"], h, EL, "h")
    g = ot.scan_backward(i, ends, i["dy"], i["dh_last"])
    g["dD"] = g["dskip"]
    for k, tol in GRADS:
        check(out[k], g[k], tol, k)


def test_scan_prompt_without_training_is_the_same():
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    K, B, D, N, G = 50, 2, 48, 16, 2
    i = scan_inputs(K, B, D, N, G, "f32", 1)
    st = bind_scan(i, K, B, D, N, G, "f32", [50, 20])
    st.run()
    a = {k: v for k, v in st.inputs.items() if k not in ("dy", "dh_last")}
    pr = trunk.ScanStep(K, B, D, N, G).bind(**a)
    pr.run()
    assert torch.equal(pr.y, st.y) and torch.equal(pr.h, st.h)
    with pytest.raises(ValueError):
        trunk.ScanStep(K, B, D, N, G).bind(**st.inputs)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scan_without_options(dtype):
    """No gate, skip, bias, history, softplus or gradient of the last state."""
    from recurrent_cfc_cell_gb300 import _lib
    import torch

    K, B, D, N, G = 19, 2, 36, 16, 1
    i = scan_inputs(K, B, D, N, G, dtype, 4)
    i["dt"] = np.abs(i["dt"]) * 0.125
    x, dt, Bm, Cm, dy = (cuda(i[k], dtype) for k in ("x", "dt", "Bm", "Cm", "dy"))
    A = cuda(i["A"])
    y, dx, ddt = (torch.empty_like(x) for _ in range(3))
    states = torch.empty(-(-K // _lib.SCAN_PERIOD), B, D, N, device="cuda")
    dA, dB, dC = torch.empty_like(A), torch.empty_like(Bm), torch.empty_like(Cm)
    code = _lib.CFC_F32 if dtype == "f32" else _lib.CFC_BF16
    ws = torch.empty(_lib.scan_workspace_bytes(K, B, D, N, G, code, True), dtype=torch.uint8, device="cuda")
    _lib.cfc_scan_forward(x, dt, A, Bm, Cm, y, states=states, softplus=False)
    _lib.cfc_scan_backward(dy, x, dt, A, Bm, Cm, states, dx, ddt, dA, dB, dC, ws=ws, softplus=False)
    i.update(z=None, skip=np.zeros(D), dt_bias=np.zeros(D), h0=np.zeros((B, D, N)))
    check(y, ot.scan(i, [K] * B, False)[0], EL, "y")
    g = ot.scan_backward(i, [K] * B, i["dy"], np.zeros((B, D, N)), False)
    for got, k in ((dx, "dx"), (ddt, "ddt"), (dA, "dA"), (dB, "dB"), (dC, "dC")):
        check(got, g[k], SUM, k)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scan_views_and_repeats(dtype):
    """Batch-first memory, slices of packed projections off alignment, bitwise the same as
    contiguous inputs, twice, and in a graph on another stream."""
    import torch

    K, B, D, N, G = 30, 3, 40, 12, 2
    i = scan_inputs(K, B, D, N, G, dtype, 2)
    st = bind_scan(i, K, B, D, N, G, dtype)
    st.run()
    first = {k: v.clone() for k, v in st.outputs().items()}
    t = {k: cuda(i[k], dtype) for k in ("x", "dt", "z", "dy")}
    v = {"x": wide(t["x"].transpose(0, 1).contiguous(), 3).transpose(0, 1), "dt": wide(t["dt"], 2),
         "z": torch.cat([t["x"], t["z"]], -1)[..., D:], "dy": wide(t["dy"], 7)}
    bc = torch.cat([cuda(i["Bm"], dtype).flatten(2), cuda(i["Cm"], dtype).flatten(2)], -1)
    bc = wide(bc, 1)
    v["Bm"], v["Cm"] = (m.unflatten(-1, (G, N)) for m in (bc[..., :G * N], bc[..., G * N:]))
    again = bind_scan(i, K, B, D, N, G, dtype, **v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again.run()
        again.replay()
    s.synchronize()
    for k, a in again.outputs().items():
        assert torch.equal(first[k], a), k


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,N,G", [(1, 1, 1, 1), (3, 40, 16, 1), (6, 33, 5, 3), (2, 20, 64, 2),
                                     (5, 9, 100, 1), (2, 4, 128, 4)])
def test_scan_tokens_follow_the_prompt(B, D, N, G, dtype):
    """Token by token from the prompt's state, in place, against the oracle over both."""
    from recurrent_cfc_cell_gb300 import trunk

    K, P = 9, 5
    i = scan_inputs(K, B, D, N, G, dtype, 3)
    y, h, _ = ot.scan(i, [K] * B)
    t = {k: cuda(i[k], dtype) for k in ("x", "dt", "z", "Bm", "Cm")}
    par = dict(A=cuda(i["A"]), D=cuda(i["skip"]), dt_bias=cuda(i["dt_bias"]))
    prompt = trunk.ScanStep(P, B, D, N, G, act(dtype)).bind(
        **{k: v[:P] for k, v in t.items()}, **par, h0=cuda(i["h0"]))
    prompt.run()
    state = prompt.h.clone()
    tok = trunk.ScanToken(B, D, N, G, act(dtype))
    for k in range(P, K):
        yk, state = tok.bind(**{n: v[k] for n, v in t.items()}, **par, state=state).run()
        check(yk, y[k], EL * max(1.0, np.abs(y).max() / np.abs(y[k]).max()), "y")
    check(state, h, EL, "h")


def test_refusals_raise():
    import torch

    from recurrent_cfc_cell_gb300 import _lib, trunk

    x = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(8, device="cuda")
    ok = dict(x=x, w=w, b=w, y=torch.empty_like(x), stats=torch.empty(4, 2, device="cuda"))
    for k, v in (("w", w[:7]), ("w", w.bfloat16()), ("x", x.half()), ("x", x.cpu()),
                 ("y", torch.empty(8, 4, device="cuda").T), ("y", torch.empty(4, 9, device="cuda")),
                 ("stats", None)):
        with pytest.raises((ValueError, _lib.CfcError)):
            _lib.cfc_layernorm_forward(**{**ok, k: v})
    with pytest.raises(_lib.CfcError):
        _lib.cfc_layernorm_forward(**ok, eps=float("nan"))
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(_lib.CfcError):
            _lib.cfc_dropout_forward(x, None, rng, p, torch.empty_like(x))
    with pytest.raises(ValueError):
        _lib.cfc_dropout_forward(x, None, rng.int(), 0.1, torch.empty_like(x))
    with pytest.raises(_lib.CfcError):
        trunk.ConvStep(4, 2, 8, 5).bind(torch.zeros(4, 2, 8, device="cuda"),
                                        torch.zeros(8, 5, device="cuda")).run()
    with pytest.raises(_lib.CfcError):
        trunk.ScanStep(4, 2, 8, 129)
    with pytest.raises(_lib.CfcError):
        trunk.ScanStep(4, 2, 9, 4, G=2)
