"""The root-mean-square norm where numbers end (infinities, NaN, squares and products beyond fp32), beside
the borders between two 8-bit codes, in every layout to and from 8 bits, and with many rows a CTA.

Tolerances are those of the operators' tests: 1e-5 max|y| per element, 1e-4 max|y| for sums, plus 2^-8 |y|
for a rounding to bf16; what is held in 8 bits is compared bit by bit."""
import numpy as np
import pytest

import oracle.gated as og
from gated_cases import rms_inputs, rounded
from test_gated_gpu import EL, SUM, act, built, check, cuda, held_bits, wide  # noqa: F401 (built: the fixture)

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [8, 40, 37, 256, 1000, 1537, 5000, 8193])
def test_rows_that_are_not_numbers(n, dtype):
    """A NaN makes its row NaN; an infinity and squares beyond fp32 make rstd 0, so that y is 0 but for the
    infinity, which is NaN; other rows are as they were, also to 8 bits."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    x = torch.randn(12, n, device="cuda").to(act(dtype))
    w = torch.rand(n, device="cuda") + 0.5
    w[n // 2] = 1e30  # s w is beyond fp32 where s is 1e19
    clean = x.clone()
    x[2, n - 1] = float("nan")
    x[5, n // 3] = float("inf")
    x[7, 0] = -float("inf")
    x[9] = 3e19
    x[9, n // 2] = -2e38
    ok = [r for r in range(12) if r not in (2, 5, 7, 9)]
    for out8 in (False, True):
        a = trunk.RMSNormStep(12, n, act(dtype), out8=out8).bind(x, w)
        b = trunk.RMSNormStep(12, n, act(dtype), out8=out8).bind(clean, w)
        ys = []
        for st in (a, b):
            st.run()
            ys.append(trunk.Unpack8Step(12, n).bind(st.y8).run().clone() if out8 else st.y)
        y = ys[0]
        assert torch.equal(y[ok], ys[1][ok])
        assert torch.isnan(y[2]).all() and torch.isnan(a.rstd[2])
        assert not a.rstd[[5, 7, 9]].any()
        for r, c in ((5, n // 3), (7, 0)):
            bad = torch.isnan(y[r])
            block = torch.zeros(n, dtype=torch.bool, device="cuda")
            if out8:  # its whole block
                block[c // 32 * 32:c // 32 * 32 + 32] = True
            else:
                block[c] = True
            assert torch.equal(bad, block) and not y[r][~bad].any()
        assert not y[9].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [64, 1537])
def test_products_beyond_fp32_on_the_way(n, dtype):
    """s w alone is beyond fp32, or below it, and y is neither."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    big, small = torch.randn(6, n, device="cuda") * 1e17, torch.randn(6, n, device="cuda") * 1e-17
    for x, w in ((big, 1e25), (small, 1e-25)):
        x, w = x.to(act(dtype)), torch.full((n,), w, device="cuda")
        dy = torch.randn(6, n, device="cuda").to(act(dtype))
        st = trunk.RMSNormStep(6, n, act(dtype), eps=0.0).bind(x, w, dy=dy)
        st.run()
        v = x.double()
        want = (v / torch.sqrt((v * v).mean(1, keepdim=True)) * w.double()).cpu().numpy()
        check(st.y, want, EL, "y")
        st8 = trunk.RMSNormStep(6, n, act(dtype), eps=0.0, out8=True).bind(x, w)
        st8.run()
        got = trunk.Unpack8Step(6, n).bind(st8.y8).run().double().cpu().numpy()
        assert np.array_equal(got, og.held8(want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [96, 1024, 2501, 8192, 9000])
def test_codes_as_near_to_borders_as_weights_bring_them(n, dtype):
    """Weights that bring every y of a row to within half a place of a border between two codes: an error
    of 3e-8 anywhere in rstd or in the products takes the wrong code for about half of them.  What is
    within 2^-39 of a border, relative to y, is not looked at: the sums of squares keep 48 bits of each
    term, up to 2^4 roundings of 2^-48 a thread, whose parts may be 2^4 times as large."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    for seed in range(6):
        r = np.random.default_rng(100 * n + seed)
        s = rounded(r.normal(size=(1, n)), dtype)
        s = np.where(np.abs(s) < 0.05, 0.5, s)
        rstd = 1.0 / np.sqrt((s * s).mean() + float(np.float32(1e-5)))
        ties = (og.E4M3[9:] + og.E4M3[8:-1]) / 2
        u = r.choice(ties[ties < 440], size=n)
        u[::32] = 448.0 * (1 - 2.0 ** -20)  # holds the block's scale at 1, off a border
        w = (u / (s[0] * rstd)).astype(np.float32)
        y = s[0] * rstd * w.astype(np.float64)
        st = trunk.RMSNormStep(1, n, act(dtype), out8=True).bind(cuda(s, dtype), torch.from_numpy(w).cuda())
        st.run()
        got = trunk.Unpack8Step(1, n).bind(st.y8).run().double().cpu().numpy()[0]
        want = og.held8(y[None])[0]
        sure = np.abs(y / u - 1) > 2.0 ** -39
        assert np.all((got == want) | ~sure)
        assert sure.mean() > 0.99 and np.all(np.abs(y / u - 1) <= 2.0 ** -24 * 1.000001)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,pad,off", [(9, 64, 3, 0), (9, 64, 8, 0), (9, 64, 0, 1), (9, 256, 8, 4),
                                            (5, 300, 5, 0), (33, 96, 0, 3), (5, 1024, 1, 0), (3, 8200, 3, 1)])
def test_to_and_from_8_bits_anywhere(rows, n, pad, off, dtype):
    """Strided inputs, codes that start off an 8-byte border, the sum in the residual's memory."""
    import torch

    from recurrent_cfc_cell_gb300 import _lib

    i = rms_inputs(rows, n, dtype, rows * 41 + n + pad)

    def held():
        codes = torch.zeros(rows * n + off, dtype=torch.uint8, device="cuda")[off:].view(rows, n)
        return _lib.Held8((rows, n), codes=codes)

    s8, y8 = held(), held()
    x, res = wide(cuda(i["x"], dtype), pad), wide(cuda(i["residual"], dtype), pad, 7.0)
    w, rstd = cuda(i["w"]), cuda(np.zeros(rows))
    _lib.cfc_rmsnorm_forward(x, w, res, res, None, s8, y8, rstd)
    assert np.array_equal(res.double().cpu().numpy(), i["s"])
    if pad:
        assert (res._base[..., 0] == 7.0).all() and (res._base[..., 1 + n:] == 7.0).all()
    want = [og.pack8(row) for row in i["s"]]
    codes, scales = held_bits(s8)
    assert np.array_equal(scales, np.stack([s for _, s in want]))
    assert np.array_equal(codes, np.stack([c for c, _ in want]))
    y = og.rmsnorm(i["s"], i["w"], float(np.float32(1e-5)))
    assert np.array_equal(np.stack([og.unpack8(c, s) for c, s in zip(*held_bits(y8))]), og.held8(y))
    dy, ds = wide(cuda(i["dy"], dtype), pad), wide(cuda(i["ds"], dtype), pad)
    dw, again = cuda(np.zeros(n)), wide(cuda(np.zeros((rows, n)), dtype), pad)
    ws = torch.empty(max(_lib.rmsnorm_workspace_bytes(rows, n), 16), dtype=torch.uint8, device="cuda")
    _lib.cfc_rmsnorm_backward(dy, s8, w, rstd, ds, dw, ds, again, ws)  # dx in ds's place
    dx, want_dw, want_y = og.rmsnorm_backward(i["dy"], i["s"], i["w"], 1e-5, og.held8(i["s"]), i["ds"])
    check(ds, dx, SUM, "dx")
    check(dw, want_dw, SUM, "dw")
    check(again, want_y, EL, "y_again")


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_rows_in_many_turns(dtype):
    """More rows of more than 8192 columns than the GPU holds CTAs for, the sum in the residual's place."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    rows, n = 1501, 8203
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *a: torch.randn(*a, generator=g, device="cuda").to(act(dtype))  # noqa: E731
    x, res, dy, ds = r(rows, n), r(rows, n), r(rows, n), r(rows, n)
    w = torch.rand(n, generator=g, device="cuda") + 0.5
    st = trunk.RMSNormStep(rows, n, act(dtype), keep8=True).bind(x, w, res, dy, ds)
    st.run()
    s = (x.float() + res.float()).to(act(dtype))
    assert torch.equal(st.s, s)
    s = s.double()
    scale = torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-5)
    check(st.y, (s * scale * w).cpu().numpy(), EL, "y")
    held = trunk.Unpack8Step(rows, n).bind(st.s8).run().double()
    assert ((held - s).abs() <= 2.0 ** -4 * s.abs() + 2.0 ** -9).all()
    hat, gr = held * scale, dy.double() * w
    dx = scale * (gr - hat * (gr * hat).mean(1, keepdim=True)) + ds.double()
    check(st.dx, dx.cpu().numpy(), SUM, "dx")
    check(st.dw, (dy.double() * hat).sum(0).cpu().numpy(), SUM, "dw")
    check(st.y_again, (hat * w).cpu().numpy(), EL, "y_again")


@pytest.mark.parametrize("backward", [False, True])
def test_long_rows_go_side_by_side(backward):
    """64 rows of more than 8192 columns take about as long as one of them, each on an SM of its own: with
    eight rows to a CTA they would take eight times as long."""
    import torch

    from recurrent_cfc_cell_gb300 import trunk

    def us(rows):
        r = lambda *a: torch.randn(*a, device="cuda")  # noqa: E731
        st = trunk.RMSNormStep(rows, 65536).bind(r(rows, 65536), r(65536), dy=r(rows, 65536))
        run, times = st.backward if backward else st.forward, []
        st.run()
        for _ in range(40):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            run()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[20]

    one, many = us(1), us(64)
    assert many < 4 * one, f"{one} and {many} ms"
