"""The trunk operators at the sizes, alignments and state counts that choose each kernel variant:
several turns of every team of norm rows, tensors aligned unlike one another, results in an input's
memory, every run length of the convolution, every tile and split of the scan, sixteen sequences a
CTA of the token step, and strides past 32 bits.

References are float64 (trunk_plain64.py) on the values that the tested type holds.  Tolerances as
in test_trunk_gpu.py: |x - y| <= tol max|y|, 1e-5 for what a pass computes per element and 1e-4 for
sums over rows or steps, bf16 results plus 2^-8 |y|.  They cover the longer sums here: N terms of
random sign added by P threads (m = N / P each) leave sqrt(P) m 2^-25 of a term's size beside a sum of
about sqrt(N), that is sqrt(m) 2^-25 < 1e-6 of it for the m < 1000 of these sizes."""
import pytest
import torch

import trunk_plain64 as p64
from test_trunk_gpu import EL, OFFSET, SEED, SUM, act, rng_tensor
from trunk_draws import Draw, check, doubles, norm_inputs, scan_inputs

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from recurrent_cfc_cell_gb300 import build

    build.build()


class Placed:
    """A tensor's rows packed from element `offset` of a buffer on, so that it is aligned as
    wanted; what surrounds it (`fill`) has to stay."""

    def __init__(self, t, offset, fill=77.0):
        n = t.numel()
        self.buf = torch.full((n + 24,), fill, dtype=t.dtype, device="cuda")
        self.at, self.n = offset, n
        self.t = self.buf[offset:offset + n].view(t.shape)
        self.t.copy_(t)

    def alone(self):
        return bool((self.buf[:self.at] == 77.0).all() and (self.buf[self.at + self.n:] == 77.0).all())


# ---- layer norm and dropout ----

def norm_calls(i, place, p=0.2):
    """Every norm and dropout entry point on i's tensors, each put where `place` (name, tensor)
    wants it; the results by name."""
    from recurrent_cfc_cell_gb300 import _lib

    rows, n = i["x"].shape
    t = {k: place(k, v) if v.dim() == 2 else v for k, v in i.items()}
    o = {k: place(k, torch.zeros_like(i["x"])) for k in
         ("y", "dx", "drop", "ddrop", "s", "sy", "sdx", "sdres")}
    f = {k: torch.empty(n, device="cuda") for k in ("dw", "db", "sdw", "sdb")}
    stats, rng = torch.empty(rows, 2, device="cuda"), rng_tensor(SEED, OFFSET)
    ws = torch.empty(max(16, _lib.layernorm_workspace_bytes(rows, n)), dtype=torch.uint8,
                     device="cuda")
    _lib.cfc_layernorm_forward(t["x"], t["w"], t["b"], o["y"], stats)
    _lib.cfc_layernorm_backward(t["dy"], t["x"], t["w"], stats, o["dx"], f["dw"], f["db"], ws)
    _lib.cfc_dropout_forward(t["x"], t["residual"], rng, p, o["drop"])
    _lib.cfc_dropout_backward(t["dy"], rng, p, o["ddrop"])
    _lib.cfc_dropout_layernorm_forward(t["x"], t["residual"], rng, p, t["w"], t["b"], o["s"],
                                       o["sy"], stats)
    _lib.cfc_dropout_layernorm_backward(t["dy"], t["ds"], o["s"], rng, p, t["w"], stats, o["sdx"],
                                        o["sdres"], f["sdw"], f["sdb"], ws)
    return {**o, **f}


def norm_checks(i, out, p=0.2):
    rows, n = i["x"].shape
    d = doubles(i)
    check(out["y"], p64.norm(d["x"], d["w"], d["b"]), EL, "y")
    for k, v in zip(("dx", "dw", "db"), p64.norm_backward(d["dy"], d["x"], d["w"])):
        check(out[k], v, SUM, k)
    keep, scale = p64.dropout_mask(rows, n, p, SEED, OFFSET, "cuda")
    # Product and sum are rounded apart, in fp32: exactly these values.
    scale32 = torch.tensor(scale, dtype=torch.float32, device="cuda")
    zero = torch.zeros((), device="cuda")
    kept = torch.where(keep, i["x"].float() * scale32, zero)
    s = (i["residual"].float() + kept).to(i["x"].dtype)
    assert torch.equal(out["drop"], s) and torch.equal(out["s"], s)
    kept = torch.where(keep, i["dy"].float() * scale32, zero)
    assert torch.equal(out["ddrop"], kept.to(i["x"].dtype))
    s = s.double()
    check(out["sy"], p64.norm(s, d["w"], d["b"]), EL, "y of s")
    dn, dw, db = p64.norm_backward(d["dy"], s, d["w"])
    dres = dn + d["ds"]
    check(out["sdres"], dres, SUM, "dres")
    check(out["sdx"], torch.where(keep, dres * scale, 0.0), SUM, "dx of s")
    check(out["sdw"], dw, SUM, "dw of s")
    check(out["sdb"], db, SUM, "db of s")


# Widths of every team of less than a CTA, aligned and odd (which take the next wider one from seven
# columns below the team's own), with the teams that share a CTA.
TEAMS = [(32, 25, 64), (64, 57, 32), (128, 121, 16), (256, 249, 8), (512, 505, 4), (1024, 1017, 2)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["aligned", "shifted", "scalar"])
@pytest.mark.parametrize("even,odd,teams", TEAMS)
def test_norm_rows_in_many_turns(even, odd, teams, layout, dtype):
    """More rows than twice what the largest grid (1216 CTAs) takes at once, the last turn partly
    idle."""
    rows, n = 2 * 1216 * teams + teams // 2 + 3, even if layout == "aligned" else odd
    i = norm_inputs(rows, n, dtype, rows + n)
    places = {}

    def place(name, t):
        if layout != "scalar":
            return t
        places[name] = Placed(t, len(places) % 8 + 1)
        return places[name].t

    norm_checks(i, norm_calls(i, place))
    assert all(v.alone() for v in places.values())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(1, 5), (3, 7), (5, 32), (70, 31), (9, 100), (4, 256), (6, 500),
                                    (5, 1000), (7, 2501), (3, 5000), (2, 8192), (3, 8193)])
def test_norm_tensors_aligned_unlike(rows, n, dtype):
    """Every tensor starts at another place within its group of eight."""
    i = norm_inputs(rows, n, dtype, rows * 17 + n)
    places = {}

    def place(name, t):
        places[name] = Placed(t, len(places) % 8 + 1)
        return places[name].t

    norm_checks(i, norm_calls(i, place))
    assert all(v.alone() for v in places.values())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,ld", [(40, 96, 104), (9, 250, 253), (6, 1030, 1032), (5, 40, 41)])
def test_dropout_strided_rows(rows, n, ld, dtype):
    """Rows further apart than they are long; nothing is written beside them."""
    i = norm_inputs(rows, n, dtype, 9)
    bigs = []

    def place(name, t):
        big = torch.full((rows, ld), 77.0, dtype=t.dtype, device="cuda")
        big[:, :n] = t
        bigs.append(big)
        return big[:, :n]

    norm_checks(i, norm_calls(i, place))
    assert all(bool((b[:, n:] == 77.0).all()) for b in bigs)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(700, 8192), (700, 8185), (400, 4104), (400, 4090)])
def test_widest_rows_in_many_turns(rows, n, dtype):
    """The rows that take most of the shared memory, more of them than CTAs."""
    i = norm_inputs(rows, n, dtype, rows + n)
    norm_checks(i, norm_calls(i, lambda name, t: t))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(3000, 32), (3000, 25), (3000, 256), (3001, 249), (1500, 1003),
                                    (700, 2504), (700, 2501), (300, 8185), (50, 8193)])
def test_results_in_an_inputs_memory(rows, n, dtype):
    """The calls that may write where they read, against the same calls that do not, bit by bit."""
    from recurrent_cfc_cell_gb300 import _lib

    i = norm_inputs(rows, n, dtype, n)
    x, dy, w = i["x"], i["dy"], i["w"]
    stats, rng = torch.empty(rows, 2, device="cuda"), rng_tensor(SEED, OFFSET)
    ws = torch.empty(max(16, _lib.layernorm_workspace_bytes(rows, n)), dtype=torch.uint8,
                     device="cuda")
    _lib.cfc_layernorm_forward(x, w, i["b"], torch.empty_like(x), stats)

    def backward(dy, x, dx):
        dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        _lib.cfc_layernorm_backward(dy, x, w, stats, dx, dw, db, ws)
        return dx, dw, db

    want = backward(dy, x, torch.empty_like(x))
    for over in ("dy", "x"):
        a = dict(dy=dy.clone(), x=x.clone())
        got = backward(a["dy"], a["x"], a[over])
        assert all(torch.equal(g, v) for g, v in zip(got, want)), over
    want = torch.empty_like(x)
    _lib.cfc_dropout_forward(x, i["residual"], rng, 0.3, want)
    for over in ("x", "residual"):
        a = dict(x=x.clone(), residual=i["residual"].clone())
        _lib.cfc_dropout_forward(a["x"], a["residual"], rng, 0.3, a[over])
        assert torch.equal(a[over], want), over
    _lib.cfc_dropout_backward(dy, rng, 0.3, want)
    g = dy.clone()
    _lib.cfc_dropout_backward(g, rng, 0.3, g)
    assert torch.equal(g, want)


# ---- causal convolution ----

# 64 sequences of 1024 channels take, with these steps, runs of 16 steps (fp32) and 8 (bf16), of 32 and
# 16, of 64 and 32, and of 64; 1030 bf16 channels are no whole vectors and go one by one.
CONVS = [(100, 64, 1024, 4), (200, 64, 1024, 2), (400, 64, 1024, 4), (600, 64, 1024, 4),
         (600, 64, 1024, 3), (600, 64, 1030, 4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,B,D,W", CONVS)
def test_conv_runs(K, B, D, W, dtype):
    """Long runs, with sequences that end before, at and after the edges of runs and blocks."""
    from recurrent_cfc_cell_gb300 import trunk

    d = Draw(K + W, dtype)
    ends = d.lengths(B, K, 0, 1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 18, 19, 20, 31, 32, 33, 34, 35, 63,
                     64, 65, 66, 67, 68, 95, 96, 97, K, K - 1, K - 2, K - 3, K - 4)
    t = dict(x=d.normal(K, B, D), w=d.uniform(D, W, lo=-0.5, hi=0.5), bias=d.f32(D, std=0.1),
             x0=d.normal(B, W - 1, D), du=d.normal(K, B, D))
    want = p64.conv(**doubles(t), ends=ends.long())
    late = torch.arange(K, device="cuda")[:, None] >= ends
    for k in ("x", "du"):  # what lies beyond a sequence's end is not read
        t[k][late] = float("nan")
    st = trunk.ConvStep(K, B, D, W, act(dtype)).bind(t["x"], t["w"], t["bias"], t["x0"], ends,
                                                     t["du"])
    for v in (st.u, st.last, st.dx, st.dx0):
        v.fill_(float("nan"))
    st.run()
    out = st.outputs()
    assert torch.equal(out["last"].double(), want["last"])
    for k, tol in (("u", EL), ("dx", SUM), ("dx0", SUM), ("dw", SUM), ("dbias", SUM)):
        check(out[k], want[k], tol, k)


# ---- selective scan ----

GRADS = (("y", EL), ("h", EL), ("dx", EL * 10), ("ddt", SUM), ("dz", SUM), ("dA", SUM), ("dB", SUM),
         ("dC", SUM), ("dD", SUM), ("ddt_bias", SUM), ("dh0", SUM))


# Tiles of the backward pass (groups of eight channels a warp, times 16, 32 or 64 states), by the
# sizes that choose them, with channels that do not fill the last tile and odd state counts: four
# groups from 3648 warps' worth, two from 38912 steps of those, one below.
TILES = [(17, 40, 740, 16, 1), (17, 40, 752, 16, 2), (9, 40, 740, 13, 1), (16, 40, 740, 4, 1),
         (80, 8, 500, 16, 1), (80, 8, 500, 5, 2), (100, 8, 500, 8, 1),
         (17, 40, 372, 32, 1), (11, 40, 372, 24, 2), (80, 8, 252, 32, 2), (100, 8, 252, 23, 1),
         (17, 20, 364, 64, 1), (9, 20, 364, 40, 2), (90, 3, 72, 50, 1), (33, 4, 66, 128, 2)]
# Steps that both passes split over CTAs, for every number of states a tile holds.
SPLITS = [(300, 2, 40, 4, 1), (300, 3, 40, 7, 2), (333, 2, 70, 16, 1), (300, 2, 40, 24, 1),
          (300, 2, 36, 32, 2), (280, 2, 40, 64, 1), (300, 2, 40, 100, 1), (300, 1, 33, 128, 1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,B,D,N,G", TILES + SPLITS)
def test_scan_tiles_and_splits(K, B, D, N, G, dtype):
    from recurrent_cfc_cell_gb300 import trunk

    i = scan_inputs(K, B, D, N, G, dtype, K + N)
    ends = Draw(3).lengths(B, K, K, K - 5, 0, K // 2, 1)
    want = p64.scan(doubles(i), ends.long())
    late = torch.arange(K, device="cuda")[:, None] >= ends
    for k in ("x", "dt", "z", "dy", "Bm", "Cm"):
        i[k][late] = float("nan")
    st = trunk.ScanStep(K, B, D, N, G, act(dtype), train=True)
    for v in vars(st).values():
        if hasattr(v, "fill_") and v.is_floating_point():
            v.fill_(float("nan"))
    i["D"] = i.pop("skip")
    st.bind(**i, lengths=ends).run()
    out = st.outputs()
    for k, tol in GRADS:
        check(out[k], want[k], tol, k)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,D,N,G", [(530, 600, 64, 1), (4901, 1000, 4, 2), (1231, 1000, 16, 4),
                                     (2437, 1000, 5, 1), (300, 1000, 128, 1)])
def test_scan_tokens_of_many_sequences(B, D, N, G, dtype):
    """So many that a CTA takes sixteen sequences, the last one fewer; the state in place."""
    from recurrent_cfc_cell_gb300 import trunk

    i = scan_inputs(1, B, D, N, G, dtype, N)
    want = p64.scan(doubles(i), torch.ones(B, dtype=torch.int64, device="cuda"), backward=False)
    new = torch.full_like(i["h0"], float("nan"))
    t = {k: i[k][0] for k in ("x", "dt", "z", "Bm", "Cm")}
    t.update(A=i["A"], D=i["skip"], dt_bias=i["dt_bias"], state=i["h0"])
    tok = trunk.ScanToken(B, D, N, G, act(dtype))
    y = tok.bind(**t, new_state=new).run()[0].clone()
    check(y, want["y"][0], EL, "y")
    check(new, want["h"], EL, "h")
    again, state = tok.bind(**t).run()
    assert torch.equal(again, y) and torch.equal(state, new) and state is i["h0"]


# ---- strides past 32 bits ----

def far(t, stride, buf, at):
    """t [R, ..] with its first dimension `stride` elements apart in `buf` from element `at` on."""
    v = buf.as_strided(t.shape, (stride, *t.stride()[1:]), at)
    v.copy_(t)
    return v


def test_strides_past_32_bits():
    """Rows and sequences 2^30 and more elements apart, three of them."""
    from recurrent_cfc_cell_gb300 import _lib

    stride = (1 << 30) + 24
    buf = torch.empty(2 * stride + (1 << 22), dtype=torch.bfloat16, device="cuda")
    put = lambda t, slot: far(t, stride, buf, slot << 18)  # noqa: E731
    i = norm_inputs(3, 200, "bf16", 1)
    slots = iter(range(16))
    norm_checks(i, norm_calls(i, lambda name, t: put(t, next(slots))))

    K, B, D, N, W = 20, 3, 40, 16, 4
    ends = torch.full((B,), K, device="cuda")

    def first(t, slot):  # batch-first memory of a [K, B, ..] tensor
        return put(t.transpose(0, 1).contiguous(), slot).transpose(0, 1)

    d = Draw(2, "bf16")
    t = dict(x=d.normal(K, B, D), w=d.uniform(D, W, lo=-0.5, hi=0.5), bias=d.f32(D, std=0.1),
             x0=d.normal(B, W - 1, D), du=d.normal(K, B, D))
    want = p64.conv(**doubles(t), ends=ends)
    x, du = first(t["x"], 0), first(t["du"], 1)
    u, dx = first(torch.zeros_like(t["x"]), 2), first(torch.zeros_like(t["x"]), 3)
    dw, db = torch.empty(D, W, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(_lib.conv_workspace_bytes(B, K, D, W, _lib.CFC_BF16), dtype=torch.uint8,
                     device="cuda")
    _lib.cfc_conv_forward(x, t["w"], u, t["bias"], t["x0"])
    _lib.cfc_conv_backward(du, x, t["w"], dx, dw, db, t["bias"], t["x0"], ws=ws)
    for got, k, tol in ((u, "u", EL), (dx, "dx", SUM), (dw, "dw", SUM), (db, "dbias", SUM)):
        check(got, want[k], tol, k)

    i = scan_inputs(K, B, D, N, 1, "bf16", 4)
    want = p64.scan(doubles(i), ends)
    v = {k: first(i[k], n) for n, k in enumerate(("x", "dt", "z", "dy"))}
    v.update({k: first(i[k], 4 + n) for n, k in enumerate(("Bm", "Cm"))})
    o = {k: first(torch.zeros_like(i["x"]), 6 + n) for n, k in enumerate(("y", "dx", "ddt", "dz"))}
    f = {k: torch.empty_like(i[k[1:]] if k != "h" else i["h0"]) for k in ("dA", "dh0", "h")}
    f.update(dB=torch.empty_like(i["Bm"]), dC=torch.empty_like(i["Cm"]))
    opt = dict(D=i["skip"], dt_bias=i["dt_bias"], z=v["z"], h0=i["h0"])
    states = torch.empty(-(-K // _lib.SCAN_PERIOD), B, D, N, device="cuda")
    ws = torch.empty(max(_lib.scan_workspace_bytes(K, B, D, N, 1, _lib.CFC_BF16, True), 16),
                     dtype=torch.uint8, device="cuda")
    ins = (v["x"], v["dt"], i["A"], v["Bm"], v["Cm"])
    _lib.cfc_scan_forward(*ins, o["y"], h_last=f["h"], states=states, **opt)
    _lib.cfc_scan_backward(v["dy"], *ins, states, o["dx"], o["ddt"], f["dA"], f["dB"], f["dC"],
                           dz=o["dz"], dh0=f["dh0"], dh_last=i["dh_last"], ws=ws, **opt)
    for k, tol in GRADS:
        if k in {**o, **f}:
            check({**o, **f}[k], want[k], tol, k)
