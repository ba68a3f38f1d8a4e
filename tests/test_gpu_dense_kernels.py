"""Every kernel of the dense matrix operators (dense_cases.py): whole numbers
whose sums float32 holds exactly, so that every output is compared bit for bit;
ordinary float32 numbers against float64; the same bits under shuffled launches
and poisoned memory, on two streams and in a graph.  And the layer norm's row
widths and rounds that the other tests leave out."""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import dense_bounds as B
from dense_cases import CASES
from test_gpu_dense import _all_calls, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _exact(a, b):
    """a b in float64, and that every sum and partial sum of it stays below 2^24."""
    assert float((a.abs() @ b.abs()).max()) < 2 ** 24
    return a @ b


def _same(got, want, what):
    """want: float64 whole numbers that float32 holds, so that one rounding gives got."""
    want = want.float().to(got.dtype)
    bad = got != want
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


# the widest and the longest matrices: offsets of a tile's rows near 2^30 bytes, many
# tiles and chunks
FAR = [(t, *s) for t in ("bf16", "f32") for s in ((70, 16, 1000003), (70, 1000003, 16), (5, 1048575, 24), (3, 24, 1048575),
                                                  (300, 1048568, 8), (2000003, 8, 5), (600000, 72, 130))]


@pytest.mark.parametrize("dtype,rows,d,f", CASES + FAR)
def test_whole_numbers(dtype, rows, d, f):
    T = B.TORCH[dtype]
    g = torch.Generator(device=DEV).manual_seed(rows + d + f)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV).double()  # noqa: E731
    x, w, w2, b, r, dy, add = ints(rows, d), ints(d, f), ints(d, f), ints(f), ints(rows, f), ints(rows, f), ints(rows, d)
    t = lambda a: a.to(T)  # noqa: E731
    z = _exact(x, w) + b
    y, zs = moe.moe_linear_fwd(t(x), t(w), t(b), t(r), "relu", save_z=True)
    _same(zs, z, "z")
    _same(y, z.clamp_min(0) + r, "y")
    # dz is 0 or dy: no rounding
    dz = dy * (z > 0)
    dx, dw, db = moe.moe_linear_bwd(t(dy), t(x), t(w), zs, "relu", dx_add=t(add))
    _same(dx, _exact(dz, w.t()) + add, "dx")
    _same(dw, _exact(x.t(), dz), "dw")
    _same(db, dz.sum(0), "db")
    gate, up = _exact(x, w), _exact(x, w2)
    a, gs, us = moe.moe_glu_fwd(t(x), t(w), t(w2), "relu", save=True)
    _same(gs, gate, "g")
    _same(us, up, "u")
    _same(a, (gate.clamp_min(0).float() * up.float()).double(), "a")   # one rounding of the float32 product
    # small saved values, so that dg and du are small whole numbers
    gate, up = ints(rows, f), ints(rows, f)
    dg, du = dy * up * (gate > 0), dy * gate.clamp_min(0)
    dx, dwg, dwu = moe.moe_glu_bwd(t(dy), t(x), t(w), t(w2), gate.float(), up.float(), "relu", dx_add=t(add), grad_dtype=T)
    _same(dx, _exact(torch.cat([dg, du], 1), torch.cat([w, w2], 1).t()) + add, "dx of the gated product")
    _same(dwg, _exact(x.t(), dg), "dwg")
    _same(dwu, _exact(x.t(), du), "dwu")


@pytest.mark.parametrize("dtype,rows,d,f", [c for c in CASES if c[0] == "f32"])
def test_float32_numbers(dtype, rows, d, f):
    """All 24 bits of ordinary numbers: (2 n + 10) 2^-24 of the products'
    magnitudes (dense_bounds.py), and one rounding."""
    t = _inputs(rows, d, f, torch.float32, seed=f)
    D = {n: v.double() for n, v in t.items()}

    def check(got, a, b, what):
        ref, tol = a @ b, (2 * a.shape[1] + 10) * B.E * (a.abs() @ b.abs())
        bad = ~((got.double() - ref).abs() <= tol + B.E * (ref.abs() + tol))
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off"

    check(moe.moe_linear_fwd(t["x"], t["w"])[0], D["x"], D["w"], "y")
    dx, dw, _ = moe.moe_linear_bwd(t["dy"], t["x"], t["w"], need_db=False)
    check(dx, D["dy"], D["w"].t(), "dx")
    check(dw, D["x"].t(), D["dy"], "dw")
    _, g, u = moe.moe_glu_fwd(t["x"], t["w"], t["w2"], "none", save=True)
    check(g, D["x"], D["w"], "g")
    check(u, D["x"], D["w2"], "u")
    one = torch.ones_like(t["dy"])
    dx, dwg, dwu = moe.moe_glu_bwd(t["dy"], t["x"], t["w"], t["w2"], one, one, "none")
    check(dx, torch.cat([D["dy"], D["dy"]], 1), torch.cat([D["w"], D["w2"]], 1).t(), "dx of the gated product")
    check(dwg, D["x"].t(), D["dy"], "dwg")
    assert torch.equal(dwg, dwu)


@pytest.mark.parametrize("dtype,rows,d,f", CASES)
def test_bits_do_not_depend_on_order_or_old_memory(dtype, rows, d, f):
    t = _inputs(rows, d, f, B.TORCH[dtype])
    ref = _all_calls(t, 0, 0.0)
    for seed, poison in ((0, float("nan")), (0x5EED, float("nan")), (2 ** 63 + 11, 1.0)):
        for i, (a, b) in enumerate(zip(ref, _all_calls(t, seed, poison))):
            assert torch.equal(a, b), (i, seed)


@pytest.mark.parametrize("pair", [(("bf16", 8602, 5720, 136), ("bf16", 277, 1168, 7936)), (("f32", 725, 480, 4192), ("f32", 212, 706, 4649))])
def test_large_tiles_on_two_streams_and_in_graphs(pair):
    ts = [_inputs(*c[1:], B.TORCH[c[0]], seed=i) for i, c in enumerate(pair)]
    ref = [_all_calls(t, 0, 0.0) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(2):
        got = []
        for st, t in zip(streams, ts):
            with torch.cuda.stream(st):
                got.append(_all_calls(t, 0, float("nan")))
        torch.cuda.synchronize()
        for g, r in zip(got, ref):
            for i, (a, b) in enumerate(zip(g, r)):
                assert torch.equal(a, b), i
        del got
    graphs = []
    for t in ts:
        graph = torch.cuda.CUDAGraph()
        n, f = t["x"].shape[0], t["w"].shape[1]
        gu = [torch.empty((n, f), dtype=t["x"].dtype, device=DEV) for _ in range(2)]
        with torch.cuda.graph(graph, stream=streams[0]):
            y, z = moe.moe_linear_fwd(t["x"], t["w"], t["b"], t["dy"], "gelu", save_z=True)
            out = [y, z, *moe.moe_linear_bwd(t["dy"], t["x"], t["w"], z, "gelu")]
            out += moe.moe_glu_fwd(t["x"], t["w"], t["w2"], g=gu[0], u=gu[1])
            out += moe.moe_glu_bwd(t["dy"], t["x"], t["w"], t["w2"], *gu)
        graphs.append((graph, out))
    for i in range(3):
        for _, out in graphs:
            for o in out:
                o.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, out), r in zip(graphs, ref):
            for j, (a, b) in enumerate(zip(out, r[6:])):   # after the layer norm's six
                assert torch.equal(a, b), (i, j)
        _all_calls(ts[i % 2], 0x5EED, 1.0)   # eager work between the replays
        torch.cuda.synchronize()


# ------------------------------------------------------------------ layer norm
# more rows than the launch holds at a time (2048 workgroups of 256 threads, 512 of
# 1024; the backward's blocks of several rows), and widths between 1024 and 2048
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(9001, 40), (9000, 512), (8300, 1030), (2200, 1500), (2300, 2048), (2100, 2051), (2065, 4096),
                                       (1100, 4100), (1061, 8192), (700, 8300), (530, 16384), (2051, 1999)])
def test_layernorm_rounds(dtype, rows, cols):
    rng = np.random.default_rng(rows + cols)
    scale = np.exp(rng.standard_normal((rows, 1)))
    x, hx = B.values(rng, (rows, cols), dtype, scale, 0.3)
    dy, hdy = B.values(rng, (rows, cols), dtype)
    w, hw = B.values(rng, (cols,), dtype, 0.2, 1.0)
    b, hb = B.values(rng, (cols,), dtype, 0.1)
    x, dy, w, b = (t.to(DEV) for t in (x, dy, w, b))
    y, mean, rstd = moe.moe_layernorm_fwd(x, w, b)
    ref, tol = B.norm_bounds(dtype, hx, hw, hb, 1e-5)
    B.check(y, ref, tol, "y")
    out = moe.moe_layernorm_bwd(dy, x, w, mean, rstd, dx_add=dy)
    refs, tols = B.norm_bwd_bounds(dtype, hdy, hx, hw, 1e-5, hdy)
    for n, g, r, t in zip(("dx", "dweight", "dbias"), out, refs, tols):
        B.check(g, r, t, n)
    for seed in (0x5EED, 2 ** 63 + 11):
        nan = torch.full_like(x, float("nan"))
        y2, m2, r2 = moe.moe_layernorm_fwd(x, w, b, y=nan, shuffle_seed=seed)
        assert torch.equal(y2, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)
        for p, q in zip(out, moe.moe_layernorm_bwd(dy, x, w, mean, rstd, dx_add=dy, shuffle_seed=seed)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3000001, 3), (140000, 16384)])
def test_layernorm_of_many_rows(dtype, rows, cols):
    """More than 2^31 elements, and very short rows: the first, some middle and the
    last rows, and the sums over all rows of a constant gradient."""
    T = B.TORCH[dtype]
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = torch.empty(rows, cols, dtype=T, device=DEV)
    for i in range(0, rows, 20000):
        x[i:i + 20000] = torch.randn(min(20000, rows - i), cols, generator=g, device=DEV).to(T)
    y, mean, rstd = moe.moe_layernorm_fwd(x)
    at = torch.cat([torch.arange(40), torch.arange(40) + rows // 2 + 11, torch.arange(40) + rows - 40]).to(DEV)
    hx = B.host(x[at])
    ref, tol = B.norm_bounds(dtype, hx, None, None, 1e-5)
    B.check(y[at], ref, tol, "y")
    dx, dw, db = moe.moe_layernorm_bwd(y, x, None, mean, rstd)
    hdy = B.host(y[at])
    refs, tols = B.norm_bwd_bounds(dtype, hdy, hx, None, 1e-5, None)
    B.check(dx[at], refs[0], tols[0], "dx")
    want, mag = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    wantw, magw = torch.zeros_like(want), torch.zeros_like(want)
    for i in range(0, rows, 20000):
        d = y[i:i + 20000].double()
        h = (x[i:i + 20000].double() - mean[i:i + 20000, None].double()) * rstd[i:i + 20000, None].double()
        want += d.sum(0)
        mag += d.abs().sum(0)
        wantw += (d * h).sum(0)
        magw += (d * h).abs().sum(0)
    # h in float32 is off by 3 roundings, each sum by at most one of 2^-24 a row
    assert bool(((db.double() - want).abs() <= (rows + 10) * B.E * mag).all())
    assert bool(((dw.double() - wantw).abs() <= (rows + 14) * B.E * magw + 4 * B.E * magw).all())
