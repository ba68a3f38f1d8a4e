"""The dense operators (layer norm, linear map, gated product) on the GPU
against the float64 oracle, element by element within the bounds of
dense_bounds.py, over types, sizes from one row on, odd sizes, row strides,
activations, saved types and splits; what they leave untouched; bit
identity under shuffled launches and poisoned memory; streams and graphs;
and a block of them together with the expert layer."""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import dense_bounds as B
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _strided(t, pad):
    """t's values on the device, rows `pad` elements further apart, the gaps NaN."""
    if t is None:
        return None
    if pad == 0:
        return t.to(DEV)
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    buf[:, : t.shape[1]] = t.to(DEV)
    return buf[:, : t.shape[1]]


# ------------------------------------------------------------------ layer norm
NORM = [(0, 64), (1, 1), (1, 2048), (2, 7), (5, 1001), (33, 512), (37, 520), (130, 1024), (600, 2048), (9, 2050),
        (3, 4096), (7, 4097), (5, 8192), (2, 8200), (3, 16384), (2500, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", NORM)
def test_layernorm(dtype, rows, cols):
    rng = np.random.default_rng(rows * 20011 + cols)
    pad = [0, 0, 3, 8][(rows + cols) % 4]
    scale = np.exp(rng.standard_normal((rows, 1)))
    x, hx = B.values(rng, (rows, cols), dtype, scale, 0.3)
    dy, hdy = B.values(rng, (rows, cols), dtype)
    w, hw = B.values(rng, (cols,), dtype, 0.2, 1.0) if cols % 2 else (None, None)
    if cols % 2 == 0 and cols != 512:
        w, hw = B.values(rng, (cols,), dtype, 0.2, 1.0)
    b, hb = B.values(rng, (cols,), dtype, 0.1) if cols != 2050 else (None, None)
    add, hadd = B.values(rng, (rows, cols), dtype) if rows % 2 else (None, None)
    up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    dx_in = _strided(x, pad)
    y, mean, rstd = moe.moe_layernorm_fwd(dx_in, up(w), up(b), EPS)
    dx, dw, db = moe.moe_layernorm_bwd(_strided(dy, pad), dx_in, up(w), mean, rstd, dx_add=_strided(add, pad))
    if rows == 0:
        assert y.shape == (0, cols) and dx.shape == (0, cols) and not dw.any() and not db.any()
        return
    ref, tol = B.norm_bounds(dtype, hx, hw, hb, EPS)
    B.check(y, ref, tol, "y")
    refs, tols = B.norm_bwd_bounds(dtype, hdy, hx, hw, EPS, hadd)
    for n, g, r, t in zip(("dx", "dweight", "dbias"), (dx, dw, db), refs, tols):
        B.check(g, r, t, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm_far_from_zero_and_constant_rows(dtype):
    # a mean a thousand times the spread, and rows of one value (variance 0)
    rng = np.random.default_rng(5)
    x, hx = B.values(rng, (16, 768), dtype, 1.0, 1000.0)
    x[8:] = 3.0
    hx[8:] = 3.0
    y, mean, rstd = moe.moe_layernorm_fwd(x.to(DEV), None, None, EPS)
    ref, tol = B.norm_bounds(dtype, hx, None, None, EPS)
    B.check(y, ref, tol, "y")
    assert torch.equal(y[8:].cpu(), torch.zeros_like(x[8:]))


def test_layernorm_nan_and_inf_stay_in_their_rows():
    x = torch.randn(6, 300, device=DEV)
    x[1, 7] = float("nan")
    x[4, 299] = float("inf")
    clean = moe.moe_layernorm_fwd(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))[0]
    y = moe.moe_layernorm_fwd(x)[0]
    bad = torch.isnan(y).any(1)
    assert bad.tolist() == [False, True, False, False, True, False]
    assert torch.equal(y[~bad], clean[~bad])


# ---------------------------------------------------------------------- linear
# (rows, d_in, d_out): one row, few rows, their border (16, 64), tiles, odd
# sizes, more columns than a tile, long contractions that split, sizes of one
LINEAR = [(1, 256, 512), (1, 1000, 130), (3, 33, 5), (16, 96, 64), (17, 264, 200), (33, 512, 264), (64, 128, 136),
          (65, 130, 72), (2, 1, 1), (70, 1, 3), (100, 72, 1), (129, 520, 264), (257, 256, 520), (300, 1001, 517),
          (512, 2048, 256), (70, 2056, 300), (1030, 64, 96)]


def _linear_case(dtype, rows, d, f, act, bias, residual, pad, zdtype, gdtype, ints=False, seed=0):
    rng = np.random.default_rng(rows * 1000003 + d * 1009 + f + seed)
    make = B.small_ints if ints else B.values
    x, hx = make(rng, (rows, d), dtype)
    w, hw = make(rng, (d, f), dtype) if ints else B.values(rng, (d, f), dtype, d ** -0.5)
    b, hb = (make(rng, (f,), dtype) if ints else B.values(rng, (f,), dtype, 0.3)) if bias else (None, None)
    r, hr = make(rng, (rows, f), dtype) if residual else (None, None)
    dy, hdy = make(rng, (rows, f), dtype)
    add, hadd = B.values(rng, (rows, d), dtype) if residual else (None, None)
    dx_, dw_, db_ = _strided(x, pad), _strided(w, pad), None if b is None else b.to(DEV)
    z = None
    if act != "none":
        z = torch.full((rows, f + pad), float("nan"), dtype=B.TORCH[zdtype], device=DEV)[:, :f]
    yb = torch.full((rows + 2, f + pad), 7.0, dtype=B.TORCH[dtype], device=DEV)
    y, z2 = moe.moe_linear_fwd(dx_, dw_, db_, _strided(r, pad), act, y=yb[:rows, :f], z=z)
    assert z2 is z
    ref, hz, tol, ez = B.linear_bounds(dtype, hx, hw, hb, hr, act)
    B.check(y, ref, tol, "y")
    assert bool((yb[rows:] == 7).all()) and bool((yb[:, f:] == 7).all()), "rows or columns past y were written"
    if z is not None:
        ez = B.rounded(ez, hz, B.U[zdtype] if not ints else 0.0)
        B.check(z, hz, ez, "z")
    dx, dw, db = moe.moe_linear_bwd(_strided(dy, pad), dx_, dw_, z, act, dx_add=_strided(add, pad), need_db=bias,
                                    grad_dtype=B.TORCH[gdtype])
    refs, tols = B.linear_bwd_bounds(dtype, gdtype, hdy, hx, hw, hz, 0 * ez if ints else ez, act, hadd)
    B.check(dx, refs[0], tols[0], "dx")
    B.check(dw, refs[1], tols[1], "dw")
    assert dw.dtype == B.TORCH[gdtype]
    if bias:
        B.check(db, refs[2], tols[2], "db")
    else:
        assert db is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,f", LINEAR)
def test_linear(dtype, rows, d, f):
    act = ["none", "silu", "gelu", "relu2"][(rows + f) % 4]
    _linear_case(dtype, rows, d, f, act, bias=rows % 3 != 0, residual=f % 3 != 0, pad=[0, 8, 5][(rows + d) % 3],
                 zdtype=dtype if d % 2 else "f32", gdtype="f32" if rows % 2 else dtype)


# few rows and few columns: the rows of the weights are split between workgroups
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,f", [(1, 16384, 72), (5, 8200, 264), (12, 4100, 130), (48, 6001, 40), (64, 4099, 72),
                                      (29, 4100, 136)])
def test_few_rows_in_chunks(dtype, rows, d, f):
    _linear_case(dtype, rows, d, f, "silu", True, True, 8 if f % 8 == 0 else 3, "f32", "f32")
    test_glu(dtype, rows, d, f)


@pytest.mark.parametrize("act", list(moe.ACTIVATIONS))
@pytest.mark.parametrize("rows", [5, 130])
def test_linear_activations(act, rows):
    # ReLU on small whole numbers, whose z is exact and often 0
    _linear_case("bf16", rows, 96, 136, act, True, True, 0, "f32", "bf16", ints=act == "relu", seed=1)
    _linear_case("f32", rows, 96, 136, act, True, True, 4, "f32", "f32", ints=act == "relu", seed=2)


@pytest.mark.parametrize("zero", ["rows"])
def test_linear_zero_rows(zero):
    x, w = torch.empty(0, 24, device=DEV), torch.randn(24, 10, device=DEV)
    y, z = moe.moe_linear_fwd(x, w, act="gelu", save_z=True)
    assert y.shape == (0, 10) and z.shape == (0, 10)
    dx, dw, db = moe.moe_linear_bwd(y, x, w, z, "gelu")
    assert dx.shape == (0, 24) and dw.shape == (24, 10) and not dw.any() and not db.any()
    a, g, u = moe.moe_glu_fwd(x, w, w.clone(), save=True)
    dx, dwg, dwu = moe.moe_glu_bwd(a, x, w, w.clone(), g, u)
    assert dx.shape == (0, 24) and not dwg.any() and not dwu.any()


# ----------------------------------------------------------------------- gated
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,f", LINEAR)
def test_glu(dtype, rows, d, f):
    act = ["silu", "gelu", "none", "relu2"][(rows + d) % 4]
    rng = np.random.default_rng(rows * 7919 + d * 31 + f)
    pad = [0, 8, 5][(rows + f) % 3]
    x, hx = B.values(rng, (rows, d), dtype)
    wg, hg = B.values(rng, (d, f), dtype, d ** -0.5)
    wu, hu = B.values(rng, (d, f), dtype, d ** -0.5)
    da, hda = B.values(rng, (rows, f), dtype)
    add, hadd = B.values(rng, (rows, d), dtype) if d % 2 == 0 else (None, None)
    zdt = dtype if f % 2 else "f32"
    gdt = "f32" if rows % 2 else dtype
    xd = _strided(x, pad)
    if f % 8 == 0:   # the halves of one matrix
        both = torch.cat([wg, wu], 1).to(DEV)
        wgd, wud = both[:, :f], both[:, f:]
    else:
        wgd, wud = _strided(wg, pad), _strided(wu, pad)
    g, u = (torch.full((rows, f + pad), float("nan"), dtype=B.TORCH[zdt], device=DEV)[:, :f] for _ in range(2))
    ab = torch.full((rows + 2, f + pad), 7.0, dtype=B.TORCH[dtype], device=DEV)
    a, g2, u2 = moe.moe_glu_fwd(xd, wgd, wud, act, a=ab[:rows, :f], g=g, u=u)
    assert g2 is g and u2 is u
    ref, rg, ru, tol, eg, eu = B.glu_bounds(dtype, hx, hg, hu, act)
    B.check(a, ref, tol, "a")
    assert bool((ab[rows:] == 7).all()) and bool((ab[:, f:] == 7).all()), "rows or columns past a were written"
    eg, eu = B.rounded(eg, rg, B.U[zdt]), B.rounded(eu, ru, B.U[zdt])
    B.check(g, rg, eg, "g")
    B.check(u, ru, eu, "u")
    dx, dwg, dwu = moe.moe_glu_bwd(_strided(da, pad), xd, wgd, wud, g, u, act, dx_add=_strided(add, pad),
                                   grad_dtype=B.TORCH[gdt])
    refs, tols = B.glu_bwd_bounds(dtype, gdt, hda, hx, hg, hu, rg, ru, eg, eu, act, hadd)
    for n, got, r, t in zip(("dx", "dwg", "dwu"), (dx, dwg, dwu), refs, tols):
        B.check(got, r, t, n)


def test_inference_call_matches_the_saving_one():
    x, wg, wu = (torch.randn(s, device=DEV).bfloat16() for s in ((200, 256), (256, 320), (256, 320)))
    a, g, u = moe.moe_glu_fwd(x, wg, wu)
    assert g is None and u is None
    assert torch.equal(a, moe.moe_glu_fwd(x, wg, wu, save=True)[0])
    y, z = moe.moe_linear_fwd(x, wg, act="gelu")
    assert z is None
    assert torch.equal(y, moe.moe_linear_fwd(x, wg, act="gelu", save_z=True)[0])


def test_leading_dimensions_and_one_vector():
    x, w = torch.randn(2, 3, 40, device=DEV), torch.randn(40, 24, device=DEV)
    y, _ = moe.moe_linear_fwd(x, w)
    assert y.shape == (2, 3, 24)
    assert torch.equal(y.reshape(6, 24), moe.moe_linear_fwd(x.reshape(6, 40), w)[0])
    v, _ = moe.moe_linear_fwd(x[0, 0], w)
    assert v.shape == (24,) and torch.equal(v, moe.moe_linear_fwd(x[0, :1], w)[0][0])
    n, mean, _ = moe.moe_layernorm_fwd(x)
    assert n.shape == x.shape and mean.shape == (2, 3)
    dx, dw, db = moe.moe_linear_bwd(y, x, w)
    assert dx.shape == x.shape and dw.shape == w.shape and db.shape == (24,)


@pytest.mark.parametrize("rows", [3, 300])
def test_residual_and_gradient_in_place(rows):
    x, w, r = (torch.randn(s, device=DEV).bfloat16() for s in ((rows, 264), (264, 136), (rows, 136)))
    want, _ = moe.moe_linear_fwd(x, w, residual=r)
    y = r.clone()
    moe.moe_linear_fwd(x, w, residual=y, y=y)
    assert torch.equal(y, want)
    add = torch.randn(rows, 264, device=DEV).bfloat16()
    want = moe.moe_linear_bwd(r, x, w, dx_add=add)[0]
    dx = add.clone()
    moe.moe_linear_bwd(r, x, w, dx_add=dx, dx=dx)
    assert torch.equal(dx, want)


@pytest.mark.parametrize("rows", [4, 40, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_inf_stay_in_their_rows(rows, dtype):
    # 200 columns end inside a tile and 70 inputs inside a slice: what lies
    # past them must not turn into NaN, and a NaN row must not leave its row
    torch.manual_seed(1)
    x, w = torch.randn(rows, 70, device=DEV).to(dtype), torch.randn(70, 200, device=DEV).to(dtype)
    want, _ = moe.moe_linear_fwd(x, w)
    assert torch.isfinite(want).all()
    x2 = x.clone()
    x2[1, 69] = float("nan")
    x2[3, 0] = float("inf")
    got, _ = moe.moe_linear_fwd(x2, w)
    ok = torch.tensor([i not in (1, 3) for i in range(rows)], device=DEV)
    assert torch.equal(got[ok], want[ok])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[3]).any()
    w2 = w.clone()
    w2[69, 199] = float("inf")
    got, _ = moe.moe_linear_fwd(x, w2)
    assert torch.equal(got[:, :199], want[:, :199]) and not torch.isfinite(got[:, 199]).any()


# products for each of the bf16 tiles, whole and ragged, split and unsplit, of one
# or two slices
@pytest.mark.parametrize("rows,d,f", [(1030, 1032, 1040), (2000, 2056, 2049), (2049, 512, 2320), (1100, 2048, 4360),
                                      (130, 4104, 264), (50, 1032, 2056), (128, 1001, 600),
                                      (3000, 128, 264), (2000, 72, 1000)])
def test_bf16_tiles(rows, d, f):
    _linear_case("bf16", rows, d, f, "gelu", True, True, 8 if f % 8 == 0 else 0, "f32", "bf16")
    test_glu("bf16", rows, d, f)


# ------------------------------------------------ float32 products in three parts
@pytest.mark.parametrize("rows,d,f", [(2050, 1031, 2047), (1900, 1540, 2052), (4100, 2049, 260)])
@pytest.mark.parametrize("gated", [False, True])
def test_large_float32_products(rows, d, f, gated):
    if gated:
        test_glu("f32", rows, d, f)
    else:
        _linear_case("f32", rows, d, f, "gelu", True, True, 3 if d % 2 else 0, "f32", "f32")


@pytest.mark.parametrize("n,d,f", [(2048, 512, 2048), (2051, 515, 2047)])
def test_large_float32_products_at_the_ends_of_the_range(n, d, f):
    """Infinite, NaN, near-largest and very small numbers give what float32
    products of them give: each in its row, the finite ones within the bound."""
    rng = np.random.default_rng(n)
    x, w = (rng.standard_normal(s).astype(np.float32) for s in ((n, d), (d, f)))
    top = np.finfo(np.float32).max
    x[5] *= 2.0 ** -130                      # denormal
    x[700] *= 2.0 ** -112
    x[900] = 0
    x[1000, 3] = top                         # above the largest bf16; its row stays finite:
    w[3] *= 2.0 ** -10                       # |w| < 0.01
    x[1, d - 1] = np.nan
    x[300, 0] = np.inf
    xd, wd = torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV)
    y, _ = moe.moe_linear_fwd(xd, wd)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[300]).any()
    assert torch.equal(y[300].sign(), wd[0].sign())
    assert not y[900].any()
    rows = np.array([i for i in range(n) if i not in (1, 300)])
    x64, w64 = x[rows].astype(np.float64), w.astype(np.float64)
    # a number below 2^-126 is kept to 2^-150, and so is each sum
    def tol(a, b):
        return B.rounded(B.prod_err(a.shape[1], np.abs(a), np.abs(b)) + a.shape[1] * 2.0 ** -147, a @ b, B.U["f32"])
    B.check(y[torch.from_numpy(rows).to(DEV)], x64 @ w64, tol(x64, w64), "y")
    # a gradient that is small throughout
    dy = (rng.standard_normal((n, f)) * 2.0 ** -120).astype(np.float32)
    x[[1, 300, 1000]] = 1
    xd = torch.from_numpy(x).to(DEV)
    dx, dw, _ = moe.moe_linear_bwd(torch.from_numpy(dy).to(DEV), xd, wd, need_db=False)
    a, x64 = dy.astype(np.float64), x.astype(np.float64)
    B.check(dx, a @ w64.T, tol(a, w64.T), "dx")
    B.check(dw, x64.T @ a, tol(x64.T, a), "dw")
    da = torch.from_numpy(x[:, :1] * np.ones((1, f), np.float32)).to(DEV)
    da[7, 9] = float("nan")
    wu = torch.from_numpy(rng.standard_normal((d, f)).astype(np.float32)).to(DEV)
    a, g, u = moe.moe_glu_fwd(xd, wd, wu, "relu", save=True)
    xn = xd.clone()
    xn[2, 2] = float("-inf")
    an = moe.moe_glu_fwd(xn, wd, wu, "none")[0]
    assert not torch.isfinite(an[2]).any()
    keep = torch.arange(n, device=DEV) != 2
    assert torch.equal(an[keep], moe.moe_glu_fwd(xd, wd, wu, "none")[0][keep])
    want = moe.moe_glu_bwd(da.nan_to_num(0.5), xd, wd, wu, g, u, "relu")
    got = moe.moe_glu_bwd(da, xd, wd, wu, g, u, "relu")
    keep = torch.arange(n, device=DEV) != 7
    assert torch.isnan(got[0][7]).all() and torch.equal(got[0][keep], want[0][keep])
    cols = torch.arange(f, device=DEV) != 9
    for i in (1, 2):
        assert torch.isnan(got[i][:, 9]).all() and torch.equal(got[i][:, cols], want[i][:, cols])


# --------------------------------------------------------- order and workspaces
def _all_calls(t, seed, poison):
    """Every call on the inputs t, with given workspaces and outputs filled
    with `poison` before the call.  Returns the outputs."""
    n, d = t["x"].shape
    f = t["w"].shape[1]
    dt = t["x"].dtype
    name = {torch.bfloat16: "bf16", torch.float32: "f32"}[dt]
    E = lambda *s, dtype=dt: torch.full(s, poison, dtype=dtype, device=DEV)  # noqa: E731
    W = lambda k: torch.full((max(k, 1),), 0xFF if poison != poison else 0x55, dtype=torch.uint8, device=DEV)  # noqa: E731
    lw = moe.moe_linear_workspace_size(n, d, f, name, "gelu")
    gw = moe.moe_glu_workspace_size(n, d, f, name)
    f32 = torch.float32
    y, mean, rstd = moe.moe_layernorm_fwd(t["x"], t["nw"], t["nb"], EPS, y=E(n, d), mean=E(n, dtype=f32),
                                          rstd=E(n, dtype=f32), shuffle_seed=seed)
    out = [y, mean, rstd]
    out += moe.moe_layernorm_bwd(t["dx"], t["x"], t["nw"], mean, rstd, dx=E(n, d), dweight=E(d, dtype=f32),
                                 dbias=E(d, dtype=f32), ws=W(moe.moe_layernorm_workspace_size(n, d)), shuffle_seed=seed)
    y, z = moe.moe_linear_fwd(t["x"], t["w"], t["b"], t["dy"], "gelu", y=E(n, f), z=E(n, f, dtype=f32), ws=W(lw[0]),
                              shuffle_seed=seed)
    out += [y, z]
    out += moe.moe_linear_bwd(t["dy"], t["x"], t["w"], z, "gelu", dx=E(n, d), dw=E(d, f, dtype=f32), db=E(f, dtype=f32),
                              ws=W(lw[1]), shuffle_seed=seed)
    a, g, u = moe.moe_glu_fwd(t["x"], t["w"], t["w2"], a=E(n, f), g=E(n, f), u=E(n, f), ws=W(gw[0]), shuffle_seed=seed)
    out += [a, g, u]
    out += moe.moe_glu_bwd(t["dy"], t["x"], t["w"], t["w2"], g, u, dx=E(n, d), dwg=E(d, f, dtype=f32),
                           dwu=E(d, f, dtype=f32), ws=W(gw[1]), shuffle_seed=seed)
    return out


def _inputs(n, d, f, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    return dict(x=r(n, d), w=r(d, f) * d ** -0.5, w2=r(d, f) * d ** -0.5, b=r(f), dy=r(n, f), dx=r(n, d), nw=r(d), nb=r(d))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d,f", [(7, 1024, 520), (333, 1032, 264), (1500, 256, 768)])
def test_bits_do_not_depend_on_order_or_old_memory(dtype, n, d, f):
    t = _inputs(n, d, f, dtype)
    ref = _all_calls(t, 0, 0.0)
    for seed, poison in ((0, float("nan")), (0x5EED, float("nan")), (12345, 1.0), (2 ** 63 + 11, float("nan"))):
        got = _all_calls(t, seed, poison)
        for i, (a, b) in enumerate(zip(ref, got)):
            assert torch.equal(a, b), (i, seed)


@pytest.mark.parametrize("n,d,f", [(3, 512, 264), (400, 520, 264)])
def test_side_stream_and_two_graphs(n, d, f):
    ts = [_inputs(n, d, f, torch.bfloat16, s) for s in (1, 2)]
    ref = [[o.clone() for o in _all_calls(t, 0, 0.0)] for t in ts]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all_calls(ts[0], 0, float("nan"))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref[0], got))
    graphs = []
    for t in ts:   # both graphs allocate their workspaces inside the calls
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            y, mean, rstd = moe.moe_layernorm_fwd(t["x"], t["nw"], t["nb"], EPS)
            out = [y, mean, rstd, *moe.moe_layernorm_bwd(t["dx"], t["x"], t["nw"], mean, rstd)]
            y, z = moe.moe_linear_fwd(t["x"], t["w"], t["b"], t["dy"], "gelu", save_z=True)
            out += [y, z, *moe.moe_linear_bwd(t["dy"], t["x"], t["w"], z, "gelu")]
            gu = [torch.empty((n, f), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            out += moe.moe_glu_fwd(t["x"], t["w"], t["w2"], g=gu[0], u=gu[1])
            out += moe.moe_glu_bwd(t["dy"], t["x"], t["w"], t["w2"], *gu)
        graphs.append((g, out))
    torch.cuda.synchronize()
    for i in range(3):
        for _, out in graphs:
            for o in out:
                o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, out), r in zip(graphs, ref):
            for j, (a, b) in enumerate(zip(out, r)):
                assert torch.equal(a, b), (i, j)
        _all_calls(ts[i % 2], 0x5EED, 1.0)   # eager work between the replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_streams_at_once(dtype):
    ts = [_inputs(n, 520, 264, dtype, s) for n, s in ((200, 1), (1100, 2))]
    ref = [[o.clone() for o in _all_calls(t, 0, 0.0)] for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(3):
        got = []
        for st, t in zip(streams, ts):
            with torch.cuda.stream(st):
                got.append(_all_calls(t, 0, float("nan")))
        torch.cuda.synchronize()
        for g, r in zip(got, ref):
            for j, (a, b) in enumerate(zip(g, r)):
                assert torch.equal(a, b), j
        del got


@pytest.mark.parametrize("n", [7, 300])
def test_one_tensor_as_several_inputs(n):
    torch.manual_seed(n)
    x, w = torch.randn(n, 264, device=DEV).bfloat16(), torch.randn(264, 264, device=DEV).bfloat16()
    assert torch.equal(moe.moe_linear_fwd(x, w, residual=x)[0], moe.moe_linear_fwd(x, w, residual=x.clone())[0])
    a, g, u = moe.moe_glu_fwd(x, w, w, save=True)
    b, g2, u2 = moe.moe_glu_fwd(x, w, w.clone(), save=True)
    assert torch.equal(a, b) and torch.equal(g, u) and torch.equal(u, u2)
    one = moe.moe_linear_bwd(x, x, w, dx_add=x)
    two = moe.moe_linear_bwd(x.clone(), x.clone(), w, dx_add=x.clone())
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    one = moe.moe_glu_bwd(x, x, w, w, g, g, dx_add=x)
    two = moe.moe_glu_bwd(x.clone(), x, w, w.clone(), g, g2, dx_add=x.clone())
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_rows_past_two_gib():
    """Activations beyond 2 GiB (and 2^31 elements): the first, a middle and
    the last rows, and the weight gradients, whose contraction is cut into chunks
    that 32-bit offsets reach."""
    n, d, f = 1 << 20, 64, 2304
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((n, d), generator=g, device=DEV).bfloat16()
    w = (torch.randn((d, f), generator=g, device=DEV) / 8).bfloat16()
    y, _ = moe.moe_linear_fwd(x, w)
    rows = torch.cat([torch.arange(64), torch.arange(64) + 932067, torch.arange(64) + n - 64])
    want, _, tol, _ = B.linear_bounds("bf16", B.host(x[rows.to(DEV)]), B.host(w), None, None, "none")
    B.check(y[rows.to(DEV)], want, tol, "y")
    dx, dw, db = moe.moe_linear_bwd(y, x, w)
    sub = y[rows.to(DEV)]
    refs, tols = B.linear_bwd_bounds("bf16", "f32", B.host(sub), B.host(x[rows.to(DEV)]), B.host(w), B.host(sub),
                                     np.zeros(sub.shape), "none", None)
    B.check(dx[rows.to(DEV)], refs[0], tols[0], "dx")
    # dw: the sum over all rows in float64 on the device, 2^17 rows at a time
    ref = torch.zeros((d, f), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    for i in range(0, n, 1 << 17):
        xs, ys = x[i:i + (1 << 17)].double(), y[i:i + (1 << 17)].double()
        ref += xs.t() @ ys
        mag += xs.abs().t() @ ys.abs()
    # a chunk's sum has n / 4 products at most on one accumulator; the bound
    # takes all n
    assert bool(((dw.double() - ref).abs() <= (2 * n + 10) * B.E * mag).all())
    # and far inside it, the error of random roundings: sqrt(n) of them
    assert float((dw.double() - ref).norm() / ref.norm()) < 2e-5


# ------------------------------------------------------------ a block of them
@pytest.mark.parametrize("rows", [40, 600])
def test_block_with_the_expert_layer(rows):
    """norm -> routed experts and gated shared expert -> down projection with
    the routed output as its residual, forward and backward in float32, against
    the oracle's chain; and its gradient against differences of the oracle's loss."""
    rng = np.random.default_rng(17)
    D, F, E, k = 64, 192, 4, 2
    f32 = lambda *s, sc=1.0: (rng.standard_normal(s) * sc).astype(np.float32)  # noqa: E731
    P = dict(x=f32(rows, D), nw=1 + f32(D, sc=0.1), nb=f32(D, sc=0.1), wr=f32(E, D, sc=D ** -0.5), w1=f32(E, D, F, sc=D ** -0.5),
             w2=f32(E, F, D, sc=F ** -0.5), wg=f32(D, F, sc=D ** -0.5), wu=f32(D, F, sc=D ** -0.5), wd=f32(F, D, sc=F ** -0.5),
             bd=f32(D, sc=0.1), dy=f32(rows, D))
    t = {n: torch.from_numpy(v).to(DEV) for n, v in P.items()}
    prob = moe.Problem(rows, D, F, E, k, dtype="f32")
    logits = moe.moe_router_fwd(prob, t["x"], t["wr"])
    xn, mean, rstd = moe.moe_layernorm_fwd(t["x"], t["nw"], t["nb"], EPS)
    routing, h, ym = moe.moe_fwd(prob, logits, xn, t["w1"], t["w2"])
    a, g, u = moe.moe_glu_fwd(xn, t["wg"], t["wu"], save=True)
    y, _ = moe.moe_linear_fwd(a, t["wd"], t["bd"], residual=ym)
    da, dwd, dbd = moe.moe_linear_bwd(t["dy"], a, t["wd"])
    dxm, dprob, dh = moe.moe_bwd_dgrad_dprob(prob, routing, t["dy"], t["w1"], t["w2"], h)
    dxn, dwg, dwu = moe.moe_glu_bwd(da, xn, t["wg"], t["wu"], g, u, dx_add=dxm)
    _, _, dxr = moe.moe_router_bwd(prob, routing, dprob, t["x"], t["wr"])
    dx, dnw, dnb = moe.moe_layernorm_bwd(dxn, t["x"], t["nw"], mean, rstd, dx_add=dxr)

    Q = {n: v.astype(np.float64) for n, v in P.items()}
    idx = routing.topk_idx.cpu().numpy()

    def forward(Q):
        lg = Q["x"] @ Q["wr"].T
        sel = np.take_along_axis(lg, idx, 1)
        p = np.exp(sel - sel.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        n = oracle.layernorm_forward(Q["x"], Q["nw"], Q["nb"], EPS)[0]
        r = np.zeros((rows, D))
        for j in range(k):
            for e in range(E):
                m = idx[:, j] == e
                r[m] += p[m, j:j + 1] * (np.maximum(n[m] @ Q["w1"][e], 0) ** 2 @ Q["w2"][e])
        act = oracle.glu_forward(n, Q["wg"], Q["wu"], "silu")[0]
        return oracle.linear_forward(act, Q["wd"], Q["bd"], r, "none")[0]

    # float32 through four products in a row: 64 n roundings of relative size 2^-24 with
    # n = 192 stay far below 1e-4 of the largest values
    ref = forward(Q)
    assert np.abs(B.host(y) - ref).max() <= 1e-4 * np.abs(ref).max()
    loss = lambda Q: float((forward(Q) * Q["dy"]).sum())  # noqa: E731
    grads = dict(x=dx, nw=dnw, nb=dnb, wg=dwg, wu=dwu, wd=dwd, bd=dbd)
    for n, gr in grads.items():
        v = rng.standard_normal(P[n].shape)
        # central difference of the float64 oracle along v, step 1e-6: truncation
        # 1e-12 and rounding 1e-10 of the terms
        s = 1e-6
        up, dn = dict(Q), dict(Q)
        up[n], dn[n] = Q[n] + s * v, Q[n] - s * v
        want = (loss(up) - loss(dn)) / (2 * s)
        got = float((B.host(gr) * v).sum())
        scale = float(np.abs(B.host(gr) * v).sum())
        assert abs(got - want) <= 1e-4 * scale, (n, got, want, scale)
