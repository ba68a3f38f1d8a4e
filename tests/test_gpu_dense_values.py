"""The dense operators' values where the numbers themselves are hard: small
numbers times large ones in float32 products, and the activations over their
whole range, tails included; element by element against float64."""
import numpy as np
import pytest
import torch
from scipy.special import erfc, expit

import bitwise_deterministic_moe_amd as moe
import dense_bounds as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
TINY = (-118, -120, -122, -124, -130)   # the last one is below float32's normal numbers


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _spread(rng, shape, rows, cols):
    """Numbers near 2^50, but some rows and columns near 2^-118 and less."""
    a = rng.standard_normal(shape).astype(np.float32) * np.float32(2.0 ** 50)
    for i, e in zip(rows, TINY):
        a[i] = rng.standard_normal(shape[1]) * 2.0 ** e
    for i, e in zip(cols, TINY):
        a[:, i] = rng.standard_normal(shape[0]) * 2.0 ** e
    return a


def _check(got, a, b, what):
    """got = a b: a float32 product of n numbers is off by at most (2 n + 10)
    2^-24 of the products' magnitudes, and a product below 2^-126 (a small number
    times a small one) by 2^-149."""
    a, b = a.astype(np.float64), b.astype(np.float64)
    ref, tol = a @ b, B.prod_err(a.shape[1], np.abs(a), np.abs(b)) + a.shape[1] * 2.0 ** -148
    B.check(got, ref, B.rounded(tol, ref, B.U["f32"]), what)


# the float32 tiles of 128 x 128 and of 64 x 64, whole and ragged
@pytest.mark.parametrize("n,d,f", [(2048, 512, 2048), (2051, 515, 2047), (200, 130, 140)])
def test_small_times_large_float32_numbers(n, d, f):
    """A number far below 1 against one far above it: every bit of both counts,
    whatever else the tile holds."""
    rng = np.random.default_rng(n)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    x = _spread(rng, (n, d), (0, 5, 70, 131, n - 1), (1, 64, 100, 127, d - 1))
    w = _spread(rng, (d, f), (2, 33, 66, 128, d - 2), (0, 63, 65, 139, f - 1))
    w2 = _spread(rng, (d, f), (3, 34, 67, 129, d - 3), (1, 60, 66, 131, f - 2))
    dy = _spread(rng, (n, f), (4, 35, 68, 130, n - 4), (2, 61, 67, 132, f - 3))
    xd, wd, wd2, dyd = up(x), up(w), up(w2), up(dy)
    y = moe.moe_linear_fwd(xd, wd)[0]
    _check(y, x, w, "y")
    dx, dw, _ = moe.moe_linear_bwd(dyd, xd, wd, need_db=False)
    _check(dx, dy, w.T, "dx")
    _check(dw, x.T, dy, "dw")
    _, g, u = moe.moe_glu_fwd(xd, wd, wd2, "none", save=True)
    _check(g, x, w, "g")
    _check(u, x, w2, "u")
    one = torch.ones(n, f, device=DEV)   # then dg = du = dy
    dx, dwg, dwu = moe.moe_glu_bwd(dyd, xd, wd, wd2, one, one, "none")
    _check(dx, np.concatenate([dy, dy], 1), np.concatenate([w, w2], 1).T, "dx of the gated product")
    _check(dwg, x.T, dy, "dwg")
    _check(dwu, x.T, dy, "dwu")
    # the other rows and columns keep their bits where the small ones are ordinary
    x1, w1 = x.copy(), w.copy()
    rows, cols = [0, 5, 70, 131, n - 1], [0, 63, 65, 139, f - 1]
    x1[rows], w1[:, cols] = 1.5, -0.25
    y1 = moe.moe_linear_fwd(up(x1), up(w))[0]
    keep = torch.tensor([i not in rows for i in range(n)], device=DEV)
    assert torch.equal(y1[keep], y[keep])
    y1 = moe.moe_linear_fwd(up(x), up(w1))[0]
    keep = torch.tensor([i not in cols for i in range(f)], device=DEV)
    assert torch.equal(y1[:, keep], y[:, keep])


@pytest.mark.parametrize("n,d,f", [(5, 264, 136), (200, 264, 136), (2048, 512, 2048), (600, 2048, 1100)])
def test_small_times_large_bf16_numbers(n, d, f):
    """The same in bf16: numbers below its normal ones count too."""
    rng = np.random.default_rng(n)
    b = lambda a: torch.from_numpy(a).bfloat16()  # noqa: E731
    x = b(_spread(rng, (n, d), (0, 2, 3, 4, n - 1), (1, 64, 100, 127, d - 1)))
    w = b(_spread(rng, (d, f), (2, 33, 66, 128, d - 2), (0, 63, 65, 131, f - 1)))
    dy = b(_spread(rng, (n, f), (1, 2, 3, 4, n - 1), (2, 61, 67, 132, f - 3)))
    hx, hw, hdy = B.host(x), B.host(w), B.host(dy)
    x, w, dy = x.to(DEV), w.to(DEV), dy.to(DEV)

    def check(got, a, c, what):
        ref, tol = a @ c, B.prod_err(a.shape[1], np.abs(a), np.abs(c)) + a.shape[1] * 2.0 ** -148
        B.check(got, ref, B.rounded(tol, ref, B.U["bf16" if got.dtype == torch.bfloat16 else "f32"]) + 2.0 ** -134, what)

    check(moe.moe_linear_fwd(x, w)[0], hx, hw, "y")
    dx, dw, _ = moe.moe_linear_bwd(dy, x, w, need_db=False)
    check(dx, hdy, hw.T, "dx")
    check(dw, hx.T, hdy, "dw")
    _, g, u = moe.moe_glu_fwd(x, w, w, "none", save=True)
    check(g, hx, hw, "g")
    assert torch.equal(g, u)


# ----------------------------------------------------------------- activations
def _truth(name, z):
    """Value and derivative in float64, and the magnitudes of the derivative's two
    terms, without cancellation in the tails."""
    if name == "silu":
        s, c = expit(z), expit(-z)
        return z * s, s + z * s * c, s * (1 + np.abs(z) * c), s
    p, e = 0.5 * erfc(-z / np.sqrt(2.0)), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    return z * p, p + z * e, p + np.abs(z) * e, p


def _errors(name, dtype, z, truth):
    """Bounds of the float32 value and derivative, from the arithmetic, with E =
    2^-24 a float32 rounding, exponential and reciprocal within 2 E, 2^-120 for what
    lies below the exponential's range.
    Accurate form: SiLU 4 E (the exponential in two parts), 3 E (1 + e), 2 E, E, E; GELU
    the fit 0.4 E, t 3 E times its condition 2.4, a sum of 9 terms with twice its value
    in magnitudes 9 E, the products and the exponential 6 E.
    For bf16: SiLU's exponential has an argument error of 1.5 E |z|, and 1 - s another
    E; GELU 20 E for the fit, 12 E for t, 12 E for the sum, (1.3 z^2 + 5) E for the
    exponential and products."""
    v, _, mag, s = truth
    a, E = np.abs(z), B.E
    if dtype == "f32":
        k = 12 if name == "silu" else 24
        return k * E * np.abs(v) + 2.0 ** -120, (k + 4) * E * mag + 2.0 ** -120
    if name == "silu":
        return (2 * a + 8) * E * np.abs(v) + 2.0 ** -120, (2 * a + 16) * E * (1 + a) * s + 2.0 ** -120
    return (3 * a * a + 64) * E * np.abs(v) + 2.0 ** -120, (3 * a * a + 68) * E * mag + 2.0 ** -120


def _sweep(dtype):
    z = np.concatenate([np.linspace(-14, 14, 1793), np.linspace(-86, 86, 173), [0.0, 1e-30, -1e-30, 1e-6, -1e-6, 300.0, -300.0]])
    t = torch.from_numpy(z.astype(np.float32)).to(B.TORCH[dtype]).to(DEV)
    return t.reshape(1, -1), B.host(t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [1, 70, 1100])
def test_activations_over_their_range(name, dtype, rows):
    """act(1 z) and its derivative for one input of 1, so that z is exact: the
    weight-streaming kernel, and tiles of both sizes."""
    w, z = _sweep(dtype)
    n = z.size
    x = torch.ones(rows, 1, dtype=w.dtype, device=DEV)
    truth = _truth(name, z)
    ev, ed = _errors(name, dtype, z, truth)
    y, zs = moe.moe_linear_fwd(x, w, act=name, save_z=True)
    assert torch.equal(zs, w.float().expand(rows, n))
    B.check(y[0], truth[0], B.rounded(ev, truth[0], B.U[dtype]), "y")
    assert torch.equal(y, y[:1].expand(rows, n))
    a = moe.moe_glu_fwd(x, w, torch.ones_like(w), name)[0]
    assert torch.equal(a, y)
    # the bias gradient is the sum over rows of the unrounded dz, here one row of dy
    dy = torch.zeros(rows, n, dtype=w.dtype, device=DEV)
    dy[rows // 2] = 1
    dx, dw, db = moe.moe_linear_bwd(dy, x, w, zs, name)
    B.check(db, truth[1], B.rounded(ed, truth[1], B.E), "db")
    B.check(dw[0], truth[1], B.rounded(B.rounded(ed, truth[1], B.U[dtype]), truth[1], B.E), "dw")
    # dg = da u act'(g) and du = da act(g)
    dx, dwg, dwu = moe.moe_glu_bwd(dy, x, w, torch.ones_like(w), zs, torch.ones_like(zs), name)
    B.check(dwg[0], truth[1], B.rounded(B.rounded(ed, truth[1], B.U[dtype]), truth[1], B.E), "dwg")
    B.check(dwu[0], truth[0], B.rounded(B.rounded(ev, truth[0], B.U[dtype]), truth[0], B.E), "dwu")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activations_of_infinite_and_nan_numbers(name, dtype):
    z = torch.tensor([[float("inf"), float("nan"), 1.0]], dtype=B.TORCH[dtype], device=DEV)
    y = moe.moe_linear_fwd(torch.ones(1, 1, dtype=z.dtype, device=DEV), z, act=name)[0][0]
    assert y[0] == float("inf") and torch.isnan(y[1]) and torch.isfinite(y[2])
