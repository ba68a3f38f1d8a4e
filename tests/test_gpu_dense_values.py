"""The dense operators' values where the numbers themselves are hard: small
numbers times large ones in float32 products, element by element against
float64 within the bounds of dense_bounds.py."""
import numpy as np
import pytest
import torch

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
