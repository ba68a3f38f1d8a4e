"""The dense matrix operators on matrices that start at any element: slices of
larger tensors, halves of one weight matrix at an odd column, contiguous outputs
inside a buffer; against the float64 oracle within the bounds of
dense_bounds.py, and what lies around the outputs untouched."""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import dense_bounds as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _at(t, off, pad):
    """t's values in a slice that starts `off` elements after a 16-byte address,
    rows `pad` further apart, NaN around it."""
    r, c = t.shape
    buf = torch.full((off + r * (c + pad) + 8,), float("nan"), dtype=t.dtype, device=DEV)
    v = buf[off:off + r * (c + pad)].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


class _Out:
    """A [r, c] output slice in a buffer of sevens."""

    def __init__(self, r, c, dtype, off, pad=0):
        self.buf = torch.full((off + (r + 1) * (c + pad) + 8,), 7.0, dtype=dtype, device=DEV)
        self.off, self.r, self.c, self.ld = off, r, c, c + pad
        self.t = self.buf[off:off + r * (c + pad)].view(r, c + pad)[:, :c]

    def check(self):
        keep = torch.ones_like(self.buf, dtype=torch.bool)
        keep[self.off:self.off + self.r * self.ld].view(self.r, self.ld)[:, :self.c] = False
        assert bool((self.buf[keep] == 7).all()), "elements around an output were written"


# one row, few rows, tiles of each kind; widths that vectors divide, so that only the
# address is odd, and odd ones
SIZES = [(1, 64, 72), (20, 256, 136), (45, 128, 264), (64, 264, 96), (130, 72, 200), (300, 520, 264), (1100, 1032, 1040),
         (33, 67, 35), (257, 129, 131)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", [1, 3, 4])
@pytest.mark.parametrize("rows,d,f", SIZES)
def test_slices_at_any_element(dtype, off, rows, d, f):
    rng = np.random.default_rng(rows + d + f + off)
    T = B.TORCH[dtype]
    pad = 8 if f % 8 == 0 else 0
    x, hx = B.values(rng, (rows, d), dtype)
    w, hw = B.values(rng, (d, f), dtype, d ** -0.5)
    w2, hw2 = B.values(rng, (d, f), dtype, d ** -0.5)
    b, hb = B.values(rng, (f,), dtype, 0.3)
    r, hr = B.values(rng, (rows, f), dtype)
    dy, hdy = B.values(rng, (rows, f), dtype)
    add, hadd = B.values(rng, (rows, d), dtype)
    xv, wv, rv, dyv, av = _at(x, off, pad), _at(w, off, pad), _at(r, off, pad), _at(dy, off, pad), _at(add, off, pad)
    bv = _at(b.reshape(1, -1), off, 0)[0]
    y, z = _Out(rows, f, T, off, pad), _Out(rows, f, torch.float32, off, pad)
    moe.moe_linear_fwd(xv, wv, bv, rv, "silu", y=y.t, z=z.t)
    ref, hz, tol, ez = B.linear_bounds(dtype, hx, hw, hb, hr, "silu")
    B.check(y.t, ref, tol, "y")
    ez = B.rounded(ez, hz, B.U["f32"])
    B.check(z.t, hz, ez, "z")
    dx, dw, db = _Out(rows, d, T, off), _Out(d, f, T, off), _Out(1, f, T, off)
    for act, zz in (("silu", z.t), ("none", None)):   # with "none", dy itself is multiplied
        moe.moe_linear_bwd(dyv, xv, wv, zz, act, dx_add=av, grad_dtype=T, dx=dx.t, dw=dw.t, db=db.t[0])
        refs, tols = B.linear_bwd_bounds(dtype, dtype, hdy, hx, hw, hz, ez if zz is not None else 0 * ez, act, hadd)
        for n, o, rr, tt in zip(("dx", "dw", "db"), (dx.t, dw.t, db.t[0]), refs, tols):
            B.check(o, rr, tt, n + " " + act)
    for o in (y, z, dx, dw, db):
        o.check()
    # the gated product; g and u of the storage type
    w2v = _at(w2, 0 if off == 4 else off, pad)
    a, g, u = _Out(rows, f, T, off, pad), _Out(rows, f, T, off, pad), _Out(rows, f, T, 0, pad)
    moe.moe_glu_fwd(xv, wv, w2v, "gelu", a=a.t, g=g.t, u=u.t)
    ref, rg, ru, tol, eg, eu = B.glu_bounds(dtype, hx, hw, hw2, "gelu")
    B.check(a.t, ref, tol, "a")
    eg, eu = B.rounded(eg, rg, B.U[dtype]), B.rounded(eu, ru, B.U[dtype])
    B.check(g.t, rg, eg, "g")
    B.check(u.t, ru, eu, "u")
    dwu = _Out(d, f, T, 0)
    moe.moe_glu_bwd(dyv, xv, wv, w2v, g.t, u.t, "gelu", dx_add=av, grad_dtype=T, dx=dx.t, dwg=dw.t, dwu=dwu.t)
    refs, tols = B.glu_bwd_bounds(dtype, dtype, hdy, hx, hw, hw2, rg, ru, eg, eu, "gelu", hadd)
    for n, o, rr, tt in zip(("dx", "dwg", "dwu"), (dx.t, dw.t, dwu.t), refs, tols):
        B.check(o, rr, tt, n)
    for o in (a, g, u, dx, dw, dwu):
        o.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 40, 200])
@pytest.mark.parametrize("f", [68, 35])
def test_halves_of_one_weight_matrix_and_rows_of_one_input(dtype, rows, f):
    rng = np.random.default_rng(rows + f)
    d = 41
    both, hb = B.values(rng, (d, 2 * f), dtype, d ** -0.5)
    xs, hxs = B.values(rng, (rows + 1, d), dtype)
    both, xs = both.to(DEV), xs.to(DEV)
    a, g, u = moe.moe_glu_fwd(xs[1:], both[:, :f], both[:, f:], save=True)
    ref, rg, ru, tol, eg, eu = B.glu_bounds(dtype, hxs[1:], hb[:, :f], hb[:, f:], "silu")
    B.check(a, ref, tol, "a")
    da, hda = B.values(rng, (rows, f), dtype)
    dx, dwg, dwu = moe.moe_glu_bwd(da.to(DEV), xs[1:], both[:, :f], both[:, f:], g, u)
    refs, tols = B.glu_bwd_bounds(dtype, "f32", hda, hxs[1:], hb[:, :f], hb[:, f:], rg, ru, B.rounded(eg, rg, B.E),
                                  B.rounded(eu, ru, B.E), "silu", None)
    for n, o, rr, tt in zip(("dx", "dwg", "dwu"), (dx, dwg, dwu), refs, tols):
        B.check(o, rr, tt, n)


@pytest.mark.parametrize("rows", [0, 3])
def test_no_rows_at_an_odd_address(rows):
    x, w = torch.empty(rows, 24, device=DEV).fill_(1), torch.randn(24, 10, device=DEV)
    dw = _Out(24, 10, torch.float32, 1)
    moe.moe_linear_bwd(torch.zeros(rows, 10, device=DEV), x, w, dw=dw.t)
    assert not dw.t.any()
    dw.check()


@pytest.mark.parametrize("off,pad", [(0, 3), (0, 8), (3, 0), (5, 8)])
def test_workspaces_of_the_stated_sizes(off, pad):
    """Strided and unaligned tensors with workspaces allocated beforehand."""
    n, d, f = 200, 72, 136
    torch.manual_seed(off + pad)
    r = lambda *s: _at(torch.randn(*s).bfloat16(), off, pad)  # noqa: E731
    x, w, w2, dy = r(n, d), r(d, f), r(d, f), r(n, f)
    kw = dict(ldx=d + pad, ldw=f + pad, ldy=f + pad, unaligned=("x", "w", "y") if off else ())
    W = lambda k: torch.empty(k, dtype=torch.uint8, device=DEV) if k else None  # noqa: E731
    lf, lb = moe.moe_linear_workspace_size(n, d, f, act="gelu", **kw)
    gf, gb = moe.moe_glu_workspace_size(n, d, f, **kw)
    y = _Out(n, f, torch.bfloat16, off, pad)
    _, z = moe.moe_linear_fwd(x, w, act="gelu", y=y.t, save_z=True, ws=W(lf))
    assert torch.equal(y.t, moe.moe_linear_fwd(x, w, act="gelu")[0])
    for a, b in zip(moe.moe_linear_bwd(dy, x, w, z, "gelu", ws=W(lb)), moe.moe_linear_bwd(dy, x, w, z, "gelu")):
        assert torch.equal(a, b)
    a = _Out(n, f, torch.bfloat16, off, pad)
    _, g, u = moe.moe_glu_fwd(x, w, w2, a=a.t, save=True, ws=W(gf))
    assert torch.equal(a.t, moe.moe_glu_fwd(x, w, w2)[0])
    for p, q in zip(moe.moe_glu_bwd(dy, x, w, w2, g, u, ws=W(gb)), moe.moe_glu_bwd(dy, x, w, w2, g, u)):
        assert torch.equal(p, q)
