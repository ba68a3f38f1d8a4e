"""Inputs and error bounds for the tests of the dense operators.

Bounds are first-order, element by element, from the arithmetic:
  * a rounding to type t is off by at most U[t] of the value (half a step);
  * a float32 addition or multiplication by at most 2^-24 of its result, an
    addition inside the matrix unit by at most 2^-23 (its adder may cut off), so
    a sum of n products is off by at most (2 n + 10) 2^-24 of the sum of the
    products' magnitudes, in any order and split.  Large float32 products are
    made of six products of 8-bit parts: what they leave out is below 2^-21
    of a product, 8 of the 10 above, and the six run in chains of 16 k an
    instruction, 6 n / 16 sums at 2^-23 = 0.75 n 2^-24 beside at most
    2 * 16 2^-24 inside one: below 2 n for n >= 32;
  * the activations' errors are relative, at most 12 (SiLU) and 24 (GELU) times
    2^-24 for float32 storage, 2 |z| + 8 and 3 z^2 + 64 times for bf16
    (test_gpu_dense_values.py holds them to that); act_err below is no smaller
    around 0, where these tests' z lie;
  * |act''| <= 0.5 (SiLU), 0.8 (GELU), 2 (ReLU^2): an error of z becomes at most
    that much of act'(z).  ReLU's derivative jumps at 0, so it is
    tested on inputs whose z is exact.
"""
import numpy as np
import torch

import oracle

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
E = 2.0 ** -24
# (bound of |act'|, of |act''|)
LIP = {"none": (1.0, 0.0), "relu": (1.0, 0.0), "silu": (1.1, 0.5), "gelu": (1.13, 0.8)}


def lip(name, z, ez):
    if name == "relu2":
        return 2 * (np.abs(z) + ez), 2.0
    return LIP[name]


def act_err(name, z):
    """Evaluation errors of act(z) and act'(z) in float32."""
    a = np.abs(z)
    if name == "none":
        return 0 * a, 0 * a
    if name in ("relu", "relu2"):
        return 4 * E * a * a, 4 * E * a
    return 4 * E * a * (a + 8), 8 * E * (1 + a) * (a + 8)


def values(rng, shape, dtype, scale=1.0, shift=0.0):
    """Device tensor of the storage type and its float64 values."""
    a = torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32)).to(TORCH[dtype])
    return a, a.double().numpy()


def small_ints(rng, shape, dtype, top=2):
    a = torch.from_numpy(rng.integers(-top, top + 1, shape).astype(np.float32)).to(TORCH[dtype])
    return a, a.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, tol, what):
    got = host(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {got[i]!r}, want {ref[i]!r}, "
                             f"tolerance {np.broadcast_to(tol, ref.shape)[i]:.3g}")


def rounded(tol, ref, u):
    """Tolerance after a rounding with half step u."""
    return tol + u * (np.abs(ref) + tol)


def prod_err(n, a, b):
    return (2 * n + 10) * E * (a @ b)


def linear_bounds(dtype, x, w, bias, res, name):
    """(y, z, tolerance of y, error of z before its rounding)."""
    y, z = oracle.linear_forward(x, w, bias, res, name)
    ez = prod_err(x.shape[1], np.abs(x), np.abs(w)) + 4 * E * (np.abs(z) + (0 if bias is None else np.abs(bias)))
    v = oracle.act(name, z)[0]
    ey = lip(name, z, ez)[0] * ez + act_err(name, z)[0] + 2 * E * (np.abs(v) + (0 if res is None else np.abs(res)))
    return y, z, rounded(ey, y, U[dtype]), ez


def dz_err(dtype, dy, z, ez, name):
    """Error of the float32 dz, and of the dz that the products read."""
    d = oracle.act(name, z)[1]
    e = np.abs(dy) * (lip(name, z, ez)[1] * ez + act_err(name, z)[1]) + 4 * E * np.abs(dy * d)
    r = e if name == "none" else rounded(e, dy * d, U[dtype])
    return e, r


def linear_bwd_bounds(dtype, gdtype, dy, x, w, z, ez, name, add):
    """((dx, dw, db), their tolerances); ez: error of the saved z."""
    ref = oracle.linear_backward(dy, x, w, z, name, add)
    dz = dy * oracle.act(name, z)[1]
    e32, ez2 = dz_err(dtype, dy, z, ez, name)
    m = np.abs(dz) + ez2
    T, F = dy.shape
    ax, aw = np.abs(x), np.abs(w)
    tx = ez2 @ aw.T + prod_err(F, m, aw.T) + 2 * E * (0 if add is None else np.abs(add))
    tw = ax.T @ ez2 + prod_err(T, ax.T, m)
    tb = e32.sum(0) + (T + 10) * E * np.abs(dz).sum(0)
    return ref, (rounded(tx, ref[0], U[dtype]), rounded(tw, ref[1], U[gdtype]), rounded(tb, ref[2], U[gdtype]))


def glu_bounds(dtype, x, wg, wu, name):
    """(a, g, u, tolerance of a, errors of g and u before their rounding)."""
    a, g, u = oracle.glu_forward(x, wg, wu, name)
    eg, eu = (prod_err(x.shape[1], np.abs(x), np.abs(w)) for w in (wg, wu))
    v = oracle.act(name, g)[0]
    ea = np.abs(u) * (lip(name, g, eg)[0] * eg + act_err(name, g)[0]) + (np.abs(v) + eg) * eu + 4 * E * np.abs(a)
    return a, g, u, rounded(ea, a, U[dtype]), eg, eu


def glu_bwd_bounds(dtype, gdtype, da, x, wg, wu, g, u, eg, eu, name, add):
    ref = oracle.glu_backward(da, x, wg, wu, g, u, name, add)
    v, d = oracle.act(name, g)
    l1, l2 = lip(name, g, eg)
    ev, ed = act_err(name, g)
    dg, du = da * u * d, da * v
    ed1 = l2 * eg + ed
    e0 = np.abs(da) * ((np.abs(u) + eu) * ed1 + np.abs(d) * eu) + 6 * E * np.abs(dg)
    e1 = np.abs(da) * (l1 * eg + ev) + 4 * E * np.abs(du)
    e0, e1 = rounded(e0, dg, U[dtype]), rounded(e1, du, U[dtype])
    m0, m1 = np.abs(dg) + e0, np.abs(du) + e1
    T, F = da.shape
    ax, ag, au = np.abs(x), np.abs(wg), np.abs(wu)
    tx = e0 @ ag.T + e1 @ au.T + prod_err(2 * F, m0, ag.T) + prod_err(2 * F, m1, au.T) + \
        2 * E * (0 if add is None else np.abs(add))
    t0, t1 = ax.T @ e0 + prod_err(T, ax.T, m0), ax.T @ e1 + prod_err(T, ax.T, m1)
    return ref, (rounded(tx, ref[0], U[dtype]), rounded(t0, ref[1], U[gdtype]), rounded(t1, ref[2], U[gdtype]))


# A row sum adds at most 32 elements a thread, then a tree over 64 lanes and
# up to 16 waves: fewer than 64 roundings on any path.
ROW = 64 * E


def norm_stats_err(x, eps):
    """Errors of mean and relative error of rstd."""
    _, mean, rstd = oracle.layernorm_forward(x, None, None, eps)
    em = ROW * np.abs(x).mean(1) + E * np.abs(mean)
    # a shifted mean adds its square to the variance
    return mean, rstd, em, 0.5 * (em * rstd) ** 2 + ROW


def norm_bounds(dtype, x, weight, bias, eps):
    y, _, _ = oracle.layernorm_forward(x, weight, bias, eps)
    mean, rstd, em, er = norm_stats_err(x, eps)
    h = (x - mean[:, None]) * rstd[:, None]
    eh = norm_h_err(x, mean, rstd, em, er, h)
    aw = 1.0 if weight is None else np.abs(weight)
    return y, rounded(aw * eh + 2 * E * (np.abs(h) * aw + (0 if bias is None else np.abs(bias))), y, U[dtype])


def norm_h_err(x, mean, rstd, em, er, h):
    return rstd[:, None] * (em[:, None] + E * (np.abs(x) + np.abs(mean)[:, None])) + np.abs(h) * (er[:, None] + 2 * E)


def norm_bwd_bounds(dtype, dy, x, weight, eps, add):
    ref = oracle.layernorm_backward(dy, x, weight, eps, add)
    mean, rstd, em, er = norm_stats_err(x, eps)
    h = (x - mean[:, None]) * rstd[:, None]
    eh = norm_h_err(x, mean, rstd, em, er, h)
    dh = dy * (1.0 if weight is None else weight)
    mn = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    m1, m2 = mn(dh), mn(dh * h)
    e1 = ROW * mn(np.abs(dh))
    e2 = mn(np.abs(dh) * eh) + ROW * mn(np.abs(dh * h))
    inner = np.abs(dh) + np.abs(m1) + np.abs(h * m2)
    tx = rstd[:, None] * (e1 + np.abs(h) * e2 + np.abs(m2) * eh + e2 * eh + 6 * E * inner + er[:, None] * inner) + \
        2 * E * (0 if add is None else np.abs(add))
    T = x.shape[0]
    tw = (np.abs(dy) * eh).sum(0) + (T + 20) * E * np.abs(dy * h).sum(0)
    tb = (T + 20) * E * np.abs(dy).sum(0)
    return ref, (rounded(tx, ref[0], U[dtype]), rounded(tw, ref[1], E), rounded(tb, ref[2], E))
