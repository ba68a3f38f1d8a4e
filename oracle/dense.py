"""Float64 definitions of the dense operators (layer norm, linear map with
bias, activation and residual, gated product) and their gradients."""
import numpy as np
from scipy.special import erf


def act(name: str, z: np.ndarray):
    """Value and derivative of an activation."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if name == "relu2":
        r = np.maximum(z, 0.0)
        return r * r, 2 * r
    if name == "silu":
        p = 0.5 * (1 + np.tanh(0.5 * z))
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        c = 0.5 * (1 + erf(z / np.sqrt(2.0)))
        return z * c, c + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    raise ValueError(name)


def layernorm_forward(x, weight, bias, eps):
    """(y, mean, rstd) of each row of x [T, C]; weight and bias may be None."""
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / np.sqrt((c * c).mean(1) + eps)
    h = c * rstd[:, None]
    y = h * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return y, mean, rstd


def layernorm_backward(dy, x, weight, eps, add=None):
    """(dx, dweight, dbias)."""
    _, mean, rstd = layernorm_forward(x, None, None, eps)
    h = (x - mean[:, None]) * rstd[:, None]
    dh = dy * (1.0 if weight is None else weight)
    dx = rstd[:, None] * (dh - dh.mean(1, keepdims=True) - h * (dh * h).mean(1, keepdims=True))
    return dx + (0.0 if add is None else add), (dy * h).sum(0), dy.sum(0)


def linear_forward(x, w, bias, residual, name):
    """(y, z)."""
    z = x @ w + (0.0 if bias is None else bias)
    return act(name, z)[0] + (0.0 if residual is None else residual), z


def linear_backward(dy, x, w, z, name, add=None):
    """(dx, dw, db)."""
    dz = dy * act(name, z)[1]
    return dz @ w.T + (0.0 if add is None else add), x.T @ dz, dz.sum(0)


def glu_forward(x, wg, wu, name):
    """(a, g, u)."""
    g, u = x @ wg, x @ wu
    return act(name, g)[0] * u, g, u


def glu_backward(da, x, wg, wu, g, u, name, add=None):
    """(dx, dwg, dwu)."""
    v, d = act(name, g)
    dg, du = da * u * d, da * v
    return dg @ wg.T + du @ wu.T + (0.0 if add is None else add), x.T @ dg, x.T @ du
