"""Every kernel of the products in 8-bit integers (int8_cases.py) against the definition: rows of
both ends and of the borders of tiles against the oracle, every row against calls on few rows,
which other kernels take; in place, from the caller's codes, and with shuffled launches.  The
bounds are those of test_gpu_int8.py."""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import oracle
from int8_cases import EXPERTS, LINEAR, counts, experts_kernel, linear_kernel
from test_gpu_int8 import DEV, TYPE, _check_y, _f64, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _some(rows, products):
    """Rows to compare with the oracle: both ends and borders of tiles, as many as stay below 3e8 products."""
    most = max(6, int(3e8 / products))
    near = [0, rows - 1, 63, 64, 127, 128, 255, 256, 1, rows - 2, rows // 2] + list(range(2, rows))
    return sorted({r for r in near if 0 <= r < rows} if rows <= most else set([r for r in near if 0 <= r < rows][:most]))


def _inputs(rows, k, f, dtype, seed, residual=True, experts=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g, device=DEV).to(TYPE[dtype])  # noqa: E731
    return new(rows, k), new(f) if experts is None else new(experts, f), new(rows, f + 5) if residual else None


@pytest.mark.parametrize("kernel,dtype,rows,k,f,act", LINEAR)
def test_linear(kernel, dtype, rows, k, f, act):
    assert linear_kernel(dtype, rows, k, f, act) == "linear_" + kernel
    x, bias, wide = _inputs(rows, k, f, dtype, rows)
    res = wide[:, 2:f + 2].clone()
    w, ws, c, s = _weights(f, k, k)
    some = _some(rows, k * f)
    cx, sx = oracle.int8_quantize(_f64(x[some]))
    last = None
    for b, r in ((None, None), (bias, res)):
        got = moe.moe_int8_linear(x, w, ws, bias=b, residual=r, act=act)
        y, z, scaled = oracle.int8_product(cx, sx, c, s, None if b is None else _f64(b), act, None if r is None else _f64(r[some]))
        _check_y(got[some], y, z, scaled, act, None if r is None else _f64(r[some]), dtype)
        step = 16 if rows > 16 else 1
        for i in [*range(0, min(rows, 520), step), *range(max(0, rows - 300), rows, step)]:
            part = moe.moe_int8_linear(x[i:i + step], w, ws, bias=b, residual=None if r is None else r[i:i + step], act=act)
            assert torch.equal(got[i:i + step], part), i
        for i in range(0, rows, 500):   # other tiles
            part = moe.moe_int8_linear(x[i:i + 500], w, ws, bias=b, residual=None if r is None else r[i:i + 500], act=act)
            assert torch.equal(got[i:i + 500], part), i
        last = got
    assert torch.equal(moe.moe_int8_linear(x, w, ws, bias=bias, residual=res, act=act, shuffle_seed=11), last)
    codes, scales = moe.moe_int8_quantize(x)
    assert torch.equal(moe.moe_int8_linear(codes, w, ws, x_scales=scales, bias=bias, residual=res, act=act, out_dtype=TYPE[dtype]), last)
    # y is the residual, between other columns
    edge = wide[:, [0, 1, -3, -2, -1]].clone()
    moe.moe_int8_linear(x, w, ws, bias=bias, residual=wide[:, 2:f + 2], act=act, y=wide[:, 2:f + 2])
    assert torch.equal(wide[:, 2:f + 2], last) and torch.equal(wide[:, [0, 1, -3, -2, -1]], edge)


@pytest.mark.parametrize("kernel,dtype,cycle,experts,k,f,behind,act", EXPERTS)
def test_experts(kernel, dtype, cycle, experts, k, f, behind, act):
    assert experts_kernel(dtype, cycle, experts, k, f, behind, act) == "experts_" + kernel
    n = counts(cycle, experts)
    offsets = np.concatenate(([0], np.cumsum(n)))
    end = int(offsets[-1])
    rows = end + behind
    x, bias, _ = _inputs(rows, k, f, dtype, rows, False, experts)
    x[end:] = float("nan")                               # not read
    w, ws, c, s = _weights(f, k, experts, experts)
    off = torch.from_numpy(offsets.astype(np.int32)).to(DEV)
    wide = torch.full((rows, f + 3), 7.0, dtype=TYPE[dtype], device=DEV)
    y = wide[:, 1:f + 1]
    moe.moe_int8_experts(x, w, ws, off, bias=bias, act=act, y=y)
    assert (wide[end:] == 7).all() and (wide[:, [0, -2, -1]] == 7).all()
    for seed in (4, 61):
        assert torch.equal(moe.moe_int8_experts(x, w, ws, off, bias=bias, act=act, shuffle_seed=seed)[:end], y[:end])
    codes, scales = moe.moe_int8_quantize(x)
    again = moe.moe_int8_experts(codes, w, ws, off, x_scales=scales, bias=bias, act=act, out_dtype=TYPE[dtype])
    assert torch.equal(again[:end], y[:end])
    used = [e for e in range(experts) if n[e]]
    for e in {used[0], used[-1], used[len(used) // 2], max(used, key=lambda e: n[e])}:
        a, b = int(offsets[e]), int(offsets[e + 1])
        some = [a + r for r in _some(b - a, k * f)]
        cx, sx = oracle.int8_quantize(_f64(x[some]))
        want, z, scaled = oracle.int8_product(cx, sx, c[e], s[e], _f64(bias[e]), act)
        _check_y(y[some], want, z, scaled, act, None, dtype)
    for e in used:
        a, b = int(offsets[e]), int(offsets[e + 1])
        for i in range(a, b, 400):
            j = min(i + 400, b)
            assert torch.equal(y[i:j], moe.moe_int8_linear(x[i:j], w[e], ws[e], bias=bias[e], act=act)), (e, i)
