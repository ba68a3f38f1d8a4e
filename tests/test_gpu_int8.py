"""The products in 8-bit integers on the GPU against their definition.

Codes and scales are exact.  Bounds of y, element by element: the sum is exact
in int32; its conversion, its products with the two scales and the addition of
the bias round once each, z is off by at most (3 |s| + |z|) 2^-24 to the first
order (s the scaled sum; (4 |s| + 2 |z|) covers the second); the activation adds its
own error and at most its Lipschitz constant times z's (dense_bounds.py); a
residual's addition rounds once more; the type's rounding comes last.
"""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import oracle
from dense_bounds import E, U, act_err, lip

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _f64(t):
    return t.double().cpu().numpy()


def _check_y(got, y, z, s, act, res, dtype):
    ez = (4 * np.abs(s) + 2 * np.abs(z)) * E
    bound = act_err(act, z)[0] + lip(act, z, ez)[0] * ez
    size = np.abs(y) if res is None else np.abs(y) + np.abs(res)
    bound = bound + 2 * E * size
    bound = bound + U[dtype] * (np.abs(y) + bound)
    bad = ~(np.abs(_f64(got) - y) <= bound)
    assert not bad.any(), (int(bad.sum()), np.abs(_f64(got) - y).max())


# ------------------------------------------------------------------ quantising
def _values(rows, cols, dtype, seed, wide=0, unaligned=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.randn((rows, cols + wide), generator=g, device=DEV)
    a = (a * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=DEV).float())).to(TYPE[dtype])
    if unaligned:
        b = torch.empty(a.numel() + 1, dtype=a.dtype, device=DEV)[1:].reshape(a.shape)
        a = b.copy_(a)
    return a[:, :cols]


QUANT = [(1, 1), (3, 15), (2, 16), (5, 17), (9, 64), (130, 333), (7, 2048), (5, 4096), (3, 4099), (2, 20000), (1, 131072)]


@pytest.mark.parametrize("wide,unaligned", [(0, False), (0, True), (5, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quantize(rows, cols, dtype, wide, unaligned):
    x = _values(rows, cols, dtype, rows + cols, wide, unaligned)
    # ties (half of the largest; odd units beside 254), zeros, the smallest row that is not
    # zeros and the largest that is, numbers that are not finite
    if rows >= 3 and cols >= 15:
        x[0, :6] = torch.tensor([254., 3., -125., 127., 1., -253.], device=DEV)
        x[0, 6:] = torch.randint(-126, 126, (cols - 6,), device=DEV).to(x.dtype) * 2 + 1
        x[1] = 0
        x[1, 2:5] = torch.tensor([2.0, 1.0, -1.0], device=DEV)
    if rows >= 9:
        x[2], x[3], x[4] = 0, 0, 0
        x[3, 1], x[4, 1] = 2.0 ** -101, -2.0 ** -100
        x[5, 3], x[6, 3], x[7, 3] = float("inf"), float("nan"), -float("inf")
    if rows >= 130 and dtype == "f32":   # next to a tie: a unit above and below half of the largest
        x[20, 0], x[20, 1], x[20, 2] = 16777215.0, 8388607.5, 8388607.0
        x[20, 3:] = 0.0
        top = torch.tensor(3.3333333, device=DEV)
        x[21] = (torch.arange(cols, device=DEV) % 127 + 0.5) / 127 * top
        x[21, 0] = top
    codes, scales = moe.moe_int8_quantize(x)
    k16 = (cols + 15) // 16 * 16
    assert codes.shape == (rows, k16) and scales.shape == (rows,)
    want, ws = oracle.int8_quantize(_f64(x))
    assert np.array_equal(codes[:, :cols].cpu().numpy(), want)
    assert (codes[:, cols:] == 0).all()
    assert np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
    again = moe.moe_int8_quantize(x, codes=torch.full_like(codes, 9), scales=torch.zeros_like(scales), shuffle_seed=5)
    assert torch.equal(again[0], codes) and np.array_equal(again[1].cpu().numpy(), ws, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,k,f", [(1, 1, 1), (3, 7, 5), (1, 64, 64), (2, 100, 130), (1, 1000, 65), (5, 33, 8), (1, 300, 1001)])
def test_quantize_t(batch, k, f, dtype):
    w = _values(batch * k, f, dtype, k * f).reshape(batch, k, f).contiguous()
    if f >= 5 and k >= 7:
        w[0, :, 0], w[0, :, 1], w[0, 2, 3] = 0, 2.0 ** -101, float("nan")
        w[0, :, 4] = 1.0
        w[0, 1, 4] = 2.0
    codes, scales = moe.moe_int8_quantize_t(w)
    assert codes.shape == (batch, f, (k + 15) // 16 * 16) and scales.shape == (batch, f)
    want, ws = oracle.int8_quantize(_f64(w.transpose(1, 2).reshape(batch * f, k)))
    assert np.array_equal(codes[..., :k].cpu().numpy().reshape(batch * f, k), want)
    assert (codes[..., k:] == 0).all()
    assert np.array_equal(scales.cpu().numpy().reshape(-1), ws, equal_nan=True)
    assert torch.equal(moe.moe_int8_quantize_t(w, shuffle_seed=9)[0], codes)
    # the same as the rows of the transposed matrix
    rows = moe.moe_int8_quantize(w[-1].t().contiguous())
    assert torch.equal(rows[0], codes[-1])
    one = moe.moe_int8_quantize_t(w[-1].clone())
    assert one[0].shape == codes.shape[1:] and torch.equal(one[0], codes[-1])


# --------------------------------------------------------------------- products
def _weights(f, k, seed, experts=None):
    """Codes and scales of some weights; each code row holds its extremes."""
    rng = np.random.default_rng(seed)
    shape = (f, k) if experts is None else (experts, f, k)
    c = rng.integers(-127, 128, shape).astype(np.int8)
    k16 = (k + 15) // 16 * 16
    wide = np.zeros(shape[:-1] + (k16,), np.int8)
    wide[..., :k] = c
    s = (rng.random(shape[:-1]) * 0.9 + 0.1).astype(np.float32) / np.float32(127 * np.sqrt(k))
    return torch.from_numpy(wide).to(DEV), torch.from_numpy(s).to(DEV), c, s


LINEAR = [  # rows, K, F
    (1, 1, 1), (1, 2048, 2048), (2, 100, 3), (5, 48, 65), (16, 640, 257), (17, 33, 40), (32, 512, 130), (33, 64, 64), (37, 200, 1000),
    (63, 2000, 129), (64, 128, 256), (100, 4096, 90), (129, 1000, 513), (300, 96, 700), (517, 320, 1500), (1024, 256, 1024),
    (2100, 130, 520), (4096, 64, 300), (3, 9000, 17), (40, 17, 5),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,f", LINEAR)
def test_linear(rows, k, f, dtype):
    x = _values(rows, k, dtype, rows * k)
    x = (x / x.abs().amax(1, keepdim=True).float()).to(TYPE[dtype])
    w, ws, c, s = _weights(f, k, f)
    rng = np.random.default_rng(rows)
    vec = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(DEV).to(TYPE[dtype])  # noqa: E731
    bias, res = vec(f), vec(rows, f)
    cx, sx = oracle.int8_quantize(_f64(x))
    for act, b, r in (("none", None, None), ("gelu", bias, None), ("silu", bias, res), ("relu2", None, res), ("relu", bias, res)):
        y, z, scaled = oracle.int8_product(cx, sx, c, s, None if b is None else _f64(b), act, None if r is None else _f64(r))
        got = moe.moe_int8_linear(x, w, ws, bias=b, residual=r, act=act)
        assert got.dtype is TYPE[dtype] and got.shape == (rows, f)
        _check_y(got, y, z, scaled, act, None if r is None else _f64(r), dtype)
    # launch order, and codes that the caller has
    for seed in (3, 50):
        assert torch.equal(moe.moe_int8_linear(x, w, ws, bias=bias, residual=res, act="relu", shuffle_seed=seed), got)
    codes, scales = moe.moe_int8_quantize(x)
    assert torch.equal(moe.moe_int8_linear(codes, w, ws, x_scales=scales, bias=bias, residual=res, act="relu", out_dtype=TYPE[dtype]), got)
    # y is the residual, between other columns
    wide = torch.full((rows, f + 3), 7.0, dtype=TYPE[dtype], device=DEV)
    wide[:, 1:f + 1] = res
    moe.moe_int8_linear(x, w, ws, bias=bias, residual=wide[:, 1:f + 1], act="relu", y=wide[:, 1:f + 1])
    assert torch.equal(wide[:, 1:f + 1], got) and (wide[:, 0] == 7).all() and (wide[:, f + 1:] == 7).all()


@pytest.mark.parametrize("rows", [1, 20, 70, 300])
def test_linear_types_strides_and_shapes(rows):
    k, f = 200, 136
    w, ws, c, s = _weights(f, k, 1)
    x = _values(rows, k, "bf16", 3, wide=7).contiguous()
    y = moe.moe_int8_linear(x, w, ws, out_dtype=torch.float32)
    assert y.dtype is torch.float32
    cx, sx = oracle.int8_quantize(_f64(x))
    want, z, scaled = oracle.int8_product(cx, sx, c, s)
    _check_y(y, want, z, scaled, "none", None, "f32")
    assert torch.equal(moe.moe_int8_linear(x.float(), w, ws), y)
    assert torch.equal(moe.moe_int8_linear(_values(rows, k, "bf16", 3, wide=7), w, ws, out_dtype=torch.float32), y)
    assert torch.equal(moe.moe_int8_linear(x.reshape(rows, 1, k), w, ws, out_dtype=torch.float32).reshape(rows, f), y)
    codes, scales = moe.moe_int8_quantize(x)
    wide = torch.zeros((rows, codes.shape[1] + 32), dtype=torch.int8, device=DEV)
    wide[:, 16:16 + codes.shape[1]] = codes
    out = torch.empty_like(y)
    assert moe.moe_int8_linear(wide[:, 16:16 + codes.shape[1]], w, ws, x_scales=scales, y=out) is out
    assert torch.equal(out, y)
    assert moe.moe_int8_linear(codes, w, ws, x_scales=scales).dtype is torch.bfloat16
    assert moe.moe_int8_linear(x[:0], w, ws).shape == (0, f)


def test_largest_sums_are_exact():
    """127 * 127 * 131072: the largest sum, just below 2^31."""
    k = 1 << 17
    x = torch.full((3, k), 127, dtype=torch.int8, device=DEV)
    x[1] = -127
    w = torch.full((5, k), 127, dtype=torch.int8, device=DEV)
    w[2, 0] = 126
    one = torch.ones(5, device=DEV)
    for rows in (3, 40, 200):
        xs = x[:3].repeat((rows + 2) // 3, 1)[:rows].contiguous()
        y = moe.moe_int8_linear(xs, w, one, x_scales=torch.ones(rows, device=DEV), out_dtype=torch.float32)
        big = 127 * 127 * k
        want = np.array([[np.float32(big), np.float32(big - 127)][n == 2] for n in range(5)], dtype=np.float32)
        got = y.cpu().numpy()
        assert np.array_equal(got[0], want) and np.array_equal(got[1], -want) and np.array_equal(got[2], want)


def test_numbers_that_are_not_finite_stay_in_their_rows():
    for rows in (4, 50, 200):
        x = torch.randn(rows, 96, device=DEV).to(torch.bfloat16)
        w, ws, _, _ = _weights(70, 96, 2)
        y = moe.moe_int8_linear(x, w, ws)
        x[1, 5], x[3, 7] = float("inf"), float("nan")
        x[2] = 0
        z = moe.moe_int8_linear(x, w, ws)
        assert torch.isnan(z[1]).all() and torch.isnan(z[3]).all() and (z[2] == 0).all()
        keep = [i for i in range(rows) if i not in (1, 2, 3)]
        assert torch.equal(z[keep], y[keep])


EXPERTS = [  # rows of each expert (cycled), experts, K, F, rows behind the last
    ([1], 22, 64, 48, 0), ([0, 1, 0, 3], 512, 96, 40, 5), ([0], 7, 64, 64, 9), ([5, 0, 17, 40], 9, 130, 70, 3), ([16], 33, 256, 257, 0),
    ([300, 2, 0, 65], 4, 200, 300, 20), ([64, 100, 1], 12, 64, 520, 1), ([1000, 24], 2, 320, 260, 0), ([31, 33], 1024, 32, 24, 2),
    ([700], 1, 100, 100, 7), ([129, 500, 0], 6, 1100, 140, 0), ([1], 3, 4096, 100, 0),
    ([0, 20, 0, 0, 0, 0, 0, 1], 40, 2048, 72, 2), ([2, 0, 17], 30, 2040, 33, 1), ([3, 0], 9, 2064, 48, 1), ([1], 300, 64, 1500, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,experts,k,f,behind", EXPERTS)
def test_experts(counts, experts, k, f, behind, dtype):
    n = [counts[e % len(counts)] for e in range(experts)]
    offsets = np.concatenate(([0], np.cumsum(n)))
    rows = int(offsets[-1]) + behind
    x = _values(rows, k, dtype, rows)
    x = (x / x.abs().amax(1, keepdim=True).float()).to(TYPE[dtype])
    x[offsets[-1]:] = float("nan")                       # not read
    w, ws, c, s = _weights(f, k, experts, experts)
    rng = np.random.default_rng(rows)
    bias = torch.from_numpy(rng.standard_normal((experts, f)).astype(np.float32)).to(DEV).to(TYPE[dtype])
    off = torch.from_numpy(offsets.astype(np.int32)).to(DEV)
    cx, sx = oracle.int8_quantize(_f64(x[:offsets[-1]]))
    for act, b in (("relu2", None), ("silu", bias), ("none", bias)):
        y = torch.full((rows, f), 7.0, dtype=TYPE[dtype], device=DEV)
        assert moe.moe_int8_experts(x, w, ws, off, bias=b, act=act, y=y) is y
        assert (y[offsets[-1]:] == 7).all()
        for i0, i1, want, z, scaled in oracle.int8_experts(cx, sx, c, s, offsets, None if b is None else _f64(b), act):
            _check_y(y[i0:i1], want, z, scaled, act, None, dtype)
    last = int(offsets[-1])
    for seed in (4, 61):
        assert torch.equal(moe.moe_int8_experts(x, w, ws, off, bias=bias, shuffle_seed=seed)[:last], y[:last])
    codes, scales = moe.moe_int8_quantize(x)
    assert torch.equal(moe.moe_int8_experts(codes, w, ws, off, x_scales=scales, bias=bias, out_dtype=TYPE[dtype])[:last], y[:last])
    # one expert's rows alone give the same bits (whatever kernel takes them)
    e = int(np.argmax(n))
    if n[e]:
        part = slice(int(offsets[e]), int(offsets[e + 1]))
        assert torch.equal(moe.moe_int8_linear(x[part], w[e].contiguous(), ws[e].contiguous(), bias=bias[e]), y[part])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,f", [(4076, 300, 4074), (4096, 256, 4096), (1813, 1804, 3139), (1999, 897, 1543), (2119, 794, 2577),
                                      (519, 70, 5101)])
def test_large_products(rows, k, f, dtype):
    """Sizes that each of the larger tiles takes, whole tiles and ragged ones."""
    x = _values(rows, k, dtype, 8)
    x = (x / x.abs().amax(1, keepdim=True).float()).to(TYPE[dtype])
    w, ws, c, s = _weights(f, k, 4)
    rng = np.random.default_rng(1)
    bias = torch.from_numpy(rng.standard_normal(f).astype(np.float32)).to(DEV).to(TYPE[dtype])
    wide = torch.randn((rows, f + 3), device=DEV).to(TYPE[dtype])
    res = wide[:, 1:f + 1].clone()
    some = np.r_[0:3, 120:136, 250:260, rows - 70:rows]
    cx, sx = oracle.int8_quantize(_f64(x[some]))
    for act in ("gelu", "relu2"):
        r = res if act == "gelu" else None
        got = moe.moe_int8_linear(x, w, ws, bias=bias, residual=r, act=act)
        want, z, scaled = oracle.int8_product(cx, sx, c, s, _f64(bias), act, None if r is None else _f64(r[some]))
        _check_y(got[some], want, z, scaled, act, None if r is None else _f64(r[some]), dtype)
        # in pieces, which other kernels take
        for i in range(0, rows, 500):
            piece = moe.moe_int8_linear(x[i:i + 500], w, ws, bias=bias, residual=None if r is None else r[i:i + 500], act=act)
            assert torch.equal(got[i:i + 500], piece)
        assert torch.equal(moe.moe_int8_linear(x, w, ws, bias=bias, residual=r, act=act, shuffle_seed=5), got)
        if r is not None:   # y is the residual, between other columns
            edge = wide[:, [0, -2, -1]].clone()
            moe.moe_int8_linear(x, w, ws, bias=bias, residual=wide[:, 1:f + 1], act=act, y=wide[:, 1:f + 1])
            assert torch.equal(wide[:, 1:f + 1], got) and torch.equal(wide[:, [0, -2, -1]], edge)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,rows,k,f", [(1, 4076, 300, 4074), (3, 2878, 1155, 5053), (3, 2796, 658, 2631), (3, 2824, 909, 1105),
                                              (3, 2999, 929, 1731), (3, 1016, 62, 2569)])
def test_large_products_of_experts(experts, rows, k, f, dtype):
    """The same by expert: the bits of the experts' products one by one, and nothing behind the last row."""
    x = _values(rows, k, dtype, 9)
    w, ws, _, _ = _weights(f, k, 6, experts)
    bias = torch.randn((experts, f), device=DEV).to(TYPE[dtype])
    cuts = [0, rows - 7] if experts == 1 else [0, rows // 3, rows // 3 + 1, rows - 7]
    y = torch.full((rows, f), 7.0, dtype=TYPE[dtype], device=DEV)
    moe.moe_int8_experts(x, w, ws, torch.tensor(cuts, dtype=torch.int32, device=DEV), bias=bias, act="relu2", y=y)
    assert (y[cuts[-1]:] == 7).all()
    for e in range(experts):
        for i in range(cuts[e], cuts[e + 1], 500):
            part = slice(i, min(i + 500, cuts[e + 1]))
            assert torch.equal(y[part], moe.moe_int8_linear(x[part], w[e], ws[e], bias=bias[e], act="relu2"))


@pytest.mark.parametrize("rows", [6, 200])
def test_offsets_out_of_range_touch_nothing_else(rows):
    """Offsets below 0, past the rows or descending: no row outside the matrices is touched."""
    w, ws, _, _ = _weights(40, 64, 3, 4)
    x = torch.randn(rows, 64, device=DEV)
    room = torch.full((3 * rows, 40), 7.0, device=DEV)
    for off in ([-5, 2, 2, 2, 2], [0, 3, rows + 1000, rows + 2000, 2 ** 31 - 1], [0, 5, 1, 3, 4], [-2 ** 31, -1, 0, 0, 0]):
        moe.moe_int8_experts(x, w, ws, torch.tensor(off, dtype=torch.int32, device=DEV), y=room[rows:2 * rows])
        assert (room[:rows] == 7).all() and (room[2 * rows:] == 7).all()


# ---------------------------------------------------- streams, graphs, overlap
@pytest.mark.parametrize("tokens", [1, 9, 700])
def test_streams_and_graphs(tokens):
    k, f, experts = 264, 200, 6
    w, ws, _, _ = _weights(f, k, 1)
    we, wse, _, _ = _weights(f, k, 2, experts)
    g = torch.Generator(device=DEV).manual_seed(3)
    new = lambda: dict(x=torch.randn((tokens, k), generator=g, device=DEV).to(torch.bfloat16),  # noqa: E731
                       idx=torch.randint(0, experts, (tokens, 2), generator=g, device=DEV, dtype=torch.int32))

    def step(c):
        slot_row, offsets, _ = moe.moe_sort(c["idx"], experts)
        rows = moe.moe_permute_fwd(c["x"], slot_row)
        return moe.moe_int8_linear(c["x"], w, ws, act="gelu"), moe.moe_int8_experts(rows, we, wse, offsets, act="relu2")

    a, b = new(), new()
    want = [step(a), step(b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            o1 = step(a)
        with torch.cuda.stream(s2):
            o2 = step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(o1 + o2, want[0] + want[1]))
    c = {n: t.clone() for n, t in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c)
    for inputs, wanted in ((a, want[0]), (b, want[1]), (a, want[0])):
        for n in c:
            c[n].copy_(inputs[n])
        for t in out:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, wanted))
        step(inputs)
        torch.cuda.synchronize()


def test_weights_beyond_2gib():
    """The last of 260 experts of 4096 x 2304 (2.4 GB of codes)."""
    experts, k, f = 260, 2304, 4096
    w = torch.zeros((experts, f, k), dtype=torch.int8, device=DEV)
    last, ws, c, s = _weights(f, k, 5)
    w[-1] = last
    scale = torch.ones((experts, f), device=DEV)
    scale[-1] = ws
    for rows in (3, 6000):
        x = _values(rows, k, "bf16", 1)
        x = x / x.abs().amax(1, keepdim=True)
        off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
        off[-1] = rows
        y = moe.moe_int8_experts(x, w, scale, off)
        assert torch.equal(y, moe.moe_int8_linear(x, last, ws))
        some = slice(0, 3)
        cx, sx = oracle.int8_quantize(_f64(x[some]))
        want, z, scaled = oracle.int8_product(cx, sx, c, s)
        _check_y(y[some], want, z, scaled, "none", None, "bf16")


# ----------------------------------------------------------- the pieces together
@pytest.mark.parametrize("tokens,k,experts,d,f", [(1, 4, 16, 256, 128), (70, 3, 9, 200, 96), (600, 2, 5, 128, 264)])
def test_expert_layer_from_its_pieces(tokens, k, experts, d, f):
    """A layer as a user puts it together: sort, rows to the experts, both
    products in 8-bit integers, rows back with weights, dropout into the
    residual stream; each piece against its definition on the pieces' own inputs."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    bf = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    x = bf(tokens, d)
    score = torch.sigmoid(torch.randn((tokens, experts), generator=g, device=DEV))
    top = score.topk(k, dim=1)                                   # a router of the user's own, int64 numbers
    prob = top.values / top.values.sum(1, keepdim=True)
    w1 = moe.moe_int8_quantize_t(bf(experts, d, f))
    w2 = moe.moe_int8_quantize_t(bf(experts, f, d))
    slot_row, offsets, row_src = moe.moe_sort(top.indices, experts, need_row_src=True)
    codes, scales = moe.moe_int8_quantize(x)
    rows = moe.moe_permute_fwd(codes, slot_row)                  # the tokens travel as codes
    row_scales = moe.moe_permute_fwd(scales[:, None], slot_row)
    h = moe.moe_int8_experts(rows, *w1, offsets, x_scales=row_scales, act="relu2")
    o = moe.moe_int8_experts(h, *w2, offsets)
    y = moe.moe_unpermute_fwd(o, slot_row, prob)
    rng = torch.tensor([5, 0], dtype=torch.int64, device=DEV)
    z = moe.moe_dropout_fwd(y, 0.1, rng, residual=x)
    off = offsets.cpu().numpy()
    src = row_src.cpu().numpy()
    assert off[-1] == tokens * k
    cx, sx = oracle.int8_quantize(_f64(x))
    w64 = [(c.cpu().numpy()[..., :n], s.cpu().numpy()) for (c, s), n in ((w1, d), (w2, f))]
    for i0, i1, want, zz, scaled in oracle.int8_experts(cx[src // k], sx[src // k], *w64[0], off, None, "relu2"):
        _check_y(h[i0:i1], want, zz, scaled, "relu2", None, "bf16")
    ch, sh = oracle.int8_quantize(_f64(h))
    for i0, i1, want, zz, scaled in oracle.int8_experts(ch, sh, *w64[1], off):
        _check_y(o[i0:i1], want, zz, scaled, "none", None, "bf16")
    want, size = oracle.sum_rows(_f64(o), slot_row.cpu().numpy(), _f64(prob))
    assert (np.abs(_f64(y) - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * 2 * E * size).all()
    kept = oracle.dropout_mask(tokens * d, 0.1, 5, 0).reshape(tokens, d)
    want = np.where(kept, _f64(y) / 0.9, 0) + _f64(x)
    assert (np.abs(_f64(z) - want) <= 2.0 ** -8 * np.abs(want) + 4 * E * (np.abs(_f64(y)) / 0.9 + np.abs(_f64(x)))).all()


def test_the_largest_grids():
    """The most rows and matrices that the quantisers take: 2^24 - 8 workgroups of four rows, 2^23 - 8 of a matrix."""
    rows = 4 * ((1 << 24) - 8)
    x = torch.ones((rows, 1), dtype=torch.bfloat16, device=DEV)
    x[-1], x[rows // 2] = -2, 0
    codes, scales = moe.moe_int8_quantize(x)
    assert int((codes[:, 0] == 127).sum()) == rows - 2 and int(codes[-1, 0]) == -127 and int(codes[rows // 2, 0]) == 0
    assert not codes[:, 1:].any() and scales[-1].item() == np.float32(2) / np.float32(127) and scales[rows // 2].item() == 0
    del x, codes, scales
    batch = (1 << 23) - 8
    w = torch.ones((batch, 1, 2), dtype=torch.bfloat16, device=DEV)
    w[-1, 0, 1], w[batch // 2, 0, 0] = -2, 0
    codes, scales = moe.moe_int8_quantize_t(w)
    assert int((codes[..., 0] == 127).sum()) == 2 * batch - 2 and int(codes[-1, 1, 0]) == -127 and int(codes[batch // 2, 0, 0]) == 0
    assert not codes[..., 1:].any() and scales[-1, 1].item() == np.float32(2) / np.float32(127)
    with pytest.raises(moe.MoeError, match="status 2"):
        moe.moe_int8_quantize_t(torch.ones((batch + 1, 1, 2), dtype=torch.bfloat16, device=DEV))
