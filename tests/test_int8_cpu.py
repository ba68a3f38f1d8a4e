"""The oracle of the products in 8-bit integers, and what their entry points
refuse (before any GPU call, so this runs without a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import int8_cases
import oracle


def test_codes_against_exact_fractions():
    rng = np.random.default_rng(0)
    for bits in (8, 24):
        x = rng.standard_normal((20, 64)).astype(np.float32)
        if bits == 8:
            x = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        # ties: half of the largest, and odd multiples of a largest number of 254 units
        x[3, :4], x[4, :3] = (2.0, 1.0, -1.0, 0.5), (254.0, 3.0, -125.0)
        x[4, 3:] = rng.integers(-127, 128, 61) * 2 + 1
        x[4, 3:] = np.clip(x[4, 3:], -253, 253)
        codes, scales = oracle.int8_quantize(x)
        for i in range(20):
            top = np.abs(x[i]).max()
            assert scales[i] == np.float32(top) / np.float32(127)
            assert [oracle.int8_code_exact(v, top) for v in x[i]] == codes[i].tolist()
    assert oracle.int8_quantize(np.array([[2.0, 1.0, -1.0]]))[0].tolist() == [[127, 64, -64]]


def test_codes_of_zeros_and_numbers_that_are_not_finite():
    tiny = 2.0 ** -101
    codes, scales = oracle.int8_quantize(np.array([[0.0, 0.0], [tiny, -tiny], [2.0 ** -100, 0], [np.inf, 1], [np.nan, 1]]))
    assert codes.tolist() == [[0, 0], [0, 0], [127, 0], [0, 0], [0, 0]]
    assert scales[0] == scales[1] == 0 and scales[2] > 0 and np.isnan(scales[3:]).all()


def test_product_of_the_codes_is_near_the_product():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((9, 50)), rng.standard_normal((50, 7))
    cx, sx = oracle.int8_quantize(x)
    cw, sw = oracle.int8_quantize(w.T)
    y, z, s = oracle.int8_product(cx, sx, cw, sw)
    # each factor is off by at most half a step, its scale by its rounding
    ex, ew = 0.5001 * sx[:, None].astype(float), 0.5001 * sw.astype(float)
    bound = ex * np.abs(w).sum(0) + (np.abs(x) + ex).sum(1)[:, None] * ew
    assert (np.abs(y - x @ w) <= bound).all()
    parts = oracle.int8_experts(cx, sx, np.stack([cw, cw[::-1]]), np.stack([sw, sw[::-1]]), [0, 4, 9])
    assert np.array_equal(parts[0][2], y[:4]) and np.array_equal(parts[1][2], y[4:, ::-1])


# ------------------------------------------------------------------- refusals
def _t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


I8, F32, I32 = torch.int8, torch.float32, torch.int32
W, S = (lambda *s: _t(*s, dtype=I8)), (lambda *s: _t(*s, dtype=F32))
BAD = [
    (lambda: moe.moe_int8_quantize(_t(4, 8, dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: moe.moe_int8_quantize(torch.zeros(())), "columns"),
    (lambda: moe.moe_int8_quantize(_t(8, 4).t()), "unit stride"),
    (lambda: moe.moe_int8_quantize(_t(4, 8), codes=W(4, 8)), "codes"),
    (lambda: moe.moe_int8_quantize(_t(4, 8), scales=S(3)), "scales"),
    (lambda: moe.moe_int8_quantize(S(1, (1 << 17) + 1)), "GPU|status 2"),
    (lambda: moe.moe_int8_quantize(_t(4, 8)), "GPU"),
    (lambda: moe.moe_int8_quantize_t(_t(8)), "matrices"),
    (lambda: moe.moe_int8_quantize_t(_t(8, 4).t()), "matrices"),
    (lambda: moe.moe_int8_quantize_t(_t(2, 8, 4), codes=W(2, 4, 8)), "codes"),
    (lambda: moe.moe_int8_quantize_t(_t(2, 8, 4), scales=S(4)), "scales"),
    (lambda: moe.moe_int8_quantize_t(_t(2, 8, 4)), "GPU"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 20), S(6)), "w_codes"),
    (lambda: moe.moe_int8_linear(_t(4, 20), S(6, 32), S(6)), "w_codes"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(32, 6).t(), S(6)), "w_codes"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(1, 6, 32), S(6)), "w_codes"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(5)), "w_scales"),
    (lambda: moe.moe_int8_linear(_t(4, 20, dtype=torch.float16), W(6, 32), S(6)), "float32 or bfloat16"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6), x_scales=S(4)), "together"),
    (lambda: moe.moe_int8_linear(W(4, 32), W(6, 32), S(6)), "together"),
    (lambda: moe.moe_int8_linear(W(4, 32), W(6, 32), S(6), x_scales=S(3)), "x_scales"),
    (lambda: moe.moe_int8_linear(W(4, 20), W(6, 32), S(6), x_scales=S(4)), "status 2"),
    (lambda: moe.moe_int8_linear(W(4, 40)[:, :32], W(6, 32), S(6), x_scales=S(4)), "status 2"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6), bias=S(6)), "bias"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6), residual=_t(4, 5)), "residual"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6), y=_t(4, 5)), "y"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6), act="tanh"), "act"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6), out_dtype=torch.float16), "output"),
    (lambda: moe.moe_int8_linear(_t(4, 20), W(6, 32), S(6)), "GPU"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(3, 6, 32), S(3, 6), None), "offsets"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(6, 32), S(6), _t(2, dtype=I32)), "w_codes"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(0, 6, 32), S(0, 6), _t(1, dtype=I32)), "w_codes"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(3, 6, 32), S(3, 6), _t(3, dtype=I32)), "offsets"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(3, 6, 32), S(3, 6), _t(4, dtype=torch.int64)), "offsets"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(3, 6, 32), S(2, 6), _t(4, dtype=I32)), "w_scales"),
    (lambda: moe.moe_int8_experts(_t(2, 2, 20), W(3, 6, 32), S(3, 6), _t(4, dtype=I32)), "matrix"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(1025, 6, 32), S(1025, 6), _t(1026, dtype=I32)), "status 2"),
    (lambda: moe.moe_int8_experts(_t(4, 20), W(3, 6, 32), S(3, 6), _t(4, dtype=I32)), "GPU"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    call, says = BAD[i]
    with pytest.raises(moe.MoeError, match=says):
        call()


OK, NULL, SHAPE, DTYPE, WS, MODE = 0, 1, 2, 3, 4, 5
A = 0x10000   # an address that is not followed: the calls return before any launch


def _product(experts=False, **o):
    a = dict(rows=40, d_in=32, d_out=6, num_local=3 if experts else 0, x_dtype=1, dtype=1, act=0, ldx=32, ldy=6, ldr=6, x=A, xs=None,
             w=A, ws_=A, bias=None, res=None, off=A, y=A, wk=A, nb=1 << 20)
    a.update(o)
    c = moe._CInt8(a["rows"], a["d_in"], a["d_out"], a["num_local"], a["x_dtype"], a["dtype"], a["act"], a["ldx"], a["ldy"], a["ldr"], 0)
    lib = moe.load_library()
    if experts:
        return lib.moe_int8_experts(ctypes.byref(c), a["x"], a["xs"], a["w"], a["ws_"], a["bias"], a["off"], a["y"], a["wk"], a["nb"], None)
    return lib.moe_int8_linear(ctypes.byref(c), a["x"], a["xs"], a["w"], a["ws_"], a["bias"], a["res"], a["y"], a["wk"], a["nb"], None)


CASES = [
    (DTYPE, dict(x_dtype=2)), (DTYPE, dict(x_dtype=3)), (DTYPE, dict(dtype=6)), (MODE, dict(act=5)), (MODE, dict(act=-1)),
    (SHAPE, dict(rows=-1)), (SHAPE, dict(rows=1 << 31)), (SHAPE, dict(d_in=0)), (SHAPE, dict(d_in=(1 << 17) + 1, ldx=1 << 18)),
    (SHAPE, dict(d_out=0)), (SHAPE, dict(d_out=1 << 20, ldy=1 << 20)), (SHAPE, dict(ldx=31)), (SHAPE, dict(ldy=5)),
    (SHAPE, dict(ldx=1 << 20)), (SHAPE, dict(ldr=-1)), (SHAPE, dict(x_dtype=6, xs=A, d_in=20)), (SHAPE, dict(x_dtype=6, xs=A, ldx=40)),
    (SHAPE, dict(x_dtype=6, xs=A, x=A + 8)), (NULL, dict(x_dtype=6)), (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(ws_=None)),
    (NULL, dict(y=None)), (NULL, dict(wk=None)), (WS, dict(nb=16)), (WS, dict(wk=A + 16)), (SHAPE, dict(x=A + 1)), (SHAPE, dict(w=A + 8)),
    (SHAPE, dict(ws_=A + 2)), (SHAPE, dict(y=A + 1)), (SHAPE, dict(bias=A + 1)), (OK, dict(rows=0, x=None, w=None, y=None, wk=None)),
    (SHAPE, dict(rows=(1 << 31) - 1, d_out=(1 << 20) - 1, ldy=(1 << 20) - 1, nb=1 << 50)),
    (SHAPE, dict(rows=1 << 26, nb=1 << 50)),   # quantising them
]


@pytest.mark.parametrize("experts", [False, True])
@pytest.mark.parametrize("status,o", CASES)
def test_product_status(experts, status, o):
    assert _product(experts, **o) == status


def test_product_status_of_one_kind():
    assert _product(num_local=3) == SHAPE and _product(True, num_local=0) == SHAPE and _product(True, num_local=1025) == SHAPE
    assert _product(True, off=None) == NULL and _product(True, off=A + 2) == SHAPE
    assert _product(res=A, ldr=5) == SHAPE and _product(res=A + 1) == SHAPE
    lib = moe.load_library()
    assert lib.moe_int8_linear(None, A, None, A, A, None, None, A, A, 1 << 20, None) == NULL
    assert lib.moe_int8_workspace_size(None, None) == NULL
    assert moe.moe_int8_workspace_size(50, 100, 7) >= 50 * 112 + 50 * 4
    assert moe.moe_int8_workspace_size(2, 100, 7) == 0     # quantised by the product itself
    assert moe.moe_int8_workspace_size(2, 100, 7, 3) == 0
    assert moe.moe_int8_workspace_size(2, 3000, 7, 3) > 0
    for bad in (dict(dtype="u8"), dict(out_dtype="i8")):
        with pytest.raises(moe.MoeError, match="x is f32, bf16 or i8"):
            moe.moe_int8_workspace_size(5, 100, 7, **bad)
    with pytest.raises(moe.MoeError, match="act must be"):
        moe.moe_int8_workspace_size(5, 100, 7, act="tanh")
    assert moe.moe_int8_workspace_size(5, 112, 7, dtype="i8") == 0


@pytest.mark.parametrize("x_dtype,out_dtype", [("bf16", None), ("bf16", "f32"), ("f32", None), ("f32", "bf16"), ("i8", None), ("i8", "f32")])
def test_workspace_size_of_every_call(x_dtype, out_dtype):
    """The size asked for is the one that the call needs, for every type and activation."""
    code = {"f32": 0, "bf16": 1, "i8": 6}
    out = code[out_dtype or ("bf16" if x_dtype == "i8" else x_dtype)]
    lib, n = moe.load_library(), ctypes.c_size_t()
    for rows, k, f, local in ((1, 64, 8, 0), (4, 2048, 2048, 0), (17, 8192, 64, 0), (64, 8192, 512, 0), (300, 4096, 4096, 0), (22, 2048, 2048, 512)):
        for a, act in enumerate(("none", "relu", "relu2", "silu", "gelu")):
            c = moe._CInt8(rows, k, f, local, code[x_dtype], out, a, k, f, 0, 0)
            assert lib.moe_int8_workspace_size(ctypes.byref(c), ctypes.byref(n)) == OK
            assert moe.moe_int8_workspace_size(rows, k, f, local, x_dtype, act, out_dtype) == n.value
    # x of another type than the output is quantised by a launch of its own
    assert (moe.moe_int8_workspace_size(1, 64, 8, 0, x_dtype, "none", out_dtype) > 0) == (x_dtype != "i8" and code[x_dtype] != out)


@pytest.mark.parametrize("status,o", [
    (DTYPE, dict(dt=6)), (SHAPE, dict(rows=-1)), (SHAPE, dict(rows=1 << 31)), (SHAPE, dict(cols=0)), (SHAPE, dict(cols=(1 << 17) + 1, ld=1 << 18)),
    (SHAPE, dict(ld=7)), (NULL, dict(x=None)), (NULL, dict(c=None)), (NULL, dict(s=None)), (SHAPE, dict(x=A + 1)), (SHAPE, dict(c=A + 8)),
    (SHAPE, dict(s=A + 2)), (SHAPE, dict(rows=1 << 30, ld=1 << 20)), (OK, dict(rows=0, x=None)),
    # more than 2^24 workgroups: four rows each, or one of many columns
    (SHAPE, dict(rows=1 << 26)), (SHAPE, dict(rows=1 << 24, cols=8192, ld=8192)),
])
def test_quantize_status(status, o):
    a = dict(x=A, dt=1, rows=4, cols=8, ld=8, c=A, s=A)
    a.update(o)
    assert moe.load_library().moe_int8_quantize(a["x"], a["dt"], a["rows"], a["cols"], a["ld"], a["c"], a["s"], 0, None) == status


@pytest.mark.parametrize("status,o", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(batch=-1)), (SHAPE, dict(rows=0)), (SHAPE, dict(rows=(1 << 17) + 1)), (SHAPE, dict(cols=0)),
    (SHAPE, dict(cols=1 << 20)), (SHAPE, dict(batch=1 << 30)), (NULL, dict(x=None)), (NULL, dict(c=None)), (NULL, dict(s=None)),
    (SHAPE, dict(x=A + 1)), (SHAPE, dict(c=A + 4)), (SHAPE, dict(s=A + 1)), (OK, dict(batch=0, x=None)),
    (SHAPE, dict(batch=1 << 23)),   # workgroups of 512 threads
])
def test_quantize_t_status(status, o):
    a = dict(x=A, dt=1, batch=2, rows=8, cols=8, c=A, s=A)
    a.update(o)
    assert moe.load_library().moe_int8_quantize_t(a["x"], a["dt"], a["batch"], a["rows"], a["cols"], a["c"], a["s"], 0, None) == status


# The last size inside the grid's limit and the first one outside; a pointer is missing, so that neither is launched.
LIMIT = (1 << 24) - 8


def test_grid_limits_of_the_quantisers():
    lib = moe.load_library()
    for rows, cols in ((4 * LIMIT, 8), (4 * LIMIT, 4096), (LIMIT, 4097)):      # four rows a workgroup, or one
        assert lib.moe_int8_quantize(None, 1, rows, cols, cols, A, A, 0, None) == NULL
        assert lib.moe_int8_quantize(None, 1, rows + 1, cols, cols, A, A, 0, None) == SHAPE
    most = (1 << 23) - 8
    for batch, cols in ((most, 64), (most // 8, 512)):                          # 64 columns a workgroup
        assert lib.moe_int8_quantize_t(None, 1, batch, 8, cols, A, A, 0, None) == NULL
        assert lib.moe_int8_quantize_t(None, 1, batch + 1, 8, cols, A, A, 0, None) == SHAPE


@pytest.mark.parametrize("x_dtype", ["i8", "bf16"])
@pytest.mark.parametrize("k,f,local", [(16, 16, 0), (2048, 2048, 0), (8192, 8192, 0), (16, 16, 8), (2048, 2048, 64)])
def test_grid_limits_of_the_products(x_dtype, k, f, local):
    def fits(rows):
        try:
            moe.moe_int8_workspace_size(rows, k, f, local, x_dtype)
            return True
        except moe.MoeError as e:
            assert "status 2" in str(e)
            return False

    lo, hi = 1, (1 << 31) - 1
    assert fits(lo) and not fits(hi)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if fits(mid) else (lo, mid)
    name = moe.moe_int8_stage_names(lo, k, f, local, x_dtype)[-1]
    bm, bn = (int(n) for n in name.split("_")[1].split("x"))
    units = lambda rows: (rows // bm + max(local, 1)) * ((f + bn - 1) // bn)  # noqa: E731
    # quantised four rows a workgroup, or one of more than 4096 columns
    quantised = lambda rows: 0 if x_dtype == "i8" else (rows + 3) // 4 if k <= 4096 else rows  # noqa: E731
    assert units(lo) <= LIMIT and quantised(lo) <= LIMIT
    assert units(hi) > LIMIT or quantised(hi) > LIMIT


# --------------------------------------------------------------------- kernels
def test_cases_reach_every_kernel():
    for kernel, *case in int8_cases.LINEAR:
        assert int8_cases.linear_kernel(*case) == "linear_" + kernel
    for kernel, *case in int8_cases.EXPERTS:
        assert int8_cases.experts_kernel(*case) == "experts_" + kernel
    want = {(k, t) for k in int8_cases.FEW + int8_cases.TILES for t in ("bf16", "f32")}
    assert {c[:2] for c in int8_cases.EXPERTS} == want
    assert {c[:2] for c in int8_cases.LINEAR} == want | {(k, t) for k in int8_cases.SPLITS for t in ("bf16", "f32")}
    # more than the eight steps of 64 codes that a wave has in flight, on every weight stream of both kinds (but the
    # one whose 2048 codes of a row are eight steps at most)
    for cases, at in ((int8_cases.LINEAR, 3), (int8_cases.EXPERTS, 4)):
        for kernel in int8_cases.FEW:
            if cases is int8_cases.LINEAR or kernel != "few4_quantize":
                assert any(c[0] == kernel and c[at] > 64 * 8 * int(kernel[3]) for c in cases), kernel
    # chunks of uneven numbers of slices, the last slice not full
    for kernel, _, _, k, _, _ in int8_cases.LINEAR:
        if "_split" in kernel:
            k16 = (k + 15) // 16 * 16
            assert (k16 + 127) // 128 % int(kernel[-1]) and k16 % 128, (kernel, k)


def test_stage_names():
    names = moe.moe_int8_stage_names
    assert names(0, 64, 96) == [] and names(0, 64, 96, 4, "i8") == []
    assert names(1, 2048, 2048) == ["linear_few4_quantize"] and names(5, 2048, 2048) == ["quantize", "linear_few4"]
    assert names(1, 2048, 2048, out_dtype="f32") == ["quantize", "linear_few4"] and names(1, 2048, 2048, dtype="i8") == ["linear_few4"]
    assert names(37, 2048, 8192, act="silu") == ["quantize", "linear_64x64_deep"]
    assert names(4096, 2048, 8192, act="gelu") == ["quantize", "linear_256x256"]
    assert names(4096, 2048, 8192, dtype="i8", act="gelu") == ["linear_256x256"]
    assert names(22, 2048, 2048, 512, act="relu2") == ["experts_few1_quantize"]
    assert names(8192, 1024, 2048, 8, act="relu2") == ["quantize", "experts_128x128"]
    assert names(110, 7513, 5499) == ["quantize", "linear_64x64_deep_split2", "join"]
    lib, b = moe.load_library(), ctypes.create_string_buffer(64)
    c = moe._CInt8(40, 32, 6, 0, 1, 1, 0, 32, 6, 0, 0)
    assert lib.moe_int8_stage_names(c, None, 64) == NULL and lib.moe_int8_stage_names(None, b, 64) == NULL
    assert lib.moe_int8_stage_names(c, b, 0) == WS and lib.moe_int8_stage_names(c, b, 8) == WS
    n = len(",".join(names(40, 32, 6)))
    assert lib.moe_int8_stage_names(c, b, n) == WS and lib.moe_int8_stage_names(c, b, n + 1) == OK
    with pytest.raises(moe.MoeError, match="status 2"):
        names(4, 8, 8, 1025)
    with pytest.raises(moe.MoeError, match="moe_int8_stage_names: x is f32"):
        names(4, 8, 8, dtype="u8")
