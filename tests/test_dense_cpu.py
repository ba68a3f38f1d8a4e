"""The dense operators' oracle against differences, and what their entry
points refuse (all before any GPU call, so this runs without a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import dense_cases
import oracle

ACTS = list(moe.ACTIVATIONS)


# ---------------------------------------------------------------------- oracle
def _differences(f, x, v, s=1e-6):
    return (f(x + s * v) - f(x - s * v)) / (2 * s)


@pytest.mark.parametrize("name", ACTS)
def test_oracle_activation_derivative(name):
    z = np.linspace(-4, 4, 41) + 0.013   # no kink within a step
    d = _differences(lambda t: oracle.act(name, t)[0], z, np.ones_like(z))
    # truncation s^2 |act'''| / 6 < 1e-11, rounding 2^-52 * 16 / s < 4e-9
    assert np.abs(oracle.act(name, z)[1] - d).max() < 1e-8


@pytest.mark.parametrize("name", ACTS)
def test_oracle_gradients_against_differences(name):
    rng = np.random.default_rng(2)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    x, w, w2, b, res, dy, nw, nb, dn = r(5, 7), r(7, 6), r(7, 6), r(6), r(5, 6), r(5, 6), r(7), r(7), r(5, 7)
    y, z = oracle.linear_forward(x, w, b, res, name)
    dx, dw, db = oracle.linear_backward(dy, x, w, z, name)
    loss = lambda x, w, b: (oracle.linear_forward(x, w, b, res, name)[0] * dy).sum()  # noqa: E731
    for g, f, at in ((dx, lambda t: loss(t, w, b), x), (dw, lambda t: loss(x, t, b), w), (db, lambda t: loss(x, w, t), b)):
        v = r(*at.shape)
        assert abs((g * v).sum() - _differences(f, at, v)) < 1e-6 * (1 + np.abs(g * v).sum())
    a, g, u = oracle.glu_forward(x, w, w2, name)
    dx, dwg, dwu = oracle.glu_backward(dy, x, w, w2, g, u, name)
    loss = lambda x, w, w2: (oracle.glu_forward(x, w, w2, name)[0] * dy).sum()  # noqa: E731
    for g, f, at in ((dx, lambda t: loss(t, w, w2), x), (dwg, lambda t: loss(x, t, w2), w), (dwu, lambda t: loss(x, w, t), w2)):
        v = r(*at.shape)
        assert abs((g * v).sum() - _differences(f, at, v)) < 1e-6 * (1 + np.abs(g * v).sum())
    dx, dnw, dnb = oracle.layernorm_backward(dn, x, nw, 1e-5)
    loss = lambda x, nw, nb: (oracle.layernorm_forward(x, nw, nb, 1e-5)[0] * dn).sum()  # noqa: E731
    for g, f, at in ((dx, lambda t: loss(t, nw, nb), x), (dnw, lambda t: loss(x, t, nb), nw), (dnb, lambda t: loss(x, nw, t), nb)):
        v = r(*at.shape)
        assert abs((g * v).sum() - _differences(f, at, v)) < 1e-6 * (1 + np.abs(g * v).sum())


# ------------------------------------------------------------------- refusals
def _t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


NORM_BAD = [
    (lambda: moe.moe_layernorm_fwd(_t(4, 8, dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), weight=_t(7)), "weight"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), bias=_t(8, dtype=torch.float32)), "bias"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), eps=-1.0), "eps"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), eps=float("nan")), "eps"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), eps=float("inf")), "eps"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), y=_t(4, 7)), "y"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8), mean=_t(4)), "mean"),
    (lambda: moe.moe_layernorm_fwd(_t(8, 4).t()), "unit stride"),
    (lambda: moe.moe_layernorm_fwd(_t(1, 8).expand(4, 8)), "unit stride"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 4, 8)[:, ::2]), "contiguous"),
    (lambda: moe.moe_layernorm_fwd(torch.zeros((), dtype=torch.float32)), "dimension"),
    (lambda: moe.moe_layernorm_fwd(_t(4, 8)), "GPU"),
    (lambda: moe.moe_layernorm_bwd(_t(4, 8), _t(4, 8), None, torch.zeros(4), torch.zeros(3)), "rstd"),
    (lambda: moe.moe_layernorm_bwd(_t(3, 8), _t(4, 8), None, torch.zeros(4), torch.zeros(4)), "rows"),
    (lambda: moe.moe_layernorm_bwd(_t(4, 8), _t(4, 8), None, torch.zeros(4), torch.zeros(4), dx_add=_t(4, 9)), "dx_add"),
    (lambda: moe.moe_layernorm_bwd(_t(4, 8), _t(4, 8), None, torch.zeros(4), torch.zeros(4)), "GPU"),
    (lambda: moe.moe_layernorm_workspace_size(4, 16385), "status 2"),
    (lambda: moe.moe_layernorm_workspace_size(-1, 8), "status 2"),
]
LIN_BAD = [
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(9, 6)), "x"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6, dtype=torch.float32)), "weight"),
    (lambda: moe.moe_linear_fwd(_t(4, 8, dtype=torch.float64), _t(8, 6, dtype=torch.float64)), "float32 or bfloat16"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8)), "d_in, d_out"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 0)), "without elements"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(6, 8).t()), "unit stride"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), act="tanh"), "act"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), act=None), "act"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), bias=_t(5)), "bias"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), residual=_t(1, 6).expand(4, 6)), "unit stride"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), residual=_t(3, 6)), "rows"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), z=_t(4, 6, dtype=torch.float16)), "z"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6), y=_t(4, 6, dtype=torch.float32)), "y"),
    (lambda: moe.moe_linear_fwd(_t(4, 8), _t(8, 6)), "GPU"),
    (lambda: moe.moe_linear_bwd(_t(4, 6), _t(4, 8), _t(8, 6), act="gelu"), "saved z"),
    (lambda: moe.moe_linear_bwd(_t(4, 6), _t(4, 8), _t(8, 6), grad_dtype=torch.float16), "grad_dtype"),
    (lambda: moe.moe_linear_bwd(_t(4, 6), _t(4, 8), _t(8, 6), dw=_t(8, 6)), "dw"),
    (lambda: moe.moe_linear_bwd(_t(4, 5), _t(4, 8), _t(8, 6)), "dy"),
    (lambda: moe.moe_linear_bwd(_t(4, 6), _t(4, 8), _t(8, 6), dx_add=_t(4, 6)), "dx_add"),
    (lambda: moe.moe_linear_bwd(_t(4, 6), _t(4, 8), _t(8, 6)), "GPU"),
    (lambda: moe.moe_glu_fwd(_t(4, 8), _t(8, 6), _t(8, 5)), "wu"),
    (lambda: moe.moe_glu_fwd(_t(4, 8), _t(8, 6), _t(8, 7)[:, :6]), "row distance"),
    (lambda: moe.moe_glu_fwd(_t(4, 8), _t(8, 6), _t(8, 6), g=_t(4, 6)), "together"),
    (lambda: moe.moe_glu_fwd(_t(4, 8), _t(8, 6), _t(8, 6), g=_t(4, 6), u=_t(4, 6, dtype=torch.float32)), "same type"),
    (lambda: moe.moe_glu_fwd(_t(4, 8), _t(8, 6), _t(8, 6)), "GPU"),
    (lambda: moe.moe_glu_bwd(_t(4, 6), _t(4, 8), _t(8, 6), _t(8, 6), _t(4, 6), _t(3, 6)), "rows"),
    (lambda: moe.moe_glu_bwd(_t(4, 6), _t(4, 8), _t(8, 6), _t(8, 6), _t(4, 6), _t(4, 6)), "GPU"),
    (lambda: moe.moe_linear_workspace_size(-1, 8, 8), "status 2"),
    (lambda: moe.moe_linear_workspace_size(8, 0, 8), "status 2"),
    (lambda: moe.moe_linear_workspace_size(8, 1 << 16, 1 << 15), "status 2"),   # 4 GiB of bf16 weights
    (lambda: moe.moe_linear_workspace_size(1 << 31, 8, 8), "2\\^31"),
    (lambda: moe.moe_glu_workspace_size(8, 8, 1 << 20), "status 2"),
    (lambda: moe.moe_linear_workspace_size(8, 8, 8, dtype="f32", grad_dtype="bf16"), "status 3"),
]


@pytest.mark.parametrize("i", range(len(NORM_BAD)))
def test_layernorm_refusals(i):
    call, match = NORM_BAD[i]
    with pytest.raises(moe.MoeError, match=match):
        call()


@pytest.mark.parametrize("i", range(len(LIN_BAD)))
def test_matrix_refusals(i):
    call, match = LIN_BAD[i]
    with pytest.raises(moe.MoeError, match=match):
        call()


# Status codes of the C calls: fake pointers are never read, since every check
# comes before the first launch.
NULL, SHAPE, DTYPE, WORKSPACE, MODE = 1, 2, 3, 4, 5
PTR = 0x10000


def _desc(**kw):
    v = dict(rows=100, d_in=64, d_out=96, dtype=1, grad_dtype=0, z_dtype=0, act=0, ldx=64, ldw=96, ldy=96, ldz=96, ldr=0,
             debug_shuffle_seed=0)
    v.update(kw)
    return moe._CDense(*v.values())


DESC_BAD = [(dict(dtype=2), DTYPE), (dict(grad_dtype=2), DTYPE), (dict(dtype=0, grad_dtype=1), DTYPE), (dict(z_dtype=3), DTYPE),
            (dict(act=5), MODE), (dict(act=-1), MODE), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE),
            (dict(d_in=0), SHAPE), (dict(d_out=-3), SHAPE), (dict(ldx=63), SHAPE), (dict(ldw=95), SHAPE),
            (dict(ldy=95), SHAPE), (dict(ldz=0), SHAPE), (dict(ldr=-1), SHAPE), (dict(ldx=1 << 20), SHAPE),
            (dict(d_in=1 << 19, ldx=1 << 19, ldw=1 << 19), SHAPE)]


@pytest.mark.parametrize("bad,status", DESC_BAD)
def test_description_status(bad, status):
    lib = moe.load_library()
    c = _desc(**bad)
    n = ctypes.c_size_t()
    for name in ("moe_linear_workspace_size", "moe_glu_workspace_size"):
        assert getattr(lib, name)(c, ctypes.byref(n), None) == status
    p = PTR
    assert lib.moe_linear_fwd(c, p, p, p, p, p, p, p, 1 << 40, None) == status
    assert lib.moe_linear_bwd(c, p, p, p, p, p, p, p, p, p, 1 << 40, None) == status
    assert lib.moe_glu_fwd(c, p, p, p, p, p, p, p, 1 << 40, None) == status
    assert lib.moe_glu_bwd(c, p, p, p, p, p, p, p, p, p, p, p, 1 << 40, None) == status


# more tiles, or more of x to copy, than one launch covers
@pytest.mark.parametrize("big", [dict(dtype=0, rows=(1 << 31) - 1, d_in=1, d_out=1), dict(rows=(1 << 31) - 1, d_in=4096, d_out=4096),
                                 dict(rows=1 << 22, d_in=8199, d_out=8)])
def test_rows_past_one_launch(big):
    lib, p = moe.load_library(), PTR
    v = dict(rows=100, d_in=64, d_out=96)
    v.update(big)
    v.update(ldx=v["d_in"], ldw=v["d_out"], ldy=v["d_out"], ldz=v["d_out"])
    c = _desc(**v)
    assert lib.moe_linear_fwd(c, p, p, p, None, p, p, p, 1 << 62, None) == SHAPE
    assert lib.moe_linear_bwd(c, p, p, p, p, None, p, p, p, p, 1 << 62, None) == SHAPE
    assert lib.moe_glu_fwd(c, p, p, p, p, p, p, p, 1 << 62, None) == SHAPE
    assert lib.moe_glu_bwd(c, p, p, p, p, p, p, None, p, p, p, p, 1 << 62, None) == SHAPE


def test_pointer_and_workspace_status():
    lib, p = moe.load_library(), PTR
    big = 1 << 40
    c = _desc(act=4)
    assert lib.moe_linear_fwd(None, p, p, p, p, p, p, p, big, None) == NULL
    assert lib.moe_linear_workspace_size(None, None, None) == NULL
    for i in (0, 1, 4):   # x, w, y
        a = [p] * 6
        a[3] = None       # no residual (its ld is 0)
        a[i] = None
        assert lib.moe_linear_fwd(c, *a, p, big, None) == NULL, i
        a[i] = p + 8      # 16-byte alignment
        assert lib.moe_linear_fwd(c, *a, p, big, None) == SHAPE, i
    assert lib.moe_linear_fwd(c, p, p, p, p, p, p, p, big, None) == SHAPE          # residual with ldr < d_out
    assert lib.moe_linear_fwd(c, p, p, p + 1, None, p, p, p, big, None) == SHAPE   # bias off its elements
    for i in (0, 1, 2, 3, 5, 6):   # dy, x, w, z, dx, dw
        a = [p, p, p, p, None, p, p, p]
        a[i] = None
        assert lib.moe_linear_bwd(c, *a, p, big, None) == NULL, i
        a[i] = p + 2
        assert lib.moe_linear_bwd(c, *a, p, big, None) == SHAPE, i
    assert lib.moe_linear_bwd(c, p, p, p, p, p, p, p, p, p, big, None) == SHAPE    # dx_add with ldr < d_in
    # workspaces: too small, missing, misaligned
    n = ctypes.c_size_t()
    assert lib.moe_linear_workspace_size(c, None, ctypes.byref(n)) == 0 and n.value > 0
    bwd = lambda ws, k: lib.moe_linear_bwd(c, p, p, p, p, None, p, p, p, ws, k, None)  # noqa: E731
    assert bwd(p, n.value - 1) == WORKSPACE and bwd(p + 16, n.value) == WORKSPACE and bwd(None, n.value) == NULL
    assert lib.moe_glu_fwd(c, p, p, p, p, p, None, p, big, None) == NULL           # g without u
    assert lib.moe_glu_bwd(c, p, p, p, p, p, None, None, p, p, p, p, big, None) == NULL
    # layer norm
    fwd = lambda *a: lib.moe_layernorm_fwd(*a, 0, None)  # noqa: E731
    assert fwd(p, p, p, 2, 4, 8, 8, 1e-5, p, p, p) == DTYPE
    assert fwd(p, p, p, 1, 4, 8, 7, 1e-5, p, p, p) == SHAPE
    assert fwd(p, p, p, 1, 4, 16385, 16385, 1e-5, p, p, p) == SHAPE
    assert fwd(p, p, p, 1, 1 << 30, 8, 1 << 11, 1e-5, p, p, p) == SHAPE
    assert fwd(p + 1, p, p, 1, 4, 8, 8, 1e-5, p, p, p) == SHAPE
    assert fwd(p, p, p, 1, 4, 8, 8, 1e-5, p, p, None) == NULL
    assert fwd(None, p, p, 1, 4, 8, 8, 1e-5, p, p, p) == NULL
    assert fwd(p, p, p, 1, 4, 8, 8, -1.0, p, p, p) == SHAPE
    b = lambda ws, k: lib.moe_layernorm_bwd(p, p, p, p, p, None, 1, 4, 8, 8, 8, 0, p, p, p, ws, k, 0, None)  # noqa: E731
    assert b(p, 1) == WORKSPACE and b(None, big) == NULL and b(p + 8, big) == WORKSPACE
    assert lib.moe_layernorm_workspace_size(4, 8, None) == NULL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [0, 1, 7, 64, 65, 1000, 1 << 20, (1 << 31) - 1])
def test_workspace_stays_bounded(dtype, rows):
    """Splits take at most 1 GiB of partials, and copies of aligned operands
    none."""
    for size in (moe.moe_linear_workspace_size, moe.moe_glu_workspace_size):
        fwd, bwd = size(rows, 512, 768, dtype)
        assert fwd <= 1 << 30
        nm = 2 if size is moe.moe_glu_workspace_size else 1
        es = 2 if dtype == "bf16" else 4
        # forced chunks of the weight gradient (32-bit offsets), the column
        # sums, and dz of the gated product
        forced = ((rows + 64) * 768 * 2 * 2 // (1 << 30) + 2) * 512 * 768 * 2 * 4
        assert bwd <= (1 << 30) + forced + 512 * 768 * 4 + (nm - 1) * rows * 2 * 768 * es + 4096


def test_workspace_of_unaligned_rows_holds_copies():
    fwd, _ = moe.moe_linear_workspace_size(1000, 513, 769)
    assert fwd >= 1000 * 520 * 2 + 513 * 776 * 2
    assert moe.moe_linear_workspace_size(40, 513, 769)[0] < 513 * 776 * 2   # few rows are read in place


def test_alignment_is_checked_by_argument():
    """A bias may start at any element, and lets no matrix that starts at the
    same address (a row of x, a column of w) past the matrices' own check."""
    lib, p, big = moe.load_library(), PTR, 1 << 40
    c = _desc(act=4, ldr=96)
    for odd in (p + 2, p + 8):
        for i in (0, 1, 3, 4, 5):   # x, w, residual, y, z
            a = [p, p, odd, p, p, p]
            a[i] = odd
            assert lib.moe_linear_fwd(c, *a, p, big, None) == SHAPE, (odd, i)


ANY_X, ANY_W, ANY_Y, ANY_REST = 0x100, 0x200, 0x400, 0x800


def test_addresses_that_a_description_allows():
    """moe_any: element addresses for the matrices named, 16 bytes for the others;
    the float32 matrices of a bf16 call keep to 4 bytes.  (A call that passes
    every check would be launched: here the missing workspace ends it.)"""
    lib, p = moe.load_library(), PTR
    need = lambda c, bwd: _sizes(lib, c)[bwd]  # noqa: E731
    c = _desc(act=4 | ANY_X | ANY_W)
    assert need(c, 0) > 0
    fwd = lambda c, *a: lib.moe_linear_fwd(c, *a, None, 0, None)  # noqa: E731
    assert fwd(c, p + 2, p + 6, p, None, p, p) == NULL
    assert fwd(c, p + 1, p, p, None, p, p) == SHAPE
    assert fwd(c, p + 2, p, p, None, p + 2, p) == SHAPE
    assert fwd(c, p + 2, p, p, None, p, p + 4) == SHAPE
    c = _desc(act=4 | ANY_X | ANY_Y | ANY_REST, ldr=96)
    assert fwd(c, p, p, p, p + 2, p + 2, p + 4) == NULL
    assert fwd(c, p, p, p, p + 2, p + 2, p + 2) == SHAPE      # z is float32
    assert fwd(c, p, p + 2, p, p + 2, p + 2, p + 4) == SHAPE
    bwd = lambda c, *a: lib.moe_linear_bwd(c, *a, None, 0, None)  # noqa: E731
    assert bwd(c, p + 2, p + 2, p, p + 4, None, p + 2, p + 4, p) == NULL
    assert bwd(c, p + 2, p + 2, p, p + 4, None, p + 2, p + 2, p) == SHAPE   # dw is float32
    c = _desc(act=0x1000)
    assert lib.moe_linear_workspace_size(c, None, None) == MODE


def _sizes(lib, c):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_linear_workspace_size(c, ctypes.byref(f), ctypes.byref(b)) == 0
    return f.value, b.value


def test_workspace_of_unaligned_bases_holds_copies():
    lib = moe.load_library()
    v = dict(rows=1000, d_in=512, d_out=768, ldx=512, ldw=768, ldy=768, ldz=768)
    none, allx = _sizes(lib, _desc(**v)), _sizes(lib, _desc(**v, act=ANY_X | ANY_W | ANY_Y))
    assert allx[0] >= none[0] + 1000 * 512 * 2 + 512 * 768 * 2
    assert allx[1] >= none[1] + 1000 * 512 * 2 + 512 * 768 * 2 + 1000 * 768 * 2   # and dy
    assert _sizes(lib, _desc(**v, act=ANY_REST)) == none
    f32 = dict(v, dtype=0)
    assert _sizes(lib, _desc(**f32)) == _sizes(lib, _desc(**f32, act=ANY_X | ANY_W | ANY_Y | ANY_REST))


@pytest.mark.parametrize("size", [moe.moe_linear_workspace_size, moe.moe_glu_workspace_size])
def test_workspace_size_of_strided_and_unaligned_tensors(size):
    """The sizes that the calls themselves ask for."""
    kind = "linear" if size is moe.moe_linear_workspace_size else "glu"
    plan = lambda a, *ld: moe._dense_plan(kind, 1000, 512, 768, 1, 0, 0, a, *ld, 768, 0, 0)[1:]  # noqa: E731
    kw = dict(act="gelu")
    base = size(1000, 512, 768, **kw)
    assert base == plan(4, 512, 768, 768) == size(1000, 512, 768, ldx=512, ldw=768, ldy=768, **kw)
    assert size(1000, 512, 768, ldx=515, **kw) == plan(4, 515, 768, 768) > base
    assert size(1000, 512, 768, ldw=769, **kw) == plan(4, 512, 769, 768) > base
    assert size(1000, 512, 768, ldx=520, ldw=776, **kw)[0] == base[0]
    assert size(1000, 512, 768, unaligned=("x", "w"), **kw) == plan(4 | ANY_X | ANY_W, 512, 768, 768) > base
    assert moe.moe_linear_workspace_size(1000, 512, 768, ldy=769)[1] > moe.moe_linear_workspace_size(1000, 512, 768)[1]
    for bad, match in ((dict(dtype="fp8"), "dtypes"), (dict(dtype=None, grad_dtype=None), "dtypes"), (dict(grad_dtype="i32"), "dtypes"), (dict(unaligned=("z",)), "unaligned"),
                       (dict(ldx=511), "status 2"), (dict(act="tanh"), "act")):
        with pytest.raises(moe.MoeError, match=match):
            size(1000, 512, 768, **bad)


# --------------------------------------------------------------------- kernels
def test_cases_reach_every_kernel():
    found = set().union(*[dense_cases.kernels(*c) for c in dense_cases.CASES])
    assert found == dense_cases.every_kernel()


def test_stage_names():
    names = moe.moe_linear_stage_names
    assert names(0, 64, 96, 0) == [] and names(0, 64, 96, 1) == ["zero", "zero"] and names(0, 64, 96, 2) == ["zero"]
    assert names(1, 64, 96, 0) == ["linear_few16"]
    assert names(1500, 1001, 517, 1, act="gelu")[0] == "dz_copy" and names(1500, 1001, 517, 0)[0] == "copy"
    assert names(1500, 1024, 512, 0, unaligned=("x",))[0] == "copy" and names(1500, 1024, 512, 0)[0].startswith("linear_")
    assert names(4096, 8192, 2048, 1)[0] == "sums" and names(4096, 8192, 2048, 2)[0].startswith("dx_")
    assert names(4096, 8192, 2048, 1)[-1] == "join"
    assert moe.moe_glu_stage_names(4096, 2048, 8192, 0) == ["glu_256x256"]
    lib, c = moe.load_library(), _desc()
    b = ctypes.create_string_buffer(64)
    assert lib.moe_linear_stage_names(c, 3, b, 64) == MODE and lib.moe_linear_stage_names(c, 0, None, 64) == NULL
    assert lib.moe_linear_stage_names(c, 0, b, 8) == WORKSPACE and lib.moe_linear_stage_names(None, 0, b, 64) == NULL
    assert lib.moe_glu_stage_names(_desc(act=9), 0, b, 64) == MODE
    with pytest.raises(moe.MoeError, match="status 5"):
        names(4, 8, 8, 3)


def test_few_rows_of_an_unaligned_input():
    """An x whose rows do not start on 16 bytes is copied, for the weight-streaming
    kernel as for the tiles, and does not keep more rows on that kernel."""
    names = moe.moe_linear_stage_names
    assert names(50, 512, 520, 0) == names(50, 512, 520, 0, ldx=513)[1:] and names(50, 512, 520, 0, ldx=513)[0] == "copy"
    for rows in (13, 32):
        assert names(rows, 512, 520, 0, ldx=513) == ["copy"] + names(rows, 512, 520, 0)
        assert names(rows, 512, 520, 0, unaligned=("x",)) == ["copy"] + names(rows, 512, 520, 0)
    assert names(12, 512, 520, 0, ldx=513) == ["linear_few16"]
    assert names(20, 513, 520, 0, ldx=520) == ["linear_few32"]      # rows of 16-byte starts, whatever their length
    assert names(64, 512, 521, 0) == ["linear_few64"] and names(64, 512, 521, 0, ldx=513) == ["copy", "linear_few64"]
    assert moe.moe_glu_stage_names(49, 512, 520, 0, ldx=513)[1].startswith("glu_64x64")
    assert names(20, 512, 520, 0, "f32", ldx=513) == ["linear_few32"]
