"""Calls of the dense operators that their documentation allows, beside the
ordinary ones: gradients and outputs in place, outputs left out, one tensor as
several arguments."""
import pytest
import torch

import bitwise_deterministic_moe_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(5, 7), (2100, 512), (700, 2050), (40, 4096), (33, 9000), (600, 16384)])
def test_layernorm_gradient_in_place(dtype, rows, cols):
    """dx may be dx_add: each element is read before it is written."""
    torch.manual_seed(cols)
    x, dy, add = (torch.randn(rows, cols, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn(cols, device=DEV).to(dtype)
    _, mean, rstd = moe.moe_layernorm_fwd(x, w)
    want = moe.moe_layernorm_bwd(dy, x, w, mean, rstd, dx_add=add)
    dx = add.clone()
    got = moe.moe_layernorm_bwd(dy, x, w, mean, rstd, dx_add=dx, dx=dx)
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, want))
    # one tensor as gradient, input and added gradient
    one = moe.moe_layernorm_bwd(x, x, w, mean, rstd, dx_add=x)
    two = moe.moe_layernorm_bwd(x.clone(), x, w, mean, rstd, dx_add=x.clone())
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,f", [(9, 264, 136), (50, 513, 40), (300, 264, 136), (70, 264, 4104), (1200, 1032, 264)])
def test_gated_gradient_and_strided_residual_in_place(dtype, rows, d, f):
    torch.manual_seed(rows)
    r = lambda *s: torch.randn(*s, device=DEV).to(dtype)  # noqa: E731
    x, w, w2, da, add = r(rows, d), r(d, f), r(d, f), r(rows, f), r(rows, d)
    _, g, u = moe.moe_glu_fwd(x, w, w2, save=True)
    want = moe.moe_glu_bwd(da, x, w, w2, g, u, dx_add=add)
    dx = add.clone()
    got = moe.moe_glu_bwd(da, x, w, w2, g, u, dx_add=dx, dx=dx)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # y is the residual, with rows further apart; what lies between them stays
    res = r(rows, f + 5)
    want = moe.moe_linear_fwd(x, w, residual=res[:, :f].contiguous(), act="gelu")[0]
    keep = res[:, f:].clone()
    moe.moe_linear_fwd(x, w, residual=res[:, :f], y=res[:, :f], act="gelu")
    assert torch.equal(res[:, :f], want) and torch.equal(res[:, f:], keep)


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 1), (torch.float32, 0)])
def test_outputs_left_out(dtype, code):
    """NULL statistics, weight gradient or bias gradient of the C calls."""
    lib = moe.load_library()
    rows, cols = 333, 264
    torch.manual_seed(1)
    x, dy = torch.randn(rows, cols, device=DEV).to(dtype), torch.randn(rows, cols, device=DEV).to(dtype)
    y, mean, rstd = moe.moe_layernorm_fwd(x)
    y2, dx2 = torch.empty_like(y), torch.empty_like(x)
    p, st = (lambda t: None if t is None else t.data_ptr()), torch.cuda.current_stream().cuda_stream
    assert lib.moe_layernorm_fwd(p(x), None, None, code, rows, cols, cols, 1e-5, p(y2), None, None, 0, st) == 0
    assert torch.equal(y2, y)
    dx, dw, db = moe.moe_layernorm_bwd(dy, x, None, mean, rstd)
    n = moe.moe_layernorm_workspace_size(rows, cols)
    for gw, gb in ((True, False), (False, True), (False, False)):
        a, b = (torch.full((cols,), 7.0, device=DEV) if g else None for g in (gw, gb))
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if gw or gb else None   # read for the sums alone
        assert lib.moe_layernorm_bwd(p(dy), p(x), None, p(mean), p(rstd), None, code, rows, cols, cols, cols, 0, p(dx2), p(a),
                                     p(b), p(ws), n if ws is not None else 0, 0, st) == 0
        assert torch.equal(dx2, dx) and (a is None or torch.equal(a, dw)) and (b is None or torch.equal(b, db))
