"""The oracle of the sort, the rows' copies and sums and dropout against
independent evaluations, and what their entry points refuse (before any GPU
call, so this runs without a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import oracle


# ---------------------------------------------------------------------- oracle
def test_sort_oracle_against_a_stable_sort():
    rng = np.random.default_rng(0)
    for t, k, e, begin, local in ((7, 3, 5, 0, 5), (40, 4, 9, 2, 3), (1, 1, 1, 0, 1), (6, 2, 4, 3, 1), (0, 2, 4, 0, 4)):
        idx = rng.integers(-1, e, (t, k))
        slot_row, offsets, row_src = oracle.sort_slots(idx, local, begin)
        flat = idx.reshape(-1)
        here = (flat >= begin) & (flat < begin + local)
        order = np.argsort(np.where(here, flat, 10 ** 6), kind="stable")[:here.sum()]
        assert np.array_equal(order, row_src) and offsets[-1] == here.sum()
        assert np.array_equal(slot_row.reshape(-1)[order], np.arange(order.size))
        assert (slot_row.reshape(-1)[~here] == -1).all()


def test_sum_oracle_gradients_against_differences():
    rng = np.random.default_rng(1)
    idx = rng.integers(-1, 4, (6, 3))
    slot_row, offsets, _ = oracle.sort_slots(idx, 4)
    rows, prob, dy = rng.standard_normal((20, 5)), rng.standard_normal((6, 3)), rng.standard_normal((6, 5))
    drows, dprob, _ = oracle.sum_rows_backward(dy, rows, slot_row, prob, np.zeros_like(rows))
    loss = lambda rows, prob: (oracle.sum_rows(rows, slot_row, prob)[0] * dy).sum()  # noqa: E731
    # linear in each argument: a central difference is exact but for rounding
    v, w = rng.standard_normal(rows.shape), rng.standard_normal(prob.shape)
    assert abs((loss(rows + v, prob) - loss(rows - v, prob)) / 2 - (drows * v).sum()) < 1e-12
    assert abs((loss(rows, prob + w) - loss(rows, prob - w)) / 2 - (dprob * w).sum()) < 1e-12
    # the copy's gradient is the sum without weights
    x = rng.standard_normal((6, 5))
    dr = rng.standard_normal(rows.shape)
    f = lambda x: (oracle.permute_rows(x, slot_row, np.zeros_like(rows)) * dr).sum()  # noqa: E731
    u = rng.standard_normal(x.shape)
    assert abs((f(x + u) - f(x - u)) / 2 - (oracle.sum_rows(dr, slot_row)[0] * u).sum()) < 1e-12


def test_philox_published_vectors():
    """The known answers published with the generator."""
    ff = 0xFFFFFFFF
    assert oracle.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert oracle.philox4x32((ff,) * 4, (ff,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert oracle.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_oracle_rate_and_position():
    n = 20000
    for p in (0.0, 0.1, 0.5, 1.0):
        kept = oracle.dropout_mask(n, p, 5, 9)
        # a binomial count: six standard deviations
        assert abs(kept.sum() - n * (1 - p)) <= 6 * np.sqrt(n * p * (1 - p))
    # a call that starts where another one ended continues it, also over the counter's wrap
    a = oracle.dropout_mask(40, 0.5, 5, 2 ** 64 - 4)
    assert np.array_equal(a[16:], oracle.dropout_mask(24, 0.5, 5, 0))


# ------------------------------------------------------------------- refusals
def _t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


I32, I64, F32 = torch.int32, torch.int64, torch.float32
BAD = [
    (lambda: moe.moe_sort(_t(4, 2, dtype=torch.int16), 4), "topk_idx"),
    (lambda: moe.moe_sort(_t(8, dtype=I32), 4), "topk_idx"),
    (lambda: moe.moe_sort(_t(2, 4, dtype=I32).t(), 4), "topk_idx"),
    (lambda: moe.moe_sort(_t(4, 0, dtype=I32), 4), "slots"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 0), "status 2"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 1025), "status 2"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 4, expert_begin=-1), "experts"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 4, slot_row=_t(4, 3, dtype=I32)), "slot_row"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 4, offsets=_t(4, dtype=I32)), "offsets"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 4, row_src=_t(7, dtype=I32)), "row_src"),
    (lambda: moe.moe_sort(_t(4, 2, dtype=I32), 4), "GPU"),
    (lambda: moe.moe_permute_fwd(_t(4, 8, dtype=torch.float16), _t(4, 2, dtype=I32)), "matrix"),
    (lambda: moe.moe_permute_fwd(_t(4, 2, 8), _t(4, 2, dtype=I32)), "matrix"),
    (lambda: moe.moe_permute_fwd(_t(4, 0), _t(4, 2, dtype=I32)), "matrix"),
    (lambda: moe.moe_permute_fwd(_t(8, 4).t(), _t(4, 2, dtype=I32)), "unit stride"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(4, 2, dtype=I64)), "slot_row"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(3, 2, dtype=I32)), "slot_row"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(7, dtype=I32)), "slot_row"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(0, dtype=I32)), "slot_row"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(4, 2, dtype=I32), rows=_t(8, 9)), "rows"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(4, 2, dtype=I32), rows=_t(8, 16)[:, :8]), "rows"),
    (lambda: moe.moe_permute_fwd(_t(4, 8), _t(4, 2, dtype=I32)), "GPU"),
    (lambda: moe.moe_permute_bwd(_t(8, 8, dtype=torch.int8), _t(4, 2, dtype=I32)), "float32 or bfloat16"),
    (lambda: moe.moe_permute_bwd(_t(8, 8), _t(8, dtype=I32)), "tokens"),
    (lambda: moe.moe_permute_bwd(_t(8, 8), _t(4, 2, dtype=I32), dx_add=_t(3, 8)), "residual"),
    (lambda: moe.moe_permute_bwd(_t(8, 8), _t(4, 2, dtype=I32), dx=_t(4, 9)), "output"),
    (lambda: moe.moe_unpermute_fwd(_t(8, 8), _t(4, 2, dtype=I32), _t(4, 2)), "prob"),
    (lambda: moe.moe_unpermute_fwd(_t(8, 8), _t(4, 2, dtype=I32), _t(4, 3, dtype=F32)), "prob"),
    (lambda: moe.moe_unpermute_fwd(_t(8, 8)[:, ::2], _t(4, 2, dtype=I32)), "rows"),
    (lambda: moe.moe_unpermute_fwd(_t(8, 8), _t(4, 2, dtype=I32), residual=_t(4, 8, dtype=F32)), "residual"),
    (lambda: moe.moe_unpermute_fwd(_t(8, 8), _t(4, 2, dtype=I32)), "GPU"),
    (lambda: moe.moe_unpermute_bwd(_t(4, 8), _t(8, 9), _t(4, 2, dtype=I32), _t(4, 2, dtype=F32)), "rows"),
    (lambda: moe.moe_unpermute_bwd(_t(4, 8), _t(8, 8, dtype=F32), _t(4, 2, dtype=I32), _t(4, 2, dtype=F32)), "rows"),
    (lambda: moe.moe_unpermute_bwd(_t(4, 8), _t(8, 8), _t(4, 2, dtype=I32), _t(4, 2, dtype=F32), drows=_t(7, 8)), "drows"),
    (lambda: moe.moe_unpermute_bwd(_t(4, 8), _t(8, 8), _t(4, 2, dtype=I32), _t(4, 2, dtype=F32), dprob=_t(4, 2)), "dprob"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8, dtype=torch.float16), 0.1, _t(2, dtype=I64)), "float32 or bfloat16"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), -0.1, _t(2, dtype=I64)), "p must"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), 1.1, _t(2, dtype=I64)), "p must"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), float("nan"), _t(2, dtype=I64)), "p must"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), 0.1, _t(2, dtype=I32)), "rng"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), 0.1, _t(3, dtype=I64)), "rng"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), 0.1, _t(4, dtype=I64)[::2]), "rng"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), 0.1, _t(2, dtype=I64), residual=_t(4, 7)), "residual"),
    (lambda: moe.moe_dropout_fwd(_t(4, 8), 0.1, _t(2, dtype=I64), y=_t(4, 16)[:, :8]), "output"),
    (lambda: moe.moe_dropout_fwd(torch.zeros(()), 0.1, _t(2, dtype=I64)), "columns"),
    (lambda: moe.moe_dropout_bwd(_t(4, 8), 0.1, _t(2, dtype=I64)), "GPU"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    call, says = BAD[i]
    with pytest.raises(moe.MoeError, match=says):
        call()


def test_numbers_per_slot_are_laid_out_by_token():
    """prob and dprob as [tokens, top_k], and one number of tokens from all that tell it."""
    flat, both = _t(8, dtype=I32), _t(4, 2, dtype=I32)
    p, turned = _t(4, 2, dtype=F32), _t(2, 4, dtype=F32)
    fwd, bwd = moe.moe_unpermute_fwd, moe.moe_unpermute_bwd
    for call, says in (
        (lambda: fwd(_t(8, 8), flat, p, residual=_t(2, 8)), "residual"),       # 4 tokens of 2 slots, and 2 of 4
        (lambda: fwd(_t(8, 8), flat, p, y=_t(2, 8)), "output"),
        (lambda: fwd(_t(8, 8), flat, turned, residual=_t(4, 8)), "residual"),
        (lambda: fwd(_t(8, 8), flat, _t(3, 2, dtype=F32)), "tokens"),
        (lambda: fwd(_t(8, 8), both, turned), "prob"),
        (lambda: bwd(_t(4, 8), _t(8, 8), both, turned), "prob"),
        (lambda: bwd(_t(4, 8), _t(8, 8), flat, turned), "prob"),
        (lambda: bwd(_t(4, 8), _t(8, 8), both, p, dprob=turned), "dprob"),
        # numbers that agree, in other shapes than a matrix too: refused only for want of a GPU
        (lambda: fwd(_t(8, 8), flat, p, residual=_t(4, 8), y=_t(4, 8)), "GPU"),
        (lambda: fwd(_t(8, 8), flat, _t(8, dtype=F32), residual=_t(2, 8)), "GPU"),
        (lambda: fwd(_t(8, 8), both, _t(8, dtype=F32)), "GPU"),
        (lambda: fwd(_t(8, 8), both, _t(8, 1, dtype=F32)), "GPU"),
        (lambda: fwd(_t(8, 8), flat, _t(1, 8, dtype=F32), residual=_t(2, 8)), "GPU"),
        (lambda: fwd(_t(8, 8), flat, _t(8, 1, dtype=F32)), "GPU"),
        (lambda: fwd(_t(8, 8), both, _t(2, 2, 2, dtype=F32)), "GPU"),
        (lambda: bwd(_t(4, 8), _t(8, 8), flat, p, dprob=p), "GPU"),
    ):
        with pytest.raises(moe.MoeError, match=says):
            call()


OK, NULL, SHAPE, DTYPE, WS = 0, 1, 2, 3, 4
A = 0x10000   # an address that is not followed: the calls return before any launch


def _sort(**o):
    a = dict(idx=A, dt=2, t=4, k=2, begin=0, local=4, slot=A, off=A, src=None, ws=None, nb=0)
    a.update(o)
    return moe.load_library().moe_sort(a["idx"], a["dt"], a["t"], a["k"], a["begin"], a["local"], a["slot"], a["off"], a["src"],
                                       a["ws"], a["nb"], 0, None)


@pytest.mark.parametrize("status,o", [
    (DTYPE, dict(dt=0)), (DTYPE, dict(dt=6)), (SHAPE, dict(t=-1)), (SHAPE, dict(k=0)), (SHAPE, dict(t=1 << 30, k=2)),
    (SHAPE, dict(local=0)), (SHAPE, dict(local=1025)), (SHAPE, dict(begin=-1)), (NULL, dict(idx=None)), (NULL, dict(slot=None)),
    (NULL, dict(off=None)), (SHAPE, dict(idx=A + 2)), (SHAPE, dict(dt=4, idx=A + 4)), (SHAPE, dict(slot=A + 1)),
    (SHAPE, dict(off=A + 2)), (SHAPE, dict(src=A + 2)), (NULL, dict(t=100000)), (WS, dict(t=100000, ws=A, nb=16)),
    (WS, dict(t=100000, ws=A + 4, nb=1 << 30)),
])
def test_sort_status(status, o):
    assert _sort(**o) == status


def test_sort_workspace():
    assert moe.moe_sort_workspace_size(1, 22, 512) == 0
    assert moe.moe_sort_workspace_size(4096, 22, 512) >= 512 * 4
    n = ctypes.c_size_t()
    lib = moe.load_library()
    assert lib.moe_sort_workspace_size(4, 2, 4, None) == NULL
    assert lib.moe_sort_workspace_size(4, 0, 4, ctypes.byref(n)) == SHAPE


def _permute(fwd=True, **o):
    a = dict(x=A, dt=1, t=4, k=2, cols=8, ld=8, slot=A, n=8, rows=A, add=None, ldadd=8)
    a.update(o)
    lib = moe.load_library()
    if fwd:
        return lib.moe_permute_fwd(a["x"], a["dt"], a["t"], a["k"], a["cols"], a["ld"], a["slot"], a["n"], a["rows"], 0, None)
    return lib.moe_permute_bwd(a["rows"], a["dt"], a["t"], a["k"], a["cols"], a["slot"], a["n"], a["add"], a["ldadd"], a["x"], 0,
                               None)


COMMON = [(DTYPE, dict(dt=2)), (DTYPE, dict(dt=5)), (SHAPE, dict(t=-1)), (SHAPE, dict(k=0)), (SHAPE, dict(cols=0)),
          (SHAPE, dict(cols=(1 << 24) + 1, ld=1 << 25)), (SHAPE, dict(n=-1)), (SHAPE, dict(n=1 << 31)), (NULL, dict(x=None)),
          (NULL, dict(slot=None)), (NULL, dict(rows=None)), (SHAPE, dict(x=A + 1)), (SHAPE, dict(rows=A + 1)),
          (SHAPE, dict(slot=A + 2)), (SHAPE, dict(n=1 << 30, cols=1 << 20, ld=1 << 20)), (SHAPE, dict(t=1 << 30, k=2))]


@pytest.mark.parametrize("status,o", COMMON + [(SHAPE, dict(ld=7)), (SHAPE, dict(ld=1 << 41)), (SHAPE, dict(dt=0, x=A + 2)),
                                               (OK, dict(t=0, x=None, slot=None, rows=None)), (OK, dict(n=0, rows=None))])
def test_permute_fwd_status(status, o):
    assert _permute(**o) == status


@pytest.mark.parametrize("status,o", COMMON + [(DTYPE, dict(dt=6)), (DTYPE, dict(dt=3)), (SHAPE, dict(add=A, ldadd=7)),
                                               (SHAPE, dict(add=A + 1)), (OK, dict(t=0, x=None, slot=None, rows=None))])
def test_permute_bwd_status(status, o):
    assert _permute(False, **o) == status


def _unpermute_bwd(**o):
    a = dict(dy=A, ld=8, rows=A, dt=1, t=4, k=2, cols=8, slot=A, n=8, prob=A, drows=A, dprob=A)
    a.update(o)
    return moe.load_library().moe_unpermute_bwd(a["dy"], a["ld"], a["rows"], a["dt"], a["t"], a["k"], a["cols"], a["slot"], a["n"],
                                                a["prob"], a["drows"], a["dprob"], 0, None)


@pytest.mark.parametrize("status,o", [(DTYPE, dict(dt=6)), (NULL, dict(prob=None)), (NULL, dict(drows=None)), (NULL, dict(rows=None)),
                                      (NULL, dict(dy=None)), (SHAPE, dict(prob=A + 2)), (SHAPE, dict(dprob=A + 2)),
                                      (SHAPE, dict(drows=A + 1)), (SHAPE, dict(ld=7)), (SHAPE, dict(dy=A + 1)), (OK, dict(t=0))])
def test_unpermute_bwd_status(status, o):
    assert _unpermute_bwd(**o) == status


def test_launches_beyond_the_grid():
    # far more than 2^24 workgroups, whichever kernel takes them
    t = (1 << 31) - 1
    assert _permute(t=t, k=1) == SHAPE
    assert _permute(False, t=t, k=1) == SHAPE
    assert _permute(False, t=t, k=1, cols=500) == SHAPE
    assert _unpermute_bwd(t=t, k=1) == SHAPE
    assert _unpermute_bwd(t=t, k=1, n=t, cols=500, ld=500) == SHAPE
    assert _dropout(rows=1 << 36) == SHAPE


# The last size inside the grid's limit and the first one outside, with a pointer missing, so that neither is launched:
# tokens of 32, 4 and 1 a workgroup, slots of 16 and 4, elements of 2048 and 1024.
LIMIT = (1 << 24) - 8


@pytest.mark.parametrize("call,tokens,o", [
    (lambda **o: _permute(rows=None, **o), 32 * LIMIT, dict()), (lambda **o: _permute(rows=None, **o), 4 * LIMIT, dict(cols=2048, ld=2048)),
    (lambda **o: _permute(False, rows=None, **o), 32 * LIMIT, dict()),
    (lambda **o: _permute(False, rows=None, **o), 4 * LIMIT, dict(cols=2048, ld=2048)),
    (lambda **o: _permute(False, rows=None, **o), LIMIT, dict(cols=2048, ld=2048, n=LIMIT)),
    (lambda **o: _permute(False, rows=None, **o), LIMIT, dict(dt=0, cols=1000, n=LIMIT)),
    (lambda **o: _unpermute_bwd(prob=None, **o), 16 * LIMIT, dict()),
    (lambda **o: _unpermute_bwd(prob=None, **o), 4 * LIMIT, dict(cols=1000, ld=1000, n=4 * LIMIT)),
])
def test_grid_limits_of_the_rows(call, tokens, o):
    assert call(k=1, t=tokens, **o) == NULL and call(k=1, t=tokens + 1, **o) == SHAPE


@pytest.mark.parametrize("per,o", [(2048, dict()), (2048, dict(ldx=9)), (1024, dict(cols=1, ldx=2, ldr=1)), (1024, dict(dt=0)),
                                   (1024, dict(dt=0, ldx=9))])
def test_grid_limits_of_dropout(per, o):
    cols = o.get("cols", 8)
    rows = per * LIMIT // cols
    assert _dropout(rows=rows, y=None, **o) == NULL and _dropout(rows=rows + 1, y=None, **o) == SHAPE


def _dropout(**o):
    a = dict(x=A, res=None, dt=1, rows=4, cols=8, ldx=8, ldr=8, p=0.1, rng=A, y=A)
    a.update(o)
    return moe.load_library().moe_dropout_fwd(a["x"], a["res"], a["dt"], a["rows"], a["cols"], a["ldx"], a["ldr"], a["p"], a["rng"],
                                              a["y"], 0, None)


@pytest.mark.parametrize("status,o", [
    (DTYPE, dict(dt=2)), (DTYPE, dict(dt=6)), (SHAPE, dict(p=-1e-9)), (SHAPE, dict(p=1.0000001)), (SHAPE, dict(p=float("nan"))),
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=0)), (SHAPE, dict(ldx=7)), (SHAPE, dict(res=A, ldr=7)), (NULL, dict(x=None)),
    (NULL, dict(y=None)), (NULL, dict(rng=None)), (SHAPE, dict(x=A + 1)), (SHAPE, dict(y=A + 1)), (SHAPE, dict(res=A + 1)),
    (SHAPE, dict(rng=A + 4)), (SHAPE, dict(cols=1 << 31, ldx=1 << 31)), (SHAPE, dict(rows=1 << 38)),
    (OK, dict(rows=0, x=None, y=None, rng=None)),
])
def test_dropout_status(status, o):
    assert _dropout(**o) == status
    if "res" not in o:
        a = dict(x=A, dt=1, rows=4, cols=8, ldx=8, p=0.1, rng=A, y=A)
        a.update(o)
        assert moe.load_library().moe_dropout_bwd(a["x"], a["dt"], a["rows"], a["cols"], a["ldx"], a["p"], a["rng"], a["y"], 0,
                                                  None) == status
