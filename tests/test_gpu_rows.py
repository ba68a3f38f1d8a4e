"""The sort, the rows' copies and sums and dropout on the GPU against their
definitions in float64.

Bounds, element by element: a rounding to a type is off by at most half a step
of the value (U); a float32 sum of n products in any order by at most
n 2^-24 of the products' magnitudes (n - 1 additions and n roundings of
products, or one each with fused products), here (n + 1) for the second order;
the sum with an addend counts one product more.
"""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load_library()


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, bound):
    got = _f64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.abs(got - want).max())


def _idx(t, k, experts, seed, dtype=torch.int32, low=0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.integers(low, experts, (t, k))).to(dtype).to(DEV)


# ------------------------------------------------------------------------ sort
SORTS = [  # tokens, k, expert numbers, begin, local
    (0, 2, 4, 0, 4), (1, 1, 1, 0, 1), (1, 22, 512, 0, 512), (5, 3, 7, 0, 7), (64, 1, 3, 1, 1), (333, 5, 1024, 0, 1024),
    (1000, 8, 64, 16, 8), (8192, 1, 64, 0, 64), (8193, 1, 64, 0, 64), (4096, 1, 64, 0, 64), (4097, 1, 1024, 0, 1024), (40000, 9, 1024, 0, 1024),
    (30000, 40, 7, 1, 5), (700, 22, 513, 5, 300), (4096, 22, 512, 0, 512),
    (16384, 22, 512, 100, 4), (50000, 7, 2, 0, 2), (3000, 64, 1000, 0, 1000),
]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("t,k,experts,begin,local", SORTS)
def test_sort(t, k, experts, begin, local, dtype):
    idx = _idx(t, k, experts, t + k, dtype, low=-1)
    slot_row = torch.full((t, k), 77, dtype=torch.int32, device=DEV)
    offsets = torch.full((local + 1,), 77, dtype=torch.int32, device=DEV)
    row_src = torch.full((t * k,), 77, dtype=torch.int32, device=DEV)
    moe.moe_sort(idx, local, begin, slot_row, offsets, row_src)
    want_row, want_off, want_src = oracle.sort_slots(idx.cpu().numpy(), local, begin)
    assert np.array_equal(offsets.cpu().numpy(), want_off)
    assert np.array_equal(slot_row.cpu().numpy(), want_row)
    r = want_off[-1]
    assert np.array_equal(row_src[:r].cpu().numpy(), want_src)
    assert (row_src[r:] == 77).all()           # behind the last row: as they were
    for seed in (3, 77):
        got = moe.moe_sort(idx, local, begin, need_row_src=True, shuffle_seed=seed)
        assert torch.equal(got[0], slot_row) and torch.equal(got[1], offsets) and torch.equal(got[2][:r], row_src[:r])
    assert moe.moe_sort(idx, local, begin)[2] is None


def test_sort_numbers_far_out():
    big = 1 << 40
    idx = torch.tensor([[2, -1, big + 2], [-big, 3, 2], [(1 << 32) + 2, 2 ** 63 - 1, -2 ** 63]], dtype=torch.int64, device=DEV)
    slot_row, offsets, row_src = moe.moe_sort(idx, 2, 2, need_row_src=True)
    assert slot_row.tolist() == [[0, -1, -1], [-1, 2, 1], [-1, -1, -1]]
    assert offsets.tolist() == [0, 2, 3] and row_src[:3].tolist() == [0, 5, 4]
    # nothing is local, and one expert for all
    assert moe.moe_sort(idx, 5, 100)[1].tolist() == [0] * 6
    same = torch.full((3000, 4), 6, dtype=torch.int32, device=DEV)
    slot_row, offsets, _ = moe.moe_sort(same, 8)
    assert torch.equal(slot_row.reshape(-1), torch.arange(12000, dtype=torch.int32, device=DEV))
    assert offsets.tolist() == [0] * 7 + [12000] * 2


# --------------------------------------------------------- rows there and back
ROWS = [  # tokens, k, experts, local, columns
    (1, 1, 1, 1, 1), (1, 22, 512, 512, 2048), (3, 4, 8, 8, 7), (17, 2, 5, 3, 64), (130, 9, 20, 20, 257), (64, 3, 4, 1, 1000),
    (40, 6, 16, 16, 4096), (33, 2, 3, 3, 5001), (9, 65, 70, 70, 24), (2, 3, 4, 0, 40),
    (3001, 22, 512, 30, 136), (9362, 7, 9, 9, 33),
]


def _case(t, k, experts, local, cols, dtype, seed=0, unaligned=False, strided=False):
    g = torch.Generator(device=DEV).manual_seed(seed + t)

    def mat(n, wide=0):
        a = torch.randn(n * (cols + wide) + 1, generator=g, device=DEV).to(dtype)
        a = a[1:] if unaligned else a[:-1]
        return a.reshape(n, cols + wide)[:, :cols]

    idx = _idx(t, k, experts, seed + t * k)
    if local:
        slot_row, offsets, _ = moe.moe_sort(idx, local)
    else:   # no slot has a row
        slot_row, offsets = torch.full((t, k), -1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    wide = 3 if strided else 0
    prob = torch.rand((t, k), generator=g, device=DEV)
    return dict(slot_row=slot_row, r=int(offsets[-1]), x=mat(t, wide), add=mat(t, wide), rows=mat(t * k), prob=prob, mat=mat)


@pytest.mark.parametrize("unaligned,strided", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,k,experts,local,cols", ROWS)
def test_rows_there_and_back(t, k, experts, local, cols, dtype, unaligned, strided):
    c = _case(t, k, experts, local, cols, dtype, 0, unaligned, strided)
    sr, slot = c["slot_row"].cpu().numpy(), c["slot_row"]
    u = U[dtype]
    # there: a copy, the rows behind the last one as they were
    rows = c["mat"](t * k)
    before = rows.clone()
    assert moe.moe_permute_fwd(c["x"], slot, rows=rows) is rows
    assert np.array_equal(_f64(rows), oracle.permute_rows(_f64(c["x"]), sr, _f64(before)))
    # its gradient
    for add in (None, c["add"]):
        want, size = oracle.sum_rows(_f64(c["rows"]), sr)
        if add is not None:
            want, size = want + _f64(add), size + np.abs(_f64(add))
        dx = moe.moe_permute_bwd(c["rows"], slot, dx_add=add)
        _close(dx, want, (k + 2) * E * size + u * (np.abs(want) + (k + 2) * E * size))
    # back, with weights
    for add in (None, c["add"]):
        want, size = oracle.sum_rows(_f64(c["rows"]), sr, _f64(c["prob"]))
        if add is not None:
            want, size = want + _f64(add), size + np.abs(_f64(add))
        y = moe.moe_unpermute_fwd(c["rows"], slot, c["prob"], residual=add)
        _close(y, want, (k + 2) * E * size + u * (np.abs(want) + (k + 2) * E * size))
    # gradients
    drows = c["mat"](t * k)
    before = drows.clone()
    got, dprob = moe.moe_unpermute_bwd(c["x"], c["rows"], slot, c["prob"], drows=drows)
    assert got is drows
    want, want_p, size = oracle.sum_rows_backward(_f64(c["x"]), _f64(c["rows"]), sr, _f64(c["prob"]), _f64(before))
    _close(drows, want, (u + 2 * E) * np.abs(want))
    named = np.zeros(t * k, bool)
    named[sr[sr >= 0]] = True
    assert np.array_equal(_f64(drows)[~named], _f64(before)[~named])
    _close(dprob, want_p, (cols + 1) * E * size)
    assert (dprob.cpu().numpy()[sr < 0] == 0).all()
    # launch order, in place, flat slots
    for seed in (5, 99):
        assert torch.equal(moe.moe_permute_fwd(c["x"], slot, rows=before.clone(), shuffle_seed=seed)[:c["r"]], rows[:c["r"]])
        assert torch.equal(moe.moe_unpermute_fwd(c["rows"], slot, c["prob"], residual=c["add"], shuffle_seed=seed), y)
        again = moe.moe_unpermute_bwd(c["x"], c["rows"], slot, c["prob"], shuffle_seed=seed)
        assert torch.equal(again[0][:c["r"]], drows[:c["r"]]) and torch.equal(again[1], dprob)
    own = c["rows"].clone()
    got = moe.moe_unpermute_bwd(c["x"], own, slot, c["prob"], drows=own)
    assert torch.equal(own[:c["r"]], drows[:c["r"]]) and torch.equal(got[1], dprob)
    assert torch.equal(own[c["r"]:], c["rows"][c["r"]:])
    res = c["add"].contiguous()
    assert torch.equal(moe.moe_unpermute_fwd(c["rows"], slot.reshape(-1), c["prob"], residual=res, y=res), y)
    assert torch.equal(moe.moe_permute_fwd(c["x"], slot.reshape(-1))[:c["r"]], rows[:c["r"]])


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8])
@pytest.mark.parametrize("t,k,cols", [(1, 22, 2048), (100, 3, 33), (7, 5, 16), (70, 2, 1)])
def test_permute_of_codes_and_their_scales(t, k, cols, dtype):
    codes = torch.randint(0, 127, (t, cols + 1), device=DEV).to(dtype)[:, 1:]
    scales = torch.rand((t, 1), device=DEV)
    slot_row, offsets, row_src = moe.moe_sort(_idx(t, k, 9, 4, low=-1), 9, need_row_src=True)
    r = int(offsets[-1])
    tok = row_src[:r].long() // k
    assert torch.equal(moe.moe_permute_fwd(codes, slot_row)[:r], codes[tok])
    assert torch.equal(moe.moe_permute_fwd(scales, slot_row)[:r], scales[tok])


@pytest.mark.parametrize("dtype", [torch.uint8, BF16, F32])
@pytest.mark.parametrize("t,k", [(3, 70), (700, 64), (70, 130)])
def test_permute_of_ragged_rows_and_many_slots(t, k, dtype):
    """Rows whose last pieces leave most lanes without a vector, for slots of every lane (a wave a token)."""
    size = torch.empty(0, dtype=dtype).element_size()
    for length in (516, 1008, 1028, 2100, 4112, 4600, 8204, 9000):      # bytes: 33 vectors up, past 4 KB and past 8
        cols = length // size
        x = torch.randint(0, 100, (t, cols), device=DEV).to(dtype)
        slot_row, offsets, row_src = moe.moe_sort(_idx(t, k, 5, length, low=-1), 5, need_row_src=True)
        r = int(offsets[-1])
        rows = torch.full((r + 3, cols), 7, dtype=dtype, device=DEV)
        moe.moe_permute_fwd(x, slot_row, rows=rows)
        assert torch.equal(rows[:r], x[row_src[:r].long() // k]) and (rows[r:] == 7).all(), length


def test_slots_past_the_rows_have_none():
    """A slot that names a row past the matrix: nothing is read or written for it."""
    slot_row = torch.tensor([[0, 5], [1, 2 ** 31 - 1], [-7, 2]], dtype=torch.int32, device=DEV)
    x = torch.randn(3, 40, device=DEV)
    rows = torch.full((3, 40), 7.0, device=DEV)
    moe.moe_permute_fwd(x, slot_row, rows=rows)
    assert torch.equal(rows, x)
    prob = torch.rand(3, 2, device=DEV)
    y = moe.moe_unpermute_fwd(rows, slot_row, prob)
    assert torch.equal(y, torch.stack((x[0] * prob[0, 0], x[1] * prob[1, 0], x[2] * prob[2, 1])))
    drows, dprob = moe.moe_unpermute_bwd(x, rows, slot_row, prob)
    assert torch.equal(drows, y) and dprob[0, 1] == dprob[1, 1] == dprob[2, 0] == 0
    empty = torch.empty((0, 40), device=DEV)
    assert (moe.moe_unpermute_fwd(empty, slot_row, prob) == 0).all()
    assert torch.equal(moe.moe_unpermute_fwd(empty, slot_row, prob, residual=x), x)
    assert moe.moe_permute_fwd(x, slot_row, rows=empty) is empty
    assert (moe.moe_unpermute_bwd(x, empty, slot_row, prob)[1] == 0).all()
    none = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert moe.moe_permute_fwd(x[:0], none).shape == (0, 40)
    assert moe.moe_unpermute_fwd(rows, none).shape == (0, 40)


def test_numbers_that_are_not_finite_stay_in_their_tokens():
    c = _case(40, 3, 8, 5, 100, F32)
    sr = c["slot_row"].cpu().numpy()
    bad = int(sr[sr >= 0][0])
    c["rows"][bad, 3] = float("nan")
    c["rows"][c["r"]:] = float("nan")            # behind the last row: not read
    y = _f64(moe.moe_unpermute_fwd(c["rows"], c["slot_row"], c["prob"]))
    hit = (sr == bad).any(1)
    assert np.isnan(y[hit, 3]).all() and np.isfinite(y[~hit]).all() and np.isfinite(np.delete(y, 3, 1)).all()
    _, dprob = moe.moe_unpermute_bwd(c["x"], c["rows"], c["slot_row"], c["prob"])
    assert np.array_equal(np.isnan(dprob.cpu().numpy()), sr == bad)


def test_gradients_against_differences():
    """The calls' own gradients against differences of their own values (they are
    linear in each argument, so a step of 1 has no truncation)."""
    c = _case(60, 4, 7, 7, 96, F32)
    slot, prob, rows, dy = c["slot_row"], c["prob"], c["rows"], c["x"]
    drows, dprob = moe.moe_unpermute_bwd(dy, rows, slot, prob)
    v, w = torch.randn_like(rows), torch.randn_like(prob)
    value = lambda r, p: (moe.moe_unpermute_fwd(r, slot, p).double() * dy.double()).sum().item()  # noqa: E731
    # y is off by (k + 2) 2^-24 of its terms, here below 4 standard deviations of 60 * 96 sums of 4 terms
    off = 6 * E * 60 * 96 * 4 * 16
    assert abs((value(rows + v, prob) - value(rows - v, prob)) / 2 - (drows.double() * v).sum().item()) < off
    assert abs((value(rows, prob + w) - value(rows, prob - w)) / 2 - (dprob.double() * w).sum().item()) < off


# --------------------------------------------------------------------- dropout
DROPS = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 257), (9, 1000), (2, 4096)]


def _rng(key, first):
    return torch.from_numpy(np.array([key, first], dtype=np.uint64).view(np.int64)).to(DEV)


@pytest.mark.parametrize("how", ["flat", "unaligned", "strided"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("rows,cols", DROPS)
def test_dropout(rows, cols, p, dtype, how):
    g = torch.Generator(device=DEV).manual_seed(rows * cols)

    def mat():
        a = torch.randn((rows, cols + (5 if how == "strided" else 0)), generator=g, device=DEV).to(dtype)
        if how == "unaligned":
            b = torch.empty(rows * cols + 1, dtype=dtype, device=DEV)[1:].reshape(rows, cols)
            return b.copy_(a)
        return a[:, :cols]

    x, res, dy = mat(), mat(), mat()
    key, first = 0x9ABCDEF012345678, 2 ** 64 - 3       # the counter wraps inside
    rng = _rng(key, first)
    kept = oracle.dropout_mask(rows * cols, p, key, first).reshape(rows, cols)
    s = 1 / (1 - p) if p < 1 else 0.0
    u = U[dtype]
    y = moe.moe_dropout_fwd(x, p, rng)
    assert np.array_equal(_f64(y) != 0, kept & (_f64(x) != 0))
    want = np.where(kept, _f64(x) * s, 0)
    # the scale's rounding, then the product's, then the type's
    _close(y, want, (u + 3 * E) * np.abs(want))
    y2 = moe.moe_dropout_fwd(x, p, rng, residual=res)
    want = np.where(kept, _f64(x) * s, 0) + _f64(res)
    size = np.where(kept, np.abs(_f64(x)) * s, 0) + np.abs(_f64(res))
    _close(y2, want, u * np.abs(want) + 4 * E * size)
    assert np.array_equal(_f64(y2)[~kept], _f64(res)[~kept])
    dx = moe.moe_dropout_bwd(dy, p, rng)
    assert torch.equal(dx, moe.moe_dropout_fwd(dy, p, rng))
    for seed in (7, 1234):
        assert torch.equal(moe.moe_dropout_fwd(x, p, rng, residual=res, shuffle_seed=seed), y2)
    a, b = x.contiguous().clone(), res.contiguous().clone()
    assert torch.equal(moe.moe_dropout_fwd(x.contiguous(), p, rng, residual=b, y=b), y2)
    assert torch.equal(moe.moe_dropout_fwd(a, p, rng, residual=res.contiguous(), y=a), y2)


def test_dropout_mask_does_not_depend_on_type_shape_or_layout():
    rng = _rng(11, 5)
    ones = torch.ones(3 * 4 * 50, device=DEV)
    y = moe.moe_dropout_fwd(ones, 0.3, rng) != 0
    for t in (ones.to(BF16), ones.reshape(12, 50), ones.reshape(3, 4, 50), ones.reshape(4, 150).to(BF16),
              torch.ones(12, 64, device=DEV)[:, :50], torch.ones(6, 104, device=DEV, dtype=BF16)[:, :100],
              torch.ones(75, 20, device=DEV, dtype=BF16)[:, :8]):
        assert torch.equal((moe.moe_dropout_fwd(t, 0.3, rng) != 0).reshape(-1), y)
    # a second call from where the first one ended continues its numbers
    both = moe.moe_dropout_fwd(torch.ones(1200, device=DEV), 0.3, rng) != 0
    rng[1] += 600 // 4
    assert torch.equal(moe.moe_dropout_fwd(ones, 0.3, rng) != 0, both[600:])
    assert torch.equal(y, both[:600])
    assert moe.moe_dropout_fwd(ones[:0].reshape(0, 5), 0.3, rng).shape == (0, 5)


def test_dropout_rate_and_values_that_are_not_finite():
    n = 1 << 24
    x = torch.full((n,), float("inf"), device=DEV)
    for p in (0.001, 0.25):
        y = moe.moe_dropout_fwd(x, p, _rng(3, 1))
        kept = int((y == float("inf")).sum())
        assert int((y == 0).sum()) == n - kept      # a dropped infinity is 0, not NaN
        # six standard deviations of a binomial count
        assert abs(kept - n * (1 - p)) < 6 * (n * p * (1 - p)) ** 0.5
    assert (moe.moe_dropout_fwd(x, 1.0, _rng(3, 1), residual=x) == x).all()


# ---------------------------------------------------- streams, graphs, overlap
def _step(c, rng, out):
    """The calls as a train step makes them."""
    slot_row, offsets, _ = moe.moe_sort(c["idx"], 7, slot_row=out["slot"], offsets=out["off"], ws=out["ws"])
    rows = moe.moe_permute_fwd(c["x"], slot_row, rows=out["rows"])
    y = moe.moe_unpermute_fwd(rows, slot_row, c["prob"], y=out["y"])
    moe.moe_dropout_fwd(y, 0.2, rng, residual=c["x"], y=out["z"])
    moe.moe_dropout_bwd(c["dy"], 0.2, rng, dx=out["dy"])
    moe.moe_unpermute_bwd(out["dy"], rows, slot_row, c["prob"], drows=out["drows"], dprob=out["dprob"])
    moe.moe_permute_bwd(out["drows"], slot_row, dx_add=c["dy"], dx=out["dx"])


def _buffers(t, k, cols):
    new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    i32 = torch.int32
    n = moe.moe_sort_workspace_size(t, k, 7)
    return dict(slot=new(t, k, dtype=i32), off=new(8, dtype=i32), ws=new(max(n, 1), dtype=torch.uint8), rows=new(t * k, cols),
                y=new(t, cols), z=new(t, cols), dy=new(t, cols), drows=new(t * k, cols), dprob=new(t, k, dtype=F32),
                dx=new(t, cols))


def _inputs(t, k, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    m = lambda: torch.randn((t, cols), generator=g, device=DEV).to(BF16)  # noqa: E731
    return dict(idx=_idx(t, k, 7, seed), x=m(), dy=m(), prob=torch.rand((t, k), generator=g, device=DEV))


@pytest.mark.parametrize("t,k,cols", [(5, 2, 72), (6000, 3, 264)])
def test_streams_and_graphs(t, k, cols):
    torch.manual_seed(0)
    a, b = _inputs(t, k, cols, 1), _inputs(t, k, cols, 2)
    rng = _rng(8, 0)
    want = []
    for c, first in ((a, 0), (b, 0), (a, 1000)):
        rng[1] = first
        o = _buffers(t, k, cols)
        _step(c, rng, o)
        want.append(o)
    names = ("slot", "off", "rows", "y", "z", "dy", "drows", "dprob", "dx")
    torch.cuda.synchronize()
    # two calls at once, each on a stream of its own
    rng[1] = 0
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = _buffers(t, k, cols), _buffers(t, k, cols)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            _step(a, rng, o1)
        with torch.cuda.stream(s2):
            _step(b, rng, o2)
    torch.cuda.synchronize()
    assert all(torch.equal(o1[n], want[0][n]) and torch.equal(o2[n], want[1][n]) for n in names)
    # captured: new inputs and a new counter at each replay
    c = {n: v.clone() for n, v in a.items()}
    o = _buffers(t, k, cols)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(c, rng, o)
    for inputs, first, w in ((a, 0, want[0]), (b, 0, want[1]), (a, 1000, want[2]), (a, 0, want[0])):
        for n in c:
            c[n].copy_(inputs[n])
        rng[1] = first
        for n in names:
            o[n].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(o[n], w[n]), n
        moe.moe_sort(inputs["idx"], 7)      # eager work between the replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,k,experts,local,cols,big", [(20011, 7, 64, 64, 1032, True), (40003, 8, 64, 64, 505, True),
                                                        (60000, 22, 512, 150, 700, True), (5003, 22, 512, 20, 1033, False)])
def test_many_rows(t, k, experts, local, cols, big, dtype):
    """More than 256 MB of rows (big), or few rows of many slots: every element against float64 arithmetic on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(t)
    mat = lambda n: torch.randn((n, cols), generator=g, device=DEV).to(dtype)  # noqa: E731
    sr, off, _ = moe.moe_sort(torch.randint(0, experts, (t, k), generator=g, device=DEV, dtype=torch.int32), local)
    n = int(off[-1])
    assert big == (n * cols * dtype.itemsize > 256 << 20)
    x, add, rows = mat(t), mat(t), mat(n + 3)
    p = torch.rand((t, k), generator=g, device=DEV)
    u = U[dtype]

    def near(got, want, bound):
        assert bool(((got.double() - want).abs() <= bound).all())

    there = rows.clone()
    moe.moe_permute_fwd(x, sr, rows=there)
    assert torch.equal(there[n:], rows[n:])
    y = moe.moe_unpermute_fwd(rows, sr, p, residual=add)
    dx = moe.moe_permute_bwd(rows, sr)
    drows = rows.clone()
    _, dprob = moe.moe_unpermute_bwd(x, rows, sr, p, drows=drows)
    assert torch.equal(drows[n:], rows[n:])
    xd = x.double()
    want, size, plain, whole = add.double(), add.double().abs(), torch.zeros_like(xd), torch.zeros_like(xd)
    for j in range(k):
        has = sr[:, j] >= 0
        r = sr[:, j].long()[has]
        assert torch.equal(there[r], x[has])
        v, w = rows[r].double(), p[has, j:j + 1].double()
        want[has] += v * w
        size[has] += (v * w).abs()
        plain[has] += v
        whole[has] += v.abs()
        near(drows[r], xd[has] * w, (u + 2 * E) * (xd[has] * w).abs())
        dots = xd[has] * v
        near(dprob[has, j], dots.sum(1), (cols + 1) * E * dots.abs().sum(1))
        assert bool((dprob[~has, j] == 0).all())
    near(y, want, (k + 2) * E * size + u * (want.abs() + (k + 2) * E * size))
    near(dx, plain, (k + 2) * E * whole + u * (plain.abs() + (k + 2) * E * whole))


def test_more_than_2_31_bytes_and_elements():
    """Rows past 2^31 elements: the slots' rows are the last ones of a 5 GB matrix."""
    cols, n = 1 << 16, 40000
    rows = torch.zeros((n, cols), dtype=BF16, device=DEV)
    slot_row = torch.tensor([[n - 1, 5], [n - 2, 33000]], dtype=torch.int32, device=DEV)
    x = torch.randn(2, cols, device=DEV).to(BF16)
    moe.moe_permute_fwd(x, slot_row, rows=rows)
    assert torch.equal(rows[n - 1], x[0]) and torch.equal(rows[5], x[0]) and torch.equal(rows[33000], x[1])
    prob = torch.tensor([[0.5, 0.25], [1.0, 2.0]], device=DEV)
    assert torch.equal(moe.moe_unpermute_fwd(rows, slot_row, prob), (x.float() * prob.sum(1, keepdim=True)).to(BF16))
    moe.moe_unpermute_bwd(x, rows, slot_row, prob, drows=rows)
    assert torch.equal(rows[n - 2], x[1]) and torch.equal(rows[n - 1], (x[0].float() * 0.5).to(BF16))
    assert float(rows[6:32999].abs().max()) == 0
    del rows
    # dropout counts its elements in 64 bits
    y = moe.moe_dropout_fwd(torch.ones((n, cols), dtype=BF16, device=DEV), 0.5, _rng(2, 7))
    at = n * cols - 4096
    assert np.array_equal(_f64(y.reshape(-1)[at:]) != 0, oracle.dropout_mask(4096, 0.5, 2, 7 + at // 4))


def test_the_largest_grids():
    """The most tokens of one column that the calls take: 2^24 - 8 workgroups, the numbers of the last ones looked at."""
    t = 32 * ((1 << 24) - 8)
    slot_row = torch.full((t, 1), -1, dtype=torch.int32, device=DEV)
    at = torch.tensor([0, 31, 32, t // 2, t - 33, t - 32, t - 1], device=DEV)
    slot_row[at, 0] = torch.arange(7, dtype=torch.int32, device=DEV)
    x = torch.zeros((t, 1), dtype=torch.uint8, device=DEV)
    x[at, 0] = torch.arange(1, 8, dtype=torch.uint8, device=DEV)
    assert moe.moe_permute_fwd(x, slot_row, rows=torch.zeros((7, 1), dtype=torch.uint8, device=DEV))[:, 0].tolist() == list(range(1, 8))
    del x
    rows = torch.arange(1, 8, device=DEV).to(BF16)[:, None].contiguous()
    y = moe.moe_unpermute_fwd(rows, slot_row)
    assert y[at, 0].tolist() == list(range(1, 8)) and int((y != 0).sum()) == 7
    del y
    n = t // 2                                    # 16 slots a workgroup
    slot_row = slot_row[n:]
    prob = torch.full((n, 1), 3.0, device=DEV)
    drows, dprob = moe.moe_unpermute_bwd(torch.full((n, 1), 2.0, dtype=BF16, device=DEV), rows, slot_row, prob)
    assert drows[3:, 0].tolist() == [6.0] * 4     # the named rows of this half
    assert dprob[at[3:] - n, 0].tolist() == [8.0, 10.0, 12.0, 14.0] and int((dprob != 0).sum()) == 4
    for tokens, call in ((t + 1, lambda s: moe.moe_unpermute_fwd(rows, s)),
                         (n + 1, lambda s: moe.moe_unpermute_bwd(torch.empty((n + 1, 1), dtype=BF16, device=DEV), rows, s,
                                                                 torch.empty((n + 1, 1), device=DEV)))):
        with pytest.raises(moe.MoeError, match="status 2"):
            call(torch.full((tokens, 1), -1, dtype=torch.int32, device=DEV))
