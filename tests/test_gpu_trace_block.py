"""The tracer's train step with the dense operators around the layer: runs
are bit-identical at every op, a resumed run equals the continuous one, a
planted change is placed at the operator it enters by, and one step's
gradients match the oracle's."""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import oracle
from bitwise_deterministic_moe_amd import trace
from dense_bounds import host
from synth import CONFIGS, make_batch, make_block_inputs
from test_gpu_parity import EDGE

pytestmark = pytest.mark.gpu
OPS = {"moe_layernorm_fwd", "moe_glu_fwd", "moe_linear_fwd", "moe_linear_bwd", "moe_glu_bwd", "moe_layernorm_bwd"}


@pytest.mark.parametrize("name", ["tiny_fp32", "ragged_bf16"])
def test_block_runs_are_bit_identical_and_resume(name, tmp_path):
    cfg = CONFIGS.get(name) or EDGE[name]
    st_a, a = trace.run(cfg, 3, "ops", block=True)
    _, b = trace.run(cfg, 3, "ops", block=True)
    assert trace.first_divergence(a.records, b.records) is None
    assert OPS <= {r.op for r in a.records}
    st, _ = trace.run(cfg, 1, "ops", block=True)
    st.save(str(tmp_path / "ck.npz"))
    st2 = trace.TrainState.load(str(tmp_path / "ck.npz"), moe.Problem.from_config(cfg))
    st2, tail = trace.run(cfg, 3, "ops", st=st2, block=True)
    assert trace.first_divergence([r for r in a.records if r.step >= 1], tail.records) is None
    for n in trace.BLOCK_WEIGHTS:
        assert torch.equal(st2.master[n], st_a.master[n])
        assert not torch.equal(st_a.master[n], trace.initial_state(cfg, block=True).master[n]), f"{n} never moved"


def test_planted_change_is_placed_at_its_operator():
    cfg = CONFIGS["tiny_fp32"]

    def hook(step, where, st):
        if step == 1:
            st.runtime["wu"].view(-1)[3] += 0.5

    _, a = trace.run(cfg, 2, "ops", block=True)
    _, b = trace.run(cfg, 2, "ops", block=True, hook=hook)
    _, ra, _ = trace.first_divergence([r for r in a.records if r.phase != "metrics"],
                                      [r for r in b.records if r.phase != "metrics"])
    assert (ra.step, ra.op, ra.name) == (1, "moe_glu_fwd", "u")


def test_block_refuses_what_it_cannot_run():
    cfg = CONFIGS["bf16_e8k2"].with_(tokens=256)
    with pytest.raises(moe.MoeError, match="MXFP8"):
        trace.run(cfg, 1, mx=True, block=True)
    with pytest.raises(moe.MoeError, match="no weights"):
        trace.run(cfg, 1, st=trace.initial_state(cfg), block=True)


def test_first_step_updates_match_the_oracle():
    """The shared expert's and the projection's updates of step 0 in float32:
    master - lr grad against the oracle's gradients."""
    cfg, lr = CONFIGS["tiny_fp32"], 0.05
    st, _ = trace.run(cfg, 1, "metrics", block=True, lr=lr)
    w = {n: np.asarray(v, np.float64) for n, v in make_block_inputs(cfg).items()}
    batch = make_batch(cfg, 0)
    x, dy = (np.asarray(batch[n], np.float64) for n in ("x", "dy"))
    xn = oracle.layernorm_forward(x, w["nw"], w["nb"], 1e-5)[0]
    a, g, u = oracle.glu_forward(xn, w["wg"], w["wu"], "silu")
    da, dwd, dbd = oracle.linear_backward(dy, a, w["wd"], None, "none")
    _, dwg, dwu = oracle.glu_backward(da, xn, w["wg"], w["wu"], g, u, "silu")
    for n, grad in (("wd", dwd), ("bd", dbd), ("wg", dwg), ("wu", dwu)):
        want = w[n] - lr * grad
        # sums of at most 128 float32 products through three products in a
        # row: fewer than 3 (2 * 128 + 10) roundings of 2^-24 of the terms,
        # which stay below 16 times the largest gradient
        tol = 3 * (2 * 128 + 10) * 2.0 ** -24 * 16 * lr * np.abs(grad).max() + 2.0 ** -23 * np.abs(want)
        assert (np.abs(host(st.master[n]) - want) <= tol).all(), n
