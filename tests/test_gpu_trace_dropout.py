"""The tracer's train step with dropout: runs are bit-identical at every op, a
resumed run finds the continuous run's masks, the mask and the gradients are the
definition's, and without dropout a trace is what it was."""
import numpy as np
import pytest
import torch

import bitwise_deterministic_moe_amd as moe
import oracle
from bitwise_deterministic_moe_amd import trace
from synth import CONFIGS, make_batch
from test_gpu_parity import EDGE

pytestmark = pytest.mark.gpu
KINDS = [("tiny_fp32", {}), ("tiny_fp32", dict(block=True)), ("ragged_bf16", dict(block=True)), ("ragged_bf16", dict(mx=True))]


def _cfg(name):
    return CONFIGS.get(name) or EDGE[name]


@pytest.mark.parametrize("name,kind", KINDS)
def test_runs_are_bit_identical_and_resume(name, kind, tmp_path):
    cfg = _cfg(name)
    st_a, a = trace.run(cfg, 3, "ops", dropout=0.25, dropout_seed=77, **kind)
    _, b = trace.run(cfg, 3, "ops", dropout=0.25, dropout_seed=77, **kind)
    assert trace.first_divergence(a.records, b.records) is None
    assert {"moe_dropout_fwd", "moe_dropout_bwd"} <= {r.op for r in a.records}
    st, _ = trace.run(cfg, 1, "ops", dropout=0.25, dropout_seed=77, **kind)
    st.save(str(tmp_path / "ck.npz"))
    st2 = trace.TrainState.load(str(tmp_path / "ck.npz"), moe.Problem.from_config(cfg))
    st2, tail = trace.run(cfg, 3, "ops", st=st2, dropout=0.25, dropout_seed=77, **kind)
    assert trace.first_divergence([r for r in a.records if r.step >= 1], tail.records) is None
    assert all(torch.equal(st2.master[n], st_a.master[n]) for n in st_a.master)
    # another seed: the same layer, and another mask from its first use on
    _, c = trace.run(cfg, 1, "ops", dropout=0.25, dropout_seed=78, **kind)
    _, ra, _ = trace.first_divergence(a.records, c.records)
    assert (ra.step, ra.op) == (0, "moe_dropout_fwd")


@pytest.mark.parametrize("kind", [{}, dict(block=True)])
def test_without_dropout_nothing_changes(kind):
    cfg = CONFIGS["tiny_fp32"]
    _, a = trace.run(cfg, 2, "ops", **kind)
    _, b = trace.run(cfg, 2, "ops", dropout=0.0, dropout_seed=5, **kind)
    assert trace.first_divergence(a.records, b.records) is None
    assert not any("dropout" in r.op for r in a.records)


def test_mask_and_gradients_of_a_step():
    """Step 2's mask is the definition's at the step's counters, and the layer's
    gradients are those of the masked dy."""
    cfg, p, seed = CONFIGS["tiny_fp32"], 0.25, 77
    st, _ = trace.run(cfg, 2, dropout=p, dropout_seed=seed)
    before = {n: t.clone() for n, t in st.runtime.items()}
    _, tr = trace.run(cfg, 3, "ops", st=st, dropout=p, dropout_seed=seed)
    n = cfg.tokens * cfg.d_model
    kept = oracle.dropout_mask(n, p, seed, 2 * ((n + 3) // 4)).reshape(cfg.tokens, cfg.d_model)
    batch = make_batch(cfg, 2)
    x, dy = (torch.from_numpy(np.ascontiguousarray(batch[k], dtype=np.float32)).cuda() for k in ("x", "dy"))
    # 1 / (1 - 1/4) in float32, one product
    scale = torch.tensor(np.float32(1 / (1 - p)))
    masked = torch.where(torch.from_numpy(kept).cuda(), dy * scale.cuda(), torch.zeros_like(dy))
    prob = st.prob
    routing, h, y = moe.moe_fwd(prob, moe.moe_router_fwd(prob, x, before["wr"]), x, before["w1"], before["w2"])
    dx, dprob, dh = moe.moe_bwd_dgrad_dprob(prob, routing, masked, before["w1"], before["w2"], h)
    dw1, dw2 = moe.moe_bwd_wgrad(prob, routing, x, masked, h, dh)
    dropped = torch.where(torch.from_numpy(kept).cuda(), y * scale.cuda(), torch.zeros_like(y))
    want = {"y_dropped": dropped, "dy_dropped": masked, "dprob": dprob, "dw1": dw1, "dw2": dw2, "dx": dx}
    got = {r.name: r.fp for r in tr.records if r.step == 2}
    for name, t in want.items():
        assert got[name] == f"{moe.moe_fingerprint(t)[1]:016x}", name


def test_refusals():
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(moe.MoeError, match="dropout"):
            trace.run(CONFIGS["tiny_fp32"], 1, dropout=p)
