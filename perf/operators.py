"""Cases for the dense operators beside the expert layer: layer norm, the
gated feed-forward product and the linear map with bias, activation and
residual, forward and backward.

``own`` selects what ``run`` computes: False, the operators in elementary
torch operations in float32, rounded once at the end; True, the framework's
calls.  ``exact`` gives the float64 values.
"""
import math

import torch
import torch.nn.functional as F

own = False

_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # the norm of one new token of a 2048-wide layer while serving: latency
        dict(name="norm_token", op="norm", train=False, dtype="bf16", rows=1, d=2048, add=False),
        # a float32 train step on an odd width, rows that no block divides
        dict(name="norm_train_f32_odd", op="norm", train=True, dtype="f32", rows=1021, d=1001, add=False),
        # a train step's norm over a 16384-token shard, with the residual branch's gradient added
        dict(name="norm_train", op="norm", train=True, dtype="bf16", rows=16384, d=2048, add=True),
        # the shared gated expert for one new token: the weights are all of the traffic
        dict(name="gated_token", op="gated", train=False, dtype="bf16", rows=1, d=2048, f=2048, act="silu"),
        # the same for an uneven batch of sequences in flight and a wider block
        dict(name="gated_batch", op="gated", train=False, dtype="bf16", rows=37, d=2048, f=8192, act="silu"),
        # a train step of the wide shared expert
        dict(name="gated_train", op="gated", train=True, dtype="bf16", rows=4096, d=2048, f=8192, act="silu"),
        # a float32 train step with ragged sizes
        dict(name="gated_train_f32", op="gated", train=True, dtype="f32", rows=777, d=640, f=1000, act="gelu"),
        # down-projection of a few tokens into the residual stream
        dict(name="linear_tokens", op="linear", train=False, dtype="bf16", rows=5, d=8192, f=2048, act="none", bias=True,
             residual=True),
        # a prompt through a biased up-projection with its activation
        dict(name="linear_prompt", op="linear", train=False, dtype="bf16", rows=4096, d=2048, f=8192, act="gelu", bias=True,
             residual=False),
        # a train step of the down-projection into the residual stream
        dict(name="linear_train", op="linear", train=True, dtype="bf16", rows=4096, d=8192, f=2048, act="none", bias=True,
             residual=True),
        # a train step with sizes that no vector width divides
        dict(name="linear_train_odd", op="linear", train=True, dtype="bf16", rows=1500, d=1001, f=517, act="relu2", bias=True,
             residual=False),
    ]


def _spread(rng, lo, hi):
    """Log-uniform whole number of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 64, of 8, or any number."""
    w = _spread(rng, lo, hi)
    step = rng.choice((64, 64, 64, 8, 1))
    return max(step, w // step * step)


def draw(rng):
    op = rng.choice(("norm", "gated", "gated", "linear", "linear"))
    train = rng.random() < 0.5
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    rows = _spread(rng, 1, 16384)
    if op == "norm":
        return dict(op=op, train=train, dtype=dtype, rows=rows, d=_width(rng, 64, 8192), add=train and rng.random() < 0.5)
    d, f = _width(rng, 64, 8192), _width(rng, 64, 8192)
    case = dict(op=op, train=train, dtype=dtype, rows=rows, d=d, f=f)
    if op == "gated":
        case.update(act=rng.choice(("silu", "gelu")))
    else:
        case.update(act=rng.choice(("none", "gelu", "silu", "relu2")), bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    # no dearer than the wide shared expert's train step; float32 at a sixteenth of it
    top = 12 * 4096 * 2048 * 8192 // (16 if dtype == "f32" else 1)
    while work(case)["flops"] > top:
        case["rows"] = max(1, case["rows"] // 2 - 1)
    return case


def prepare(case, seed):
    """Inputs of one call.  Activations are near unit scale (the norm's input
    off centre, with a few rows of other scales), weights scaled by their
    fan-in, gradients small."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPE[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(t)

    n, d = case["rows"], case["d"]
    s = {"case": case}
    if case["op"] == "norm":
        spread = torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))
        s["x"] = ((torch.randn((n, d), generator=g, device="cuda") + 0.3) * spread).to(t)
        s["weight"], s["bias"] = normal(d, scale=0.2, shift=1.0), normal(d, scale=0.1)
        if case["train"]:
            s["dy"] = normal(n, d, scale=0.1)
            s["add"] = normal(n, d, scale=0.1) if case["add"] else None
        return s
    f = case["f"]
    s["x"] = normal(n, d)
    if case["op"] == "gated":
        s["wg"], s["wu"] = normal(d, f, scale=d ** -0.5), normal(d, f, scale=d ** -0.5)
    else:
        s["w"] = normal(d, f, scale=d ** -0.5)
        s["bias"] = normal(f, scale=0.1) if case["bias"] else None
        s["residual"] = normal(n, f) if case["residual"] else None
    if case["train"]:
        s["dy"] = normal(n, f, scale=0.1)
    return s


def _act(name, z):
    """Value and derivative of the activation."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu2":
        r = torch.where(z > 0, z, torch.zeros_like(z))
        return r * r, 2 * r
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    c = 0.5 * (1 + torch.erf(z * 0.7071067811865476))
    return z * c, c + z * torch.exp(-0.5 * z * z) * 0.3989422804014327


def _plain(s):
    case = s["case"]
    t = _TYPE[case["dtype"]]
    x = s["x"].float()
    if case["op"] == "norm":
        w = s["weight"].float()
        c = x - x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        h = c * rstd
        out = {"y": (h * w + s["bias"].float()).to(t)}
        if case["train"]:
            dy = s["dy"].float()
            dh = dy * w
            dx = rstd * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
            if s["add"] is not None:
                dx = dx + s["add"].float()
            out.update(dx=dx.to(t), dweight=(dy * h).sum(0), dbias=dy.sum(0))
        return out
    if case["op"] == "gated":
        wg, wu = s["wg"].float(), s["wu"].float()
        g, u = x @ wg, x @ wu
        v, dv = _act(case["act"], g)
        out = {"a": (v * u).to(t)}
        if case["train"]:
            da = s["dy"].float()
            dg, du = da * u * dv, da * v
            out.update(dx=(dg @ wg.t() + du @ wu.t()).to(t), dwg=(x.t() @ dg).to(t), dwu=(x.t() @ du).to(t))
        return out
    w = s["w"].float()
    z = x @ w
    if s["bias"] is not None:
        z = z + s["bias"].float()
    v, dv = _act(case["act"], z)
    y = v if s["residual"] is None else v + s["residual"].float()
    out = {"y": y.to(t)}
    if case["train"]:
        dz = s["dy"].float() * dv
        out.update(dx=(dz @ w.t()).to(t), dw=(x.t() @ dz).to(t))
        if s["bias"] is not None:
            out["db"] = dz.sum(0).to(t)
    return out


def _framework(s):
    import bitwise_deterministic_moe_amd as moe
    case = s["case"]
    x = s["x"]
    if case["op"] == "norm":
        y, mean, rstd = moe.moe_layernorm_fwd(x, s["weight"], s["bias"], EPS)
        out = {"y": y}
        if case["train"]:
            out["dx"], out["dweight"], out["dbias"] = moe.moe_layernorm_bwd(s["dy"], x, s["weight"], mean, rstd, dx_add=s["add"])
        return out
    if case["op"] == "gated":
        a, g, u = moe.moe_glu_fwd(x, s["wg"], s["wu"], case["act"], save=case["train"])
        out = {"a": a}
        if case["train"]:
            out["dx"], out["dwg"], out["dwu"] = moe.moe_glu_bwd(s["dy"], x, s["wg"], s["wu"], g, u, case["act"], grad_dtype=x.dtype)
        return out
    y, z = moe.moe_linear_fwd(x, s["w"], s["bias"], s["residual"], case["act"], save_z=case["train"] and case["act"] != "none")
    out = {"y": y}
    if case["train"]:
        dx, dw, db = moe.moe_linear_bwd(s["dy"], x, s["w"], z, case["act"], need_db=s["bias"] is not None, grad_dtype=x.dtype)
        out.update(dx=dx, dw=dw)
        if db is not None:
            out["db"] = db
    return out


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def work(case):
    """Bytes with each input read once and each output written once, and the
    operations of the formulas."""
    e, n, d = _SIZE[case["dtype"]], case["rows"], case["d"]
    if case["op"] == "norm":
        b, o = (2 * n * d + 2 * d) * e, 8 * n * d
        if case["train"]:
            b += (2 + bool(case["add"])) * n * d * e + 2 * d * 4
            o += 14 * n * d
        return {"bytes": b, "flops": o}
    f = case["f"]
    m = 2 if case["op"] == "gated" else 1      # weight matrices
    b = (n * d + m * d * f + n * f) * e
    o = 2 * m * n * d * f
    if case["op"] == "linear":
        b += ((f if case["bias"] else 0) + (n * f if case["residual"] else 0)) * e
    if case["train"]:
        b += (n * f + n * d + m * d * f) * e
        o += 4 * m * n * d * f
        if case["op"] == "linear" and case["bias"]:
            b += f * e
    return {"bytes": b, "flops": o}


def exact(case, seed):
    """The definition in float64: library functions and automatic
    differentiation."""
    s = prepare(case, seed)
    v = {k: a.double() for k, a in s.items() if torch.is_tensor(a)}
    x = v["x"].requires_grad_(case["train"])
    if case["op"] == "norm":
        names = {"dx": "x", "dweight": "weight", "dbias": "bias"}
        y = F.layer_norm(x, (case["d"],), v["weight"].requires_grad_(case["train"]), v["bias"].requires_grad_(case["train"]), EPS)
        out = {"y": y}
    elif case["op"] == "gated":
        names = {"dx": "x", "dwg": "wg", "dwu": "wu"}
        gate = x @ v["wg"].requires_grad_(case["train"])
        y = (F.silu if case["act"] == "silu" else F.gelu)(gate) * (x @ v["wu"].requires_grad_(case["train"]))
        out = {"a": y}
    else:
        names = {"dx": "x", "dw": "w"}
        z = x @ v["w"].requires_grad_(case["train"])
        if case["bias"]:
            names["db"] = "bias"
            z = z + v["bias"].requires_grad_(case["train"])
        y = {"none": lambda a: a, "gelu": F.gelu, "silu": F.silu, "relu2": lambda a: F.relu(a).square()}[case["act"]](z)
        if case["residual"]:
            y = y + v["residual"]
        out = {"y": y}
    if case["train"]:
        grads = torch.autograd.grad(y, [v[k] for k in names.values()], v["dy"])
        out.update(zip(names, grads))
        if case["op"] == "norm" and case["add"]:
            out["dx"] = out["dx"] + v["add"]
    return {k: a.detach() for k, a in out.items()}
