"""Cases for the pieces of an expert layer that a user puts together: rows
sorted by expert and back with weights, products in 8-bit integers, and
dropout into the residual stream.

``own`` selects what ``run`` computes: False, the operators in elementary
torch operations in float32, rounded once at the end; True, the framework's
calls.  ``exact`` gives the float64 values.
"""
import math

import numpy as np
import torch

own = False

_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
TINY = 2.0 ** -100        # rows of smaller numbers are quantised to zeros


def listed():
    return [
        # one new token of a 512-expert layer sent to its 22 experts: latency
        dict(name="dispatch_token", op="dispatch", train=False, dtype="bf16", tokens=1, k=22, experts=512, local=512, d=2048),
        # a train step's tokens sorted and copied for their experts, and the gradient back
        dict(name="dispatch_train", op="dispatch", train=True, dtype="bf16", tokens=4096, k=22, experts=512, local=512, d=2048),
        # an expert-parallel rank picks the rows of its 4 experts out of 16384 tokens
        dict(name="dispatch_shard", op="dispatch", train=False, dtype="bf16", tokens=16384, k=22, experts=512, local=4, d=2048),
        # a small float32 step of an odd width, the gradient of the weights with it
        dict(name="combine_odd", op="combine", train=True, dtype="f32", tokens=317, k=5, experts=13, local=13, d=1001,
             residual=False),
        # a train step's rows weighted, summed and added to the residual stream, and its gradients
        dict(name="combine_train", op="combine", train=True, dtype="bf16", tokens=4096, k=22, experts=512, local=512, d=2048,
             residual=True),
        # the projection of one new token: the weights are all of the traffic
        dict(name="int8_token", op="int8", dtype="bf16", rows=1, d=2048, f=2048, act="none", bias=False, residual=True),
        # an uneven batch of sequences in flight
        dict(name="int8_batch", op="int8", dtype="bf16", rows=37, d=2048, f=8192, act="silu", bias=True, residual=False),
        # a prompt through a biased up-projection with its activation
        dict(name="int8_prompt", op="int8", dtype="bf16", rows=4096, d=2048, f=8192, act="gelu", bias=True, residual=False),
        # one new token through the up-projections of its 22 experts of 512
        dict(name="experts_token", op="experts", dtype="bf16", tokens=1, k=22, experts=512, d=2048, f=2048, act="relu2"),
        # a prompt through the up-projections of 8 experts, two for each token
        dict(name="experts_prompt", op="experts", dtype="bf16", tokens=4096, k=2, experts=8, d=1024, f=2048, act="relu2"),
        # a small float32 step of an odd width
        dict(name="dropout_odd", op="dropout", train=True, dtype="f32", rows=1021, d=1001, p=0.25, residual=False),
        # a train step's 16384 tokens on their way into the residual stream
        dict(name="dropout_train", op="dropout", train=True, dtype="bf16", rows=16384, d=2048, p=0.1, residual=True),
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
    op = rng.choice(("dispatch", "combine", "int8", "int8", "experts", "experts", "dropout"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    train = rng.random() < 0.5
    if op == "dropout":
        case = dict(op=op, train=train, dtype=dtype, rows=_spread(rng, 1, 16384), d=_width(rng, 64, 8192),
                    p=rng.choice((0.05, 0.1, 0.3, 0.5)), residual=rng.random() < 0.5)
        while case["rows"] * case["d"] > 16384 * 2048:
            case["rows"] //= 2
        return case
    if op == "int8":
        case = dict(op=op, dtype=dtype, rows=_spread(rng, 1, 16384), d=_width(rng, 64, 8192), f=_width(rng, 64, 8192),
                    act=rng.choice(("none", "gelu", "silu", "relu2")), bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        while work(case)["flops"] > 2 * 4096 * 2048 * 8192:
            case["rows"] //= 2
        return case
    experts = _spread(rng, 2, 512)
    k = _spread(rng, 1, min(experts, 22))
    case = dict(op=op, dtype=dtype, tokens=_spread(rng, 1, 16384), k=k, experts=experts)
    if op == "experts":
        case.update(d=_width(rng, 64, 4096), f=_width(rng, 64, 4096), act=rng.choice(("none", "silu", "relu2")))
        # the weights of at most 512 experts of 2048 x 2048, and rows that the plain form can pad to whole experts
        while experts * case["d"] * case["f"] > 512 * 2048 * 2048:
            case["d"], case["f"] = max(64, case["d"] // 2), max(64, case["f"] // 2)
        while (case["tokens"] * k * case["d"] * case["f"] > 4096 * 2048 * 8192
               or case["tokens"] > 1 and experts * case["tokens"] * case["d"] * case["f"] > 4096 * 4 * 2048 * 8192):
            case["tokens"] //= 2
        return case
    part = rng.choice((1, 1, 2, 8))
    case.update(train=train, local=max(1, experts // part), d=_width(rng, 64, 8192))
    if op == "combine":
        case.update(residual=rng.random() < 0.5)
    while case["tokens"] * k * case["d"] * _SIZE[dtype] > 4096 * 22 * 2048 * 2:
        case["tokens"] //= 2
    return case


def _choice(case, g):
    """[T, k] expert numbers: the largest of biased scores, so that loads differ."""
    n, e = case["tokens"], case["experts"]
    score = torch.randn((n, e), generator=g, device="cuda") + 0.7 * torch.randn((1, e), generator=g, device="cuda")
    return score.topk(case["k"], dim=1).indices.to(torch.int32)


def _sorted(idx, local):
    """The slots of idx [T, k] sorted by expert, stable: each slot's row (-1 for
    an expert that is not local), the experts' first rows, and each row's slot."""
    e = idx.reshape(-1).long()
    here = (e >= 0) & (e < local)
    e = torch.where(here, e, torch.full_like(e, local))
    order = torch.sort(e, stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.zeros(local + 1, dtype=torch.long, device=e.device).index_add_(0, e, torch.ones_like(e))[:local]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    slot_row = torch.where(here, row, torch.full_like(row, -1))
    return slot_row.to(torch.int32).reshape(idx.shape), offsets.to(torch.int32), order


def prepare(case, seed):
    """Inputs of one call.  Activations are near unit scale, gradients small,
    the numbers of a token's weights those of a softmax; weights are codes of
    normal numbers with their scales, as they are laid out once for serving."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPE[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(t)

    def codes(*shape):
        """int8 codes [..., f, d up to 16] of normal weights, and scales [..., f]."""
        n = shape[-1]
        c = torch.zeros(shape[:-1] + ((n + 15) // 16 * 16,), dtype=torch.int8, device="cuda")
        for part in (c if c.dim() == 3 else (c,)):
            w = torch.randn((shape[-2], n), generator=g, device="cuda")
            part[:, :n] = torch.round(w * (127 / w.abs().amax(1, keepdim=True))).to(torch.int8)
        s = (torch.rand(shape[:-1], generator=g, device="cuda") + 3) * (n ** -0.5 / 127)
        return c, s

    d, s = case["d"], {"case": case}
    if case["op"] == "dropout":
        s["x"] = normal(case["rows"], d)
        s["rng"] = torch.tensor([seed * 7919 + 13, seed % 1000 * 12345677], dtype=torch.int64, device="cuda")
        s["residual"] = normal(case["rows"], d) if case["residual"] else None
        s["dy"] = normal(case["rows"], d, scale=0.1) if case["train"] else None
        return s
    if case["op"] == "int8":
        s["x"] = normal(case["rows"], d)
        s["w"], s["w_scale"] = codes(case["f"], d)
        s["bias"] = normal(case["f"], scale=0.1) if case["bias"] else None
        s["residual"] = normal(case["rows"], case["f"]) if case["residual"] else None
        return s
    idx = _choice(case, g)
    if case["op"] == "experts":
        s["x"] = normal(idx.numel(), d)
        s["offsets"] = _sorted(idx, case["experts"])[1]
        s["w"], s["w_scale"] = codes(case["experts"], case["f"], d)
        return s
    most = case["tokens"] * min(case["k"], case["local"])     # rows at most: a token's experts are different ones
    if case["op"] == "dispatch":
        s["idx"], s["x"] = idx, normal(case["tokens"], d)
        # the buffer of rows that the step keeps; rows behind the last one stay as they are
        s["rows"] = torch.zeros((most, d), dtype=t, device="cuda")
        s["drows"] = normal(most, d, scale=0.1) if case["train"] else None
        return s
    s["slot_row"], s["offsets"], s["row_slot"] = _sorted(idx, case["local"])
    s["prob"] = torch.softmax(torch.randn(idx.shape, generator=g, device="cuda"), 1)
    s["y_rows"] = normal(most, d)
    s["residual"] = normal(case["tokens"], d) if case["residual"] else None
    if case["train"]:
        s["dy"] = normal(case["tokens"], d, scale=0.1)
        s["rows"] = torch.zeros((most, d), dtype=t, device="cuda")
    return s


def _act(name, z):
    if name == "relu2":
        r = torch.where(z > 0, z, torch.zeros_like(z))
        return r * r
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * (0.5 * (1 + torch.erf(z * 0.7071067811865476)))
    return z


def _quantised(x):
    """Codes and scales of the rows of x: 127 x / max |x| to the nearest, in
    float64, where a float32 quotient next to a half may fall on its other side."""
    top = x.abs().amax(1, keepdim=True)
    some = top >= TINY
    q = torch.round(x.double() * 127 / torch.where(some, top, torch.ones_like(top)).double())
    return (q * some).float(), torch.where(some, top / 127, torch.zeros_like(top))


def _uniform(n, seed, first):
    """The first n 32-bit words of Philox 4x32 of 10 rounds from counter
    `first` on, under the key `seed`, as int64 (products wrap at 64 bits)."""
    low = 0xFFFFFFFF
    c = torch.arange((n + 3) // 4, device="cuda") + first
    c0, c1 = c & low, (c >> 32) & low
    c2 = c3 = torch.zeros_like(c0)
    k0, k1 = seed & low, (seed >> 32) & low

    def rounds(c0, c1, c2, c3, k0, k1):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        return ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low

    for r in range(10):
        c0, c1, c2, c3 = rounds(c0, c1, c2, c3, (k0 + r * 0x9E3779B9) & low, (k1 + r * 0xBB67AE85) & low)
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _gathered(rows, slot_row):
    """Rows of the slots, zeros for a slot without one."""
    at = slot_row.long()
    r = rows[at.clamp(min=0)].float()
    return torch.where((at >= 0)[..., None], r, torch.zeros_like(r))


def _written(out, offsets, values):
    """out with the rows up to the last expert's last one from `values`."""
    there = torch.arange(out.shape[0], device=out.device) < offsets[-1]
    return torch.where(there[:, None], values.to(out.dtype), out)


def _plain(s):
    case, t = s["case"], _TYPE[s["case"]["dtype"]]
    if case["op"] == "dropout":
        x = s["x"].float()
        kept = (_uniform(x.numel(), s["rng"][0], s["rng"][1]) >= int(round(case["p"] * 2 ** 32))).reshape(x.shape)
        y = torch.where(kept, x * (1 / (1 - case["p"])), torch.zeros_like(x))
        out = {"y": (y if s["residual"] is None else y + s["residual"].float()).to(t)}
        if case["train"]:
            out["dx"] = torch.where(kept, s["dy"].float() * (1 / (1 - case["p"])), torch.zeros_like(x)).to(t)
        return out
    if case["op"] == "dispatch":
        slot_row, offsets, slot = _sorted(s["idx"], case["local"])
        x = s["x"][slot[:s["rows"].shape[0]] // case["k"]]
        out = {"slot_row": slot_row, "offsets": offsets, "rows": _written(s["rows"], offsets, x)}
        if case["train"]:
            out["dx"] = _gathered(s["drows"], slot_row).sum(1).to(t)
        return out
    if case["op"] == "combine":
        r = _gathered(s["y_rows"], s["slot_row"])
        y = (s["prob"][..., None] * r).sum(1)
        out = {"y": (y if s["residual"] is None else y + s["residual"].float()).to(t)}
        if case["train"]:
            dy, slot = s["dy"].float(), s["row_slot"][:s["rows"].shape[0]]
            d = s["prob"].reshape(-1)[slot, None] * dy[slot // case["k"]]
            out["drows"] = _written(s["rows"], s["offsets"], d)
            out["dprob"] = (dy[:, None, :] * r).sum(2)
        return out
    q, scale = _quantised(s["x"].float())
    if case["op"] == "int8":
        z = (q @ s["w"][:, :case["d"]].float().t()) * scale * s["w_scale"]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(case["act"], z)
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(t)}
    n, e = q.shape[0], case["experts"]
    row = torch.arange(n, device="cuda")
    of = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    if n <= e:         # each row beside its own expert's weights
        w = s["w"][of][:, :, :case["d"]].float()
        z = torch.bmm(w, q[:, :, None]).squeeze(2)
    else:              # every expert's rows padded to the number of tokens
        at = s["offsets"][:-1].long()[:, None] + torch.arange(case["tokens"], device="cuda")
        a = q[at.clamp(max=n - 1)].transpose(1, 2).contiguous()
        z = torch.bmm(s["w"][:, :, :case["d"]].float(), a).transpose(1, 2)[of, row - s["offsets"].long()[of]]
    return {"y": _act(case["act"], z * scale * s["w_scale"][of]).to(t)}


def _framework(s):
    import bitwise_deterministic_moe_amd as moe
    case = s["case"]
    if case["op"] == "dropout":
        out = {"y": moe.moe_dropout_fwd(s["x"], case["p"], s["rng"], residual=s["residual"])}
        if case["train"]:
            out["dx"] = moe.moe_dropout_bwd(s["dy"], case["p"], s["rng"])
        return out
    if case["op"] == "dispatch":
        slot_row, offsets, _ = moe.moe_sort(s["idx"], case["local"])
        out = {"slot_row": slot_row, "offsets": offsets, "rows": moe.moe_permute_fwd(s["x"], slot_row, rows=s["rows"])}
        if case["train"]:
            out["dx"] = moe.moe_permute_bwd(s["drows"], slot_row)
        return out
    if case["op"] == "combine":
        out = {"y": moe.moe_unpermute_fwd(s["y_rows"], s["slot_row"], s["prob"], residual=s["residual"])}
        if case["train"]:
            out["drows"], out["dprob"] = moe.moe_unpermute_bwd(s["dy"], s["y_rows"], s["slot_row"], s["prob"], drows=s["rows"])
        return out
    if case["op"] == "int8":
        return {"y": moe.moe_int8_linear(s["x"], s["w"], s["w_scale"], bias=s["bias"], residual=s["residual"], act=case["act"])}
    return {"y": moe.moe_int8_experts(s["x"], s["w"], s["w_scale"], s["offsets"], act=case["act"])}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def work(case):
    """Bytes with each input read once and each output written once, and the
    operations of the formulas."""
    z, d = _SIZE[case["dtype"]], case["d"]
    if case["op"] == "dropout":
        n = case["rows"] * d
        return {"bytes": n * z * (2 + case["residual"] + 2 * case["train"]), "flops": n * (2 + case["train"])}
    if case["op"] == "int8":
        n, f = case["rows"], case["f"]
        return {"bytes": n * d * z + f * d + 4 * f + n * f * z * (1 + case["residual"]) + (f * z if case["bias"] else 0),
                "flops": 2 * n * d * f}
    n, k, e = case["tokens"], case["k"], case["experts"]
    if case["op"] == "experts":
        f = case["f"]
        used = e * (1 - (1 - k / e) ** n)       # experts with a row
        return {"bytes": n * k * (d + f) * z + used * f * (d + 4) + 4 * e, "flops": 2 * n * k * d * f}
    r = n * k * case["local"] / e                # rows
    if case["op"] == "dispatch":
        return {"bytes": (1 + case["train"]) * (n + r) * d * z + 8 * n * k + 4 * case["local"],
                "flops": r * d * case["train"] + n * k}
    b, o = (r + n * (1 + case["residual"])) * d * z + 8 * n * k, 2 * r * d
    if case["train"]:
        b, o = b + (2 * r + n) * d * z + 12 * n * k, o + 3 * r * d
    return {"bytes": b, "flops": o}


def _numpy_words(n, seed, first):
    """Philox 4x32-10 with numpy's unsigned integers."""
    c = np.zeros((4, (n + 3) // 4), dtype=np.uint64)
    at = np.arange(c.shape[1], dtype=np.uint64) + np.uint64(first)
    low = np.uint64(0xFFFFFFFF)
    c[0], c[1] = at & low, at >> np.uint64(32)
    key = [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = np.stack((b >> np.uint64(32) ^ c[1] ^ np.uint64(key[0]), b & low,
                      a >> np.uint64(32) ^ c[3] ^ np.uint64(key[1]), a & low))
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.ascontiguousarray(c.T).reshape(-1)[:n]


def exact(case, seed):
    """The definitions in float64, expert by expert and slot by slot."""
    s = prepare(case, seed)
    v = {n: a.double() for n, a in s.items() if torch.is_tensor(a) and a.is_floating_point()}
    if case["op"] == "dropout":
        x = v["x"]
        u = _numpy_words(x.numel(), int(s["rng"][0]), int(s["rng"][1]))
        mask = torch.from_numpy((u.astype(np.float64) >= case["p"] * 2.0 ** 32).astype(np.float64)).cuda().reshape(x.shape)
        mask = mask / (1 - case["p"])
        out = {"y": x.mul(mask) + v.get("residual", 0)}
        if case["train"]:
            out["dx"] = v["dy"] * mask
        return out
    if case["op"] == "dispatch":
        idx = s["idx"].cpu().numpy().reshape(-1)
        order = np.argsort(np.where(idx < case["local"], idx, case["local"]), kind="stable")
        r = int((idx < case["local"]).sum())
        slot_row = np.full(idx.size, -1, np.int32)
        slot_row[order[:r]] = np.arange(r)
        offsets = np.concatenate(([0], np.cumsum(np.bincount(idx[idx < case["local"]], minlength=case["local"]))))
        token = torch.from_numpy(order[:r] // case["k"]).cuda()
        rows = v["rows"].clone()
        rows[:r] = v["x"][token]
        out = {"slot_row": torch.from_numpy(slot_row.reshape(s["idx"].shape)), "offsets": torch.from_numpy(offsets.astype(np.int32)),
               "rows": rows}
        if case["train"]:
            out["dx"] = torch.zeros_like(v["x"]).index_add_(0, token, v["drows"][:r])
        return out
    if case["op"] == "combine":
        y = v["residual"].clone() if case["residual"] else torch.zeros((case["tokens"], case["d"]), dtype=torch.float64, device="cuda")
        out = {"y": y}
        if case["train"]:
            out.update(drows=v["rows"].clone(), dprob=torch.zeros_like(v["prob"]))
        for j in range(case["k"]):
            row = s["slot_row"][:, j].long()
            t = (row >= 0).nonzero().squeeze(1)
            row, p = row[t], v["prob"][t, j, None]
            y[t] += p * v["y_rows"][row]
            if case["train"]:
                out["drows"][row] = p * v["dy"][t]
                out["dprob"][t, j] = (v["dy"][t] * v["y_rows"][row]).sum(1)
        return out
    x = v["x"]
    top = x.abs().max(1, keepdim=True).values
    scale = torch.where(top < TINY, torch.zeros_like(top), top / 127)
    q = torch.where(top < TINY, torch.zeros_like(x), (x / top * 127).round())
    # 127 x / top at a half, where the quotient above may be off by its rounding: the even neighbour
    half = (254 * x).fmod(2 * top).abs() == top
    q = torch.where(half & (top >= TINY), 2 * (x / top * 127 / 2).round(), q)
    act = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "relu2": lambda z: z.clamp(min=0) ** 2}[case["act"]]
    if case["op"] == "int8":
        z = q @ s["w"][:, :case["d"]].double().t() * scale * v["w_scale"]
        return {"y": act(z + v.get("bias", 0)) + v.get("residual", 0)}
    y = torch.empty((x.shape[0], case["f"]), dtype=torch.float64, device="cuda")
    at = s["offsets"].tolist()
    for e in range(case["experts"]):
        if at[e] < at[e + 1]:
            part = slice(at[e], at[e + 1])
            y[part] = act(q[part] @ s["w"][e, :, :case["d"]].double().t() * scale[part] * v["w_scale"][e])
    return {"y": y}
