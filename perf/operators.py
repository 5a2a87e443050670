"""The operators of a decoding step's expert layer: residual RMS norm with 8-bit output, router choice, products with
4-bit weights, and the expert layer for few tokens.

Every case is served in two forms: the plain one (elementary torch operations in float32) and the library's own kernels.
Sizes follow the workloads of this package: rows of 7168 with expert width 2048, 64 experts, top-8 and 8 experts per
GPU (expert parallelism), 4096 and 8192 square products (tensor parallelism), 1024 tokens on each of 8 shards."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # the norm before the expert layer of one decoded token
        dict(name="norm_1x7168_e4m3", op="norm", rows=1, n=7168, res=True, out="e4m3", group=0),
        # the same norm over a prompt: 8 shards of 1024 tokens, scales per 128 columns as 8-bit dispatch wants them
        dict(name="norm_8192x7168_e4m3_g128", op="norm", rows=8192, n=7168, res=True, out="e4m3", group=128),
        # a ragged batch with a width that no vector divides, first layer (no residual yet), int8 rows
        dict(name="norm_333x5003_i8", op="norm", rows=333, n=5003, res=False, out="i8", group=0),
        # the router of one decoded token
        dict(name="route_1x64_top8", op="route", rows=1, experts=64, k=8, score="softmax", renorm=True, logits="f32"),
        # the router of a prompt, many experts, bf16 logits (equal logits are common)
        dict(name="route_8192x256_top8_bf16", op="route", rows=8192, experts=256, k=8, score="sigmoid", renorm=True, logits="bf16"),
        # a projection of one decoded token
        dict(name="w4_1x2048x7168_g128", op="w4", rows=1, n=2048, k=7168, group=128, zero=False, x="bf16", xgroup=0),
        # a few sequences, sizes that no tile divides, small groups with zero points
        dict(name="w4_5x8199x7200_g32z", op="w4", rows=5, n=8199, k=7200, group=32, zero=True, x="bf16", xgroup=0),
        # a full decoding batch on the square product, 8-bit rows from the norm
        dict(name="w4_64x8192x8192_g64z_i8", op="w4", rows=64, n=8192, k=8192, group=64, zero=True, x="i8", xgroup=0),
        # a small model's expert layer, three tokens
        dict(name="moe_3t_e8_512x768", op="moe", rows=3, hidden=512, width=768, experts=8, local=8, base=0, k=2, group=0, zero=False, x="bf16", xgroup=0),
        # one decoded token, every expert on this GPU
        dict(name="moe_1t_e64_7168x2048", op="moe", rows=1, hidden=7168, width=2048, experts=64, local=64, base=0, k=8, group=0, zero=False, x="bf16", xgroup=0),
        # this GPU's 8 of 64 experts for 16 tokens; some tokens have no pick here
        dict(name="moe_16t_e8of64_7168x2048", op="moe", rows=16, hidden=7168, width=2048, experts=64, local=8, base=8, k=8, group=0, zero=False, x="bf16", xgroup=0),
        # a full decoding batch over 64 experts with 4-bit weights and 8-bit rows
        dict(name="moe_64t_e64_w4g128_e4m3", op="moe", rows=64, hidden=7168, width=2048, experts=64, local=64, base=0, k=8, group=128, zero=False, x="e4m3", xgroup=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _kind(rng, k):
    """Type of the activations; 8-bit ones have a scale a row or a scale each 128 columns."""
    x = rng.choice(["bf16", "i8", "e4m3"])
    return dict(x=x, xgroup=rng.choice([0, 128]) if x != "bf16" and k % 128 == 0 else 0)


def draw(rng):
    op = rng.choice(["norm", "route", "w4", "moe"])
    if op == "norm":
        group = rng.choice([0, 128])
        n = 128 * rng.randint(1, 64) if group else _log(rng, 64, 8192)
        return dict(op=op, rows=_log(rng, 1, 7000), n=n, res=rng.random() < 0.7, out=rng.choice(["bf16", "e4m3", "i8"]), group=group)
    if op == "route":
        experts = rng.choice([rng.randint(8, 64), rng.randint(65, 256)])
        return dict(op=op, rows=_log(rng, 1, 8192), experts=experts, k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.7, logits=rng.choice(["f32", "bf16"]))
    if op == "w4":
        group = rng.choice([32, 64, 128])
        k = group * max(1, _log(rng, 512, 8192) // group)
        return dict(op=op, rows=_log(rng, 1, 64), n=_log(rng, 256, 8192), k=k, group=group, zero=rng.random() < 0.5, **_kind(rng, k))
    group = rng.choice([0, 0, 32, 64, 128])
    unit = max(group, 32)
    experts = rng.choice([8, 16, 48, 64] if group else [8, 16])
    local = rng.choice([experts, max(2, experts // 8)])
    hidden = unit * max(1, _log(rng, 512, 6144) // unit)
    return dict(op=op, rows=_log(rng, 1, 64), hidden=hidden, width=unit * max(1, _log(rng, 256, 2048) // unit),
                experts=experts, local=local, base=rng.choice([0, experts - local]), k=rng.randint(1, 8), group=group, zero=rng.random() < 0.5,
                **_kind(rng, hidden))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows8(x, kind, group):
    """Rows as the 8-bit norm leaves them: codes and float32 scales, one a row or one each `group` columns."""
    top = 127.0 if kind == "i8" else 448.0
    v = x.unflatten(-1, (-1, group or x.shape[1]))
    a = v.abs().amax(-1).clamp_min(1e-20)
    v = (v * (top / a)[..., None]).flatten(-2)
    return (torch.round(v).to(torch.int8) if kind == "i8" else v.to(E4M3)), a / top


def _acts(g, rows, k, kind, group):
    """Activations of `rows` tokens: normal, a few columns larger than the rest."""
    x = torch.randn(rows, k, generator=g, device=DEV)
    x[:, ::97] *= 6.0
    return (x.to(BF16), None) if kind == "bf16" else _rows8(x, kind, group)


def _weight4(g, lead, n, k, group, zero):
    q = torch.randint(0, 256, (*lead, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = ((torch.rand(*lead, n, k // group, generator=g, device=DEV) + 0.5) * (0.22 / math.sqrt(k))).to(BF16)
    z = torch.randint(0, 16, (*lead, n, k // group), generator=g, device=DEV, dtype=torch.uint8) if zero else None
    return q, s, z


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "norm":
        r, n = c["rows"], c["n"]
        c["xin"] = torch.randn(r, n, generator=g, device=DEV).to(BF16)
        c["r"] = (3 * torch.randn(r, n, generator=g, device=DEV)).to(BF16) if c["res"] else None
        c["gamma"] = (1 + 0.2 * torch.randn(n, generator=g, device=DEV)).to(BF16)
    elif c["op"] == "route":
        l = 2 * torch.randn(c["rows"], c["experts"], generator=g, device=DEV)
        c["l"] = l.to(BF16) if c["logits"] == "bf16" else l
    elif c["op"] == "w4":
        c["xq"], c["xs"] = _acts(g, c["rows"], c["k"], c["x"], c["xgroup"])
        c["q"], c["s"], c["z"] = _weight4(g, (), c["n"], c["k"], c["group"], c["zero"])
    else:
        t, h, f, e, k = c["rows"], c["hidden"], c["width"], c["local"], c["k"]
        c["xq"], c["xs"] = _acts(g, t, h, c["x"], c["xgroup"])
        if c["group"]:
            c["w1"] = _weight4(g, (e,), 2 * f, h, c["group"], c["zero"])
            c["w2"] = _weight4(g, (e,), h, f, c["group"], c["zero"])
        else:
            c["w1"] = torch.randn(e, 2 * f, h, generator=g, device=DEV, dtype=BF16).mul_(1 / math.sqrt(h))
            c["w2"] = torch.randn(e, h, f, generator=g, device=DEV, dtype=BF16).mul_(1 / math.sqrt(f))
        u = torch.rand(t, c["experts"], generator=g, device=DEV)
        c["topk"] = torch.argsort(u, 1)[:, :k].to(torch.int32).contiguous()
        w = torch.rand(t, k, generator=g, device=DEV) + 0.1
        c["tw"] = w / w.sum(1, keepdim=True)
    return c


# -------------------------------------------------------------- plain form
def _unpack(q, s, z, group):
    """4-bit weights as float32: the low nibble of a byte comes first."""
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).float().unflatten(-1, (-1, group))
    v = v - (8.0 if z is None else z.float().unsqueeze(-1))
    return (v * s.float().unsqueeze(-1)).flatten(-2)


def _plain_x(c):
    x = c["xq"].float()
    if c["xs"] is None:
        return x
    return (x.unflatten(-1, (c["xs"].shape[1], -1)) * c["xs"].unsqueeze(-1)).flatten(-2)


def _plain_norm(c):
    h = c["xin"].float()
    if c["res"]:
        h = h + c["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * c["gamma"].float()
    out = {"sum": h.to(BF16)} if c["res"] else {}
    if c["out"] == "bf16":
        return out | {"y": y.to(BF16)}
    top = 127.0 if c["out"] == "i8" else 448.0
    v = y.unflatten(-1, (-1, c["group"] or c["n"]))
    a = v.abs().amax(-1, keepdim=True)
    v = (v * torch.where(a > 0, top / a, 0.0)).flatten(-2)
    s = (a / top).squeeze(-1)
    if c["out"] == "e4m3":
        return out | {"q": v.to(E4M3), "scale": s}
    return out | {"y": _values8(torch.round(v), s, c["n"]), "scale": s}


def _values8(q, s, n):
    """What int8 codes and their scales stand for."""
    return (q.float().unflatten(-1, (s.shape[-1], n // s.shape[-1])) * s.unsqueeze(-1)).flatten(-2).to(BF16)


def _plain_route(c):
    l = c["l"].float()
    idx = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    w = p.gather(1, idx)
    return idx.to(torch.int32), w / w.sum(-1, keepdim=True) if c["renorm"] else w


def _plain_w4(c):
    return (_plain_x(c) @ _unpack(c["q"], c["s"], c["z"], c["group"]).t()).to(BF16)


def _plain_moe(c):
    x, f, e = _plain_x(c), c["width"], c["local"]
    pick = c["topk"].long() - c["base"]
    here = (pick >= 0) & (pick < e)
    pick, tw = pick.clamp(0, e - 1), c["tw"] * here
    few = pick.numel() < e  # fewer picks than experts: each pick's weights, else every expert on every token
    w1 = (tuple(v[pick.flatten()] if v is not None else None for v in c["w1"]) if few else c["w1"]) if c["group"] else (c["w1"][pick.flatten()] if few else c["w1"])
    w2 = (tuple(v[pick.flatten()] if v is not None else None for v in c["w2"]) if few else c["w2"]) if c["group"] else (c["w2"][pick.flatten()] if few else c["w2"])
    w1 = _unpack(*w1, c["group"]) if c["group"] else w1.float()
    w2 = _unpack(*w2, c["group"]) if c["group"] else w2.float()
    if few:
        gu = torch.bmm(w1, x.repeat_interleave(c["k"], 0).unsqueeze(-1)).squeeze(-1)
        a = gu[:, :f] / (1 + torch.exp(-gu[:, :f])) * gu[:, f:]
        y = torch.bmm(w2, a.unsqueeze(-1)).squeeze(-1)
        return (y.unflatten(0, (-1, c["k"])) * tw.unsqueeze(-1)).sum(1).to(BF16)
    gu = torch.matmul(x, w1.transpose(1, 2))
    a = gu[..., :f] / (1 + torch.exp(-gu[..., :f])) * gu[..., f:]
    gate = torch.zeros(x.shape[0], e, device=x.device).scatter_add_(1, pick, tw)
    return (torch.matmul(a, w2.transpose(1, 2)) * gate.t().unsqueeze(-1)).sum(0).to(BF16)


def _own(c):
    from sync_protocols_amd import ops

    if c["op"] == "norm":
        r = ops.add_rmsnorm(c["xin"], c["gamma"], residual=c["r"], eps=EPS, out=c["out"], group=c["group"] if c["out"] != "bf16" else 0)
        out = {"sum": r.sum} if c["res"] else {}
        if c["out"] == "bf16":
            return out | {"y": r.y}
        if c["out"] == "e4m3":
            return out | {"q": r.q, "scale": r.scale}
        return out | {"y": _values8(r.q, r.scale, c["n"]), "scale": r.scale}
    if c["op"] == "route":
        return ops.moe_route(c["l"], c["k"], score=c["score"], renorm=c["renorm"])
    if c["op"] == "w4":
        return ops.w4_linear(c["xq"], ops.W4Weight(c["q"], c["s"], c["z"]), x_scale=c["xs"])
    w1, w2 = (ops.W4Weight(*c["w1"]), ops.W4Weight(*c["w2"])) if c["group"] else (c["w1"], c["w2"])
    return ops.moe_few(c["xq"], w1, w2, c["topk"], c["tw"], expert_base=c["base"], x_scale=c["xs"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "route": _plain_route, "w4": _plain_w4, "moe": _plain_moe}[state["op"]](state)


# -------------------------------------------------------------------- work
_XB = {"bf16": 2, "i8": 1, "e4m3": 1}


def work(case):
    c = case
    if c["op"] == "norm":
        e = c["rows"] * c["n"]
        scales = 0 if c["out"] == "bf16" else 4 * c["rows"] * (c["n"] // c["group"] if c["group"] else 1)
        return {"bytes": e * (2 + 4 * c["res"] + _XB[c["out"]]) + 2 * c["n"] + scales, "flops": 8 * e}
    if c["op"] == "route":
        e = c["rows"] * c["experts"]
        return {"bytes": e * (4 if c["logits"] == "f32" else 2) + 8 * c["rows"] * c["k"], "flops": 4 * e}
    if c["op"] == "w4":
        per = 0.5 + (2 + c["zero"]) / c["group"]
        return {"bytes": c["n"] * c["k"] * per + c["rows"] * (c["k"] * _XB[c["x"]] + 2 * c["n"]), "flops": 2 * c["rows"] * c["n"] * c["k"]}
    per = 0.5 + (2 + c["zero"]) / c["group"] if c["group"] else 2
    share = min(1.0, c["k"] / c["experts"])
    active = c["local"] * (1 - (1 - share) ** c["rows"])  # expected number of experts that some token picks
    pairs = c["rows"] * c["k"] * c["local"] / c["experts"]
    return {"bytes": active * 3 * c["hidden"] * c["width"] * per + c["rows"] * c["hidden"] * (_XB[c["x"]] + 2) + 8 * c["rows"] * c["k"],
            "flops": 6 * pairs * c["hidden"] * c["width"]}


# ----------------------------------------------------- definition, 64 bits
def _exact_w(w, e, group):
    """Expert e's weights (or the one matrix, e None) in float64, element k of a row from byte k // 2."""
    if not group:
        return w[e].double()
    q, s, z = (None if v is None else v if e is None else v[e] for v in w)
    n, half = q.shape
    v = torch.empty(n, 2 * half, dtype=torch.float64, device=q.device)
    v[:, 0::2] = q.remainder(16).double()
    v[:, 1::2] = q.div(16, rounding_mode="floor").double()
    at = torch.arange(2 * half, device=q.device) // group
    v -= 8 if z is None else z.double()[:, at]
    return v.mul_(s.double()[:, at])


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm":
        h = c["xin"].double() + (c["r"].double() if c["res"] else 0)
        y = c["gamma"].double() * h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / c["n"] + EPS)
        out = {"sum": h} if c["res"] else {}
        if c["out"] == "bf16":
            return out | {"y": y}
        top, gs = (127 if c["out"] == "i8" else 448), c["group"] or c["n"]
        s = torch.stack([p.abs().max(1).values for p in y.split(gs, 1)], 1) / top
        v = y / torch.where(s > 0, s, 1).repeat_interleave(gs, 1)
        if c["out"] == "e4m3":
            return out | {"q": v.to(E4M3).double(), "scale": s}
        return out | {"y": v.round() * s.repeat_interleave(gs, 1), "scale": s}
    if c["op"] == "route":
        l = c["l"].double()
        at = torch.arange(c["experts"], device=l.device)
        beats = (l[:, None, :] > l[:, :, None]) | ((l[:, None, :] == l[:, :, None]) & (at[None, :] < at[:, None]))
        rank = beats.sum(2)  # how many experts come before this one
        idx = torch.argsort(rank, 1)[:, : c["k"]]
        p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        w = torch.take_along_dim(p, idx, 1)
        return idx.to(torch.int32), w / w.sum(1, keepdim=True) if c["renorm"] else w
    x = c["xq"].double()
    if c["xs"] is not None:
        x = x * c["xs"].double()[:, torch.arange(x.shape[1], device=x.device) * c["xs"].shape[1] // x.shape[1]]
    if c["op"] == "w4":
        return torch.mm(x, _exact_w((c["q"], c["s"], c["z"]), None, c["group"]).t())
    y = torch.zeros_like(x)
    for e in range(c["local"]):
        t, j = torch.nonzero(c["topk"] == e + c["base"], as_tuple=True)
        if not t.numel():
            continue
        gate, up = torch.mm(x[t], _exact_w(c["w1"], e, c["group"]).t()).chunk(2, 1)
        a = gate * torch.sigmoid(gate) * up
        y.index_add_(0, t, torch.mm(a, _exact_w(c["w2"], e, c["group"]).t()) * c["tw"][t, j].double()[:, None])
    return y
