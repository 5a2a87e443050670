"""Plain 64-bit forms of the decoding operators and the error bounds their tests
use. A rounding to nearest is off by at most eps / 2 of the value's type; `U` is
that of fp32. Sums in fp32 are taken as chains of independent roundings (six
times their root mean square), each of at most U times the largest partial sum."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
E4M3_HALF = 2.0 ** -4
TOP = {"i8": 127.0, "e4m3": 448.0}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, want, tol, what=""):
    """Every element within its tolerance; NaN and infinities in the same places."""
    got, want = got.double().cpu(), want.double()
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities"
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or over.max() <= 0, (
        f"{what}: {int((over > 0).sum())} of {over.numel()} off, worst {float(over.max()):.3g} over a tolerance of "
        f"{float(tol[fine][over.argmax()]):.3g}")


# -------------------------------------------------------------------- norm
def norm(x, gamma, residual, eps):
    h = x.double() + (residual.double() if residual is not None else 0.0)
    y = h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * gamma.double()
    return h, y


def groups_of(y, group):
    return y.unflatten(1, (-1, group or y.shape[1]))


# ------------------------------------------------------------------- route
def route(logits, k, score, renorm, scale):
    """Written out per row: sort by (value descending, index), NaN as -inf."""
    rows, experts = logits.shape
    l = torch.where(logits.isnan(), -math.inf, logits.double())
    topk = torch.empty(rows, k, dtype=torch.int32)
    w = torch.empty(rows, k, dtype=torch.float64)
    for r in range(rows):
        v = l[r].tolist()
        nan = logits[r].isnan().tolist()
        pick = sorted(range(experts), key=lambda e: (-v[e], nan[e], e))[:k]
        m = max(v)
        if score == "softmax":
            s = sum(math.exp(a - m) for a in v if a > -math.inf)
            p = [math.exp(v[e] - m) / s if v[e] > -math.inf else 0.0 for e in pick]
        else:
            p = [1 / (1 + math.exp(-v[e])) if v[e] > -700 else 0.0 for e in pick]
        total = sum(p)
        topk[r] = torch.tensor(pick, dtype=torch.int32)
        w[r] = torch.tensor([(a / total if total else 0.0) * scale if renorm else a * scale for a in p], dtype=torch.float64)
    return topk, w


# ---------------------------------------------------------------- products
def make_w4(g, lead, n, k, group, zero):
    q = torch.randint(0, 256, (*lead, n, k // 2), generator=g, dtype=torch.uint8)
    s = ((torch.rand(*lead, n, k // group, generator=g) + 0.5) * 0.2 / math.sqrt(k)).bfloat16()
    z = torch.randint(0, 16, (*lead, n, k // group), generator=g, dtype=torch.uint8) if zero else None
    return q, s, z


def w4_values(q, s, z):
    """float64 weights [.., n, k]."""
    k = 2 * q.shape[-1]
    v = torch.empty(*q.shape[:-1], k, dtype=torch.float64)
    v[..., 0::2] = (q % 16).double()
    v[..., 1::2] = (q // 16).double()
    rep = k // s.shape[-1]
    v -= 8.0 if z is None else z.double().repeat_interleave(rep, -1)
    return v * s.double().repeat_interleave(rep, -1)


def make_rows(g, rows, k, kind, x_group):
    """(tensor, scales, float64 values)"""
    x = torch.randn(rows, k, generator=g)
    if kind == "bf16":
        x = x.bfloat16()
        return x, None, x.double()
    v = groups_of(x, x_group)
    a = v.abs().amax(-1) if k else v.new_zeros(rows, 1)
    c = (v * (TOP[kind] / a.clamp_min(1e-30))[..., None]).flatten(1)
    q = c.round().to(torch.int8) if kind == "i8" else c.to(torch.float8_e4m3fn)
    s = a / TOP[kind]
    return q, s, (groups_of(q.double(), x_group) * s.double()[..., None]).flatten(1)


def w4_error(x, s, group):
    """Bound of the fp32 error of x [t, k] times 4-bit weights [n, k] with scales s:
    a group's sums of (128 + q) x and of x, at most 143 times a partial sum of x,
    about four root sums of squares besides its mean, are rounded once per element."""
    v = groups_of(x, group)
    part = 143.0 * (v.sum(-1).abs() + 4.0 * v.square().sum(-1).sqrt())           # [t, k / group]
    walk = 6.0 * U * math.sqrt(2.0 * group) * (part.square() @ s.double().square().t()).sqrt()
    return walk + 8.0 * U * (groups_of(x.abs(), group).sum(-1) * 15.0) @ s.double().t()


def dense_error(x, w):
    """The same for plain fp32 accumulation: one rounding per element of partial
    sums of at most four root sums of squares, and the rounding of a scale."""
    k = x.shape[1]
    part = 4.0 * (x.square() @ w.square().t()).sqrt() + (x @ w.t()).abs()
    return 6.0 * U * math.sqrt(k) * part + 8.0 * U * (x.abs() @ w.abs().t())


def moe(xv, w1, w2, topk, weights, base, w4=None):
    """(y, tolerance): w1 [E, 2F, K], w2 [E, K, F] in float64; w4: (scale1, scale2,
    group) of 4-bit weights. h is kept as two bf16 numbers (2^-16 of it)."""
    tokens, K = xv.shape
    F = w2.shape[2]
    y = torch.zeros(tokens, K, dtype=torch.float64)
    tol = torch.zeros(tokens, K, dtype=torch.float64)
    for t in range(tokens):
        for j in range(topk.shape[1]):
            e = int(topk[t, j]) - base
            if not 0 <= e < w1.shape[0]:
                continue
            x = xv[t:t + 1]
            gu = x @ w1[e].t()
            d = dense_error(x, w1[e]) if w4 is None else w4_error(x, w4[0][e], w4[2])
            g, u, dg, du = gu[:, :F], gu[:, F:], d[:, :F], d[:, F:]
            c = float(weights[t, j])
            silu = g * torch.sigmoid(g)
            h = c * silu * u
            # |silu'| <= 1.1; the exponential and the division: 8 roundings and 2 |g| of the exponent's
            dh = abs(c) * (1.1 * dg * (u.abs() + du) + silu.abs() * du) + (2.0 ** -16 + (8 + 2 * g.abs()) * U) * h.abs()
            y[t:t + 1] += h @ w2[e].t()
            tol[t:t + 1] += dh @ w2[e].abs().t() + (dense_error(h, w2[e]) if w4 is None else w4_error(h, w4[1][e], w4[2]))
    return y, tol + BF16_HALF * (y.abs() + tol) + 2.0 ** -133
