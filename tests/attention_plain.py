"""Plain 64-bit forms of the attention half's operators and the error bounds their
tests use. A rounding to nearest is off by at most half a step (`BF16_HALF`, `U` for
fp32). Weights of tokens are rounded to bf16 before they multiply the values, so
with p the exact weights (sum 1) and d a bound of the scores' error

    |out - exact| <= (BF16_HALF + (e^2d - 1) + SUM) sum_t p_t |v_t|, and BF16_HALF of the result on top:

a score off by d changes a weight and the sum of weights by a factor between e^-d
and e^d each, so p_t by one between e^-2d and e^2d. SUM: fp32 sums over a piece, the
pieces and the waves."""
from __future__ import annotations

import math

import torch

from ops_plain import BF16_HALF, E4M3_HALF, U, close, gen  # noqa: F401

SUM = 4096 * U


def page_step(lens, add, table, ring, ends, page, tokens):
    """Request by request; returns (lens, ends, starts, slots, positions) and changes table and ring (lists)."""
    head, tail = ends
    size = len(ring)
    free = min(max(tail - head, 0), size)
    width = len(table[0]) if table else 0
    asked = wanted = taken = given = back = 0
    out, starts, slots, positions = [], [0], [], []
    fresh = []
    for b, (n, a) in enumerate(zip(lens, add)):
        n = max(n, 0)
        has = -(-n // page)
        if a < 0:
            for i in range(min(has, width)):
                if back < size - free:
                    fresh.append(((tail + back) % size, table[b][i]))
                    back += 1
            out.append(0)
            starts.append(given)
            continue
        wants = -(-(n + a) // page)
        ok = wants <= width
        if ok:
            asked += wants - has
            ok = wants == has or asked <= free
        if ok:
            wanted += a
            ok = wanted <= tokens
        if ok:
            for i in range(has, wants):
                table[b][i] = ring[(head + taken) % size]
                taken += 1
            for p in range(n, n + a):
                positions.append(p)
                slots.append(table[b][p // page] * page + p % page if table[b][p // page] >= 0 else -1)
            given += a
            n += a
        out.append(n)
        starts.append(given)
    for i, v in fresh:
        ring[i] = v
    slots += [-1] * (tokens - given)
    positions += [0] * (tokens - given)
    return out, [head + taken, tail + back], starts, slots, positions


def rows8(x):
    """e4m3 codes and scales of bf16 rows, as kv_append makes them of ordinary numbers."""
    a = x.float().abs().amax(-1, keepdim=True)
    q = (x.float() * torch.where(a > 0, 448.0 / a, 0.0)).to(torch.float8_e4m3fn)
    return q, (a / 448.0).squeeze(-1)


def place(g, lens, page, width, spare=2):
    """Pages of every request in no order: table int32 [batch, width] (-1 behind the last), number of pages."""
    held = [-(-n // page) for n in lens]
    n = sum(held) + spare
    ids = torch.randperm(n, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, n


def tokens_of(cache, table, b, n, page):
    """Rows of request b's tokens 0..n-1; None for those on pages that the cache lacks."""
    t = torch.arange(n)
    ids = table[b].long()[t // page]
    there = (ids >= 0) & (ids < cache.shape[0])
    return cache[ids.clamp(0, cache.shape[0] - 1), t % page], there


def attend(scores, score_tol, values, scale):
    """(out, tolerance, lse, its tolerance) of one query: scores [n] unscaled, values [n, d] in float64."""
    if scores.numel() == 0:
        z = torch.zeros(values.shape[1], dtype=torch.float64)
        return z, z, -math.inf, 0.0
    s = scores * scale
    d = float((score_tol * scale).max()) + 8 * U + 4 * U * float(s.abs().max()) if torch.isfinite(s).all() else 0.0
    p = torch.softmax(s, 0)
    out = p @ values
    size = p @ values.abs()
    tol = (BF16_HALF + math.expm1(2 * d) * (1 + BF16_HALF) + SUM) * size
    return out, tol + BF16_HALF * (out.abs() + tol) + 2.0 ** -133, float(torch.logsumexp(s, 0)), d + SUM + 4 * U * float(s.abs().max())


def paged(q, k, v, table, lens, scale, window=0):
    """q [batch, heads, dim]; caches in float64 [n_pages, page, kv, dim] (scales applied)."""
    batch, heads, dim = q.shape
    page, kv = k.shape[1], k.shape[2]
    out = torch.zeros(batch, heads, dim, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((batch, heads), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros_like(lse)
    for b in range(batch):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        kt, there = tokens_of(k, table, b, n, page)
        vt, _ = tokens_of(v, table, b, n, page)
        if window:
            there = there & (torch.arange(n) >= n - window)
        for h in range(heads):
            kk, x = kt[there][:, h * kv // heads], q[b, h].double()
            out[b, h], tol[b, h], lse[b, h], lse_tol[b, h] = attend(kk @ x, (dim + 8) * U * (kk.abs() @ x.abs()), vt[there][:, h * kv // heads], scale)
    return out, tol, lse, lse_tol


def rounded(x, err):
    """x rounded to bf16, and how far a rounding of x +- err may be from that: a step where the two may differ."""
    r = x.float().bfloat16().double()
    step = 2 * BF16_HALF * x.abs()
    differ = ((x - err).float().bfloat16() != (x + err).float().bfloat16())
    return r, torch.where(differ, step + err, torch.zeros_like(step))


def latent(q, w, cache, table, lens, nope, scale):
    """Absorbed form: the keys' weights on the query's side are rounded to bf16, or up to 16 heads
    held as two bf16 numbers (the second, at most 2^-8 of the first, is off by 2^-8 of itself), as the operator says."""
    batch, heads, _ = q.shape
    rank, page = w.shape[2], cache.shape[1]
    out = torch.zeros(batch, heads, nope, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((batch, heads), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros_like(lse)
    w = w.double()
    for b in range(batch):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        rows, there = tokens_of(cache.double(), table, b, n, page)
        rows = rows[there]
        c, r = rows[:, :rank], rows[:, rank:]
        for h in range(heads):
            x, rot, up, down = q[b, h, :nope].double(), q[b, h, nope:].double(), w[h, :nope], w[h, nope:]
            a, a_err = x @ up, (nope + 8) * U * (x.abs() @ up.abs())
            a, a_tol = (a, 2.0 ** -16 * a.abs() + a_err) if heads <= 16 else rounded(a, a_err)
            s_tol = c.abs() @ a_tol + (rows.shape[1] + 8) * U * (c.abs() @ a.abs() + r.abs() @ rot.abs())
            mean, mean_tol, lse[b, h], lse_tol[b, h] = attend(c @ a + r @ rot, s_tol, c, scale)
            # the mean is not rounded to one bf16: take that part out of the bound again
            mean_tol = (mean_tol - BF16_HALF * mean.abs()).clamp_min(0) + 2.0 ** -15 * mean.abs()
            out[b, h] = down @ mean
            t = down.abs() @ mean_tol + (2 * rank + 8) * U * (down.abs() @ mean.abs())
            tol[b, h] = t + BF16_HALF * (out[b, h].abs() + t) + 2.0 ** -133
    return out, tol, lse, lse_tol


def prompt(q, lat, w, q_starts, k_starts, nope, scale):
    """Expanded form: keys and values are rounded to bf16, as the operator says."""
    rows, heads, _ = q.shape
    rank = w.shape[2]
    out = torch.zeros(rows, heads, nope, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros_like(lse)
    for b in range(len(q_starts) - 1):
        q0, q1, k0, k1 = q_starts[b], q_starts[b + 1], k_starts[b], k_starts[b + 1]
        c, r = lat[k0:k1, :rank].double(), lat[k0:k1, rank:].double()
        for h in range(heads):
            m = w[h].double()
            kv, kv_tol = rounded(c @ m.t(), (rank + 8) * U * (c.abs() @ m.abs().t()))
            k, kt, v, vt = kv[:, :nope], kv_tol[:, :nope], kv[:, nope:], kv_tol[:, nope:]
            for i in range(q0, q1):
                seen = max(0, (k1 - k0) - (q1 - q0) + (i - q0) + 1)
                x, rot = q[i, h, :nope].double(), q[i, h, nope:].double()
                s = k[:seen] @ x + r[:seen] @ rot
                s_tol = kt[:seen] @ x.abs() + (nope + rot.numel() + 8) * U * (k[:seen].abs() @ x.abs() + r[:seen].abs() @ rot.abs())
                out[i, h], t, lse[i, h], lse_tol[i, h] = attend(s, s_tol, v[:seen], scale)
                if seen:
                    t = t + (torch.softmax(s * scale, 0) @ vt[:seen]) * (1 + 2 * BF16_HALF)
                tol[i, h] = t
    return out, tol, lse, lse_tol
