"""The operators of a decoder layer's attention half over a paged cache: page tables and slots of a step, rows written
into the cache, attention of one new token over pages, and attention whose keys and values come from one latent vector a
token, in the absorbed form (one new token over pages) and in the expanded form (prompts).

Every case is served in two forms: the plain one (elementary torch operations in float32) and the library's own kernels.
Sizes follow the workloads of this package where it has them (8 shards of 1024 tokens, 4096 columns of attention output
as 32 heads of 128, up to 64 tokens a step); the others are generic."""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # the pages of one decoding step: 64 requests, one token each
        dict(name="pages_64_step", op="pages", batch=64, longest=8192, page=16, adds=1, mixed=False, short=False),
        # a busy scheduler: 1000 requests, some decode, some bring prompts, some have ended, some are idle, and pages run out
        dict(name="pages_1000_mixed", op="pages", batch=1000, longest=4096, page=64, adds=1024, mixed=True, short=True),
        # keys and values of one decoding step as 8-bit rows
        dict(name="append_64x8x128_e4m3", op="append", rows=64, pad=3, heads=8, dim=128, both=True, e4m3=True, page=16),
        # latent rows of a prompt: 8 shards of 1024 tokens
        dict(name="append_8192_latent", op="append", rows=8192, pad=0, heads=1, dim=576, both=False, e4m3=False, page=64),
        # four short requests of a small model, one of them a padded row
        dict(name="paged_4x300_12of4x64", op="paged", batch=4, longest=300, ragged=True, heads=12, kv=4, dim=64, page=16, window=0, e4m3=False),
        # one long document: the work has to be split over the cache's length
        dict(name="paged_1x131072_64of8x128", op="paged", batch=1, longest=131072, ragged=False, heads=64, kv=8, dim=128, page=64, window=0, e4m3=False),
        # a full decoding batch of uneven lengths, 8-bit cache
        dict(name="paged_64x16384_32of8x128_e4m3", op="paged", batch=64, longest=16384, ragged=True, heads=32, kv=8, dim=128, page=16, window=0, e4m3=True),
        # absorbed form, two requests of a small model
        dict(name="latent_2x1001_h12", op="latent", batch=2, longest=1001, ragged=False, heads=12, rank=256, rope=32, nope=64, page=16),
        # absorbed form, one long document, the heads of one GPU out of eight
        dict(name="latent_1x131072_h16", op="latent", batch=1, longest=131072, ragged=False, heads=16, rank=512, rope=64, nope=128, page=64),
        # absorbed form, a full decoding batch of uneven lengths with all heads on this GPU
        dict(name="latent_64x8192_h128", op="latent", batch=64, longest=8192, ragged=True, heads=128, rank=512, rope=64, nope=128, page=64),
        # expanded form, 512 new tokens each after earlier ones, 8 requests
        dict(name="prompt_8x1100_h16_chunk", op="prompt", batch=8, longest=1100, ragged=True, heads=16, rank=512, rope=64, nope=128, chunk=512),
        # expanded form, one long prompt
        dict(name="prompt_1x16384_h16", op="prompt", batch=1, longest=16384, ragged=False, heads=16, rank=512, rope=64, nope=128, chunk=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _latent_sizes(rng):
    return dict(rank=rng.choice([256, 512]), rope=rng.choice([32, 64]), nope=rng.choice([64, 128]))


def draw(rng):
    op = rng.choice(["pages", "append", "paged", "latent", "prompt"])
    if op == "pages":
        mixed = rng.random() < 0.5
        return dict(op=op, batch=_log(rng, 1, 1000), longest=_log(rng, 16, 4096), page=16 * rng.choice([1, 2, 3, 4, 8]),
                    adds=_log(rng, 1, 1000) if mixed else rng.randint(1, 4), mixed=mixed, short=rng.random() < 0.3)
    if op == "append":
        both = rng.random() < 0.6
        rows = _log(rng, 1, 8000 if not both else 2000)
        return dict(op=op, rows=rows, pad=rng.randint(0, max(0, min(5, rows - 1))), heads=rng.choice([1, 2, 4, 8]) if both else 1,
                    dim=rng.choice([64, 128, 256]) if both else rng.choice([288, 320, 544, 576]), both=both, e4m3=both and rng.random() < 0.5,
                    page=16 * rng.choice([1, 2, 4]))
    if op == "paged":
        kv, dim, longest = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), _log(rng, 1, 40000)
        most = max(1, min(64, (100 << 20) // (longest * kv * dim)))
        return dict(op=op, batch=_log(rng, 1, most), longest=longest, ragged=rng.random() < 0.7, heads=kv * rng.choice([1, 2, 3, 4, 7, 8, 16]), kv=kv, dim=dim,
                    page=16 * rng.choice([1, 2, 3, 4, 8]), window=rng.choice([0, 0, _log(rng, 1, 4096)]), e4m3=rng.random() < 0.5)
    if op == "latent":
        longest = _log(rng, 1, 60000)
        return dict(op=op, batch=_log(rng, 1, max(1, min(64, 160000 // longest))), longest=longest, ragged=rng.random() < 0.7,
                    heads=rng.choice([1, 8, 12, 16, 20, 32, 64, 128]), page=16 * rng.choice([1, 2, 3, 4, 8]), **_latent_sizes(rng))
    longest = _log(rng, 1, 6000)
    return dict(op=op, batch=_log(rng, 1, max(1, min(16, 24000 // longest))), longest=longest, ragged=rng.random() < 0.7, heads=rng.choice([1, 4, 8, 12, 16]),
                chunk=rng.choice([0, 0, _log(rng, 1, 1024)]), **_latent_sizes(rng))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(c):
    """Tokens of each request, the first the longest; of four and more uneven ones the last is a padded row with none."""
    if not c["ragged"]:
        return [c["longest"]] * c["batch"]
    n = [max(1, round(c["longest"] * (1 - (i * 0.6180339887 % 1.0)) ** 2)) for i in range(c["batch"])]
    if len(n) >= 4:
        n[-1] = 0
    return n


def _queries(c):
    return [min(n, c["chunk"]) if c["chunk"] else n for n in _lengths(c)]


def _shuffled(g, values):
    order = torch.randperm(len(values), generator=g, device=DEV).tolist()
    return [values[i] for i in order]


def _place(g, lens, page, spare, width):
    """Pages of every request, drawn without order: table int32 [batch, width] (-1 where a request has none), free pages."""
    held = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(held) + spare, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids[at:]


def _rows8(x):
    """Rows as 8-bit floats with one float32 scale each."""
    a = x.float().abs().amax(-1, keepdim=True)
    return (x.float() * torch.where(a > 0, 448.0 / a, 0.0)).to(E4M3), (a / 448.0).squeeze(-1)


def _cache8(x):
    """A cache as 8-bit rows; scales [pages, heads, page]."""
    q, s = _rows8(x)
    return q, s.transpose(1, 2).contiguous()


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=BF16).mul_(scale)


def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "pages":
        n, page = c["batch"], c["page"]
        lens = torch.randint(0, c["longest"] + 1, (n,), generator=g, device=DEV).tolist()
        add = [c["adds"]] * n
        if c["mixed"]:
            kind = torch.randint(0, 10, (n,), generator=g, device=DEV).tolist()  # 0-4 decode, 5-7 prompt, 8 ended, 9 idle
            size = torch.randint(1, c["adds"] + 1, (n,), generator=g, device=DEV).tolist()
            add = [1 if k < 5 else s if k < 8 else -1 if k == 8 else 0 for k, s in zip(kind, size)]
        need = sum(-(-(l + max(a, 0)) // page) - (-(-l // page)) for l, a in zip(lens, add))
        c["width"] = -(-(c["longest"] + c["adds"]) // page)
        c["table"], free = _place(g, lens, page, need * 3 // 4 if c["short"] else need + 5, c["width"])
        total = n * c["width"] + 5  # the cache's pages, those of other programs' requests among them
        head = 1000003 * (seed % 1000)  # pages have gone round the ring many times
        c["ring"] = torch.full((total,), -1, dtype=torch.int32, device=DEV)
        c["ring"][(head + torch.arange(free.numel(), device=DEV)) % c["ring"].numel()] = free
        c["ends"] = torch.tensor([head, head + free.numel()], dtype=torch.int64, device=DEV)
        c["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        c["add"] = torch.tensor(add, dtype=torch.int32, device=DEV)
        c["tokens"] = n * c["adds"]
    elif c["op"] == "append":
        r, h, d, page = c["rows"], c["heads"], c["dim"], c["page"]
        pages = -(-2 * r // page)
        shape = (pages, page, h, d)
        c["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:r]
        c["slots"][r - c["pad"]:] = -1
        for name in ("k", "v") if c["both"] else ("k",):
            # rows as a projection leaves them: slices of a wider row
            c[name] = _normal(g, r, h * d + 64)[:, :h * d].unflatten(1, (h, d))
            old = _normal(g, *shape)
            c[name + "c"], c[name + "s"] = _cache8(old) if c["e4m3"] else (old, None)
    elif c["op"] == "paged":
        n, page, kv, d = c["batch"], c["page"], c["kv"], c["dim"]
        c["host"] = _shuffled(g, _lengths(c))
        c["table"], free = _place(g, c["host"], page, 3, max(1, -(-c["longest"] // page)))
        pages = sum(-(-l // page) for l in c["host"]) + 3
        for name in ("k", "v"):
            x = _normal(g, pages, page, kv, d)
            if name == "v":
                x += _normal(g, kv, d)  # values of a head have a mean of their own
            c[name + "c"], c[name + "s"] = _cache8(x) if c["e4m3"] else (x, None)
        c["q"] = _normal(g, n, c["heads"], d, scale=1.5)
        c["lens"] = torch.tensor(c["host"], dtype=torch.int32, device=DEV)
    else:
        h, r, p, m = c["heads"], c["rank"], c["rope"], c["nope"]
        c["w"] = _normal(g, h, 2 * m, r, scale=1 / math.sqrt(r))
        if c["op"] == "latent":
            page = c["page"]
            c["host"] = _shuffled(g, _lengths(c))
            c["table"], free = _place(g, c["host"], page, 3, max(1, -(-c["longest"] // page)))
            c["cache"] = _normal(g, sum(-(-l // page) for l in c["host"]) + 3, page, r + p)
            c["q"] = _normal(g, c["batch"], h, m + p, scale=1.5)
            c["lens"] = torch.tensor(c["host"], dtype=torch.int32, device=DEV)
        else:
            both = _shuffled(g, list(zip(_queries(c), _lengths(c))))
            c["hq"], c["hk"] = [q for q, _ in both], [k for _, k in both]
            c["q_starts"], c["k_starts"] = _starts(c["hq"]), _starts(c["hk"])
            c["lat"] = _normal(g, sum(c["hk"]), r + p)
            c["q"] = _normal(g, sum(c["hq"]), h, m + p, scale=1.5)
    return c


# -------------------------------------------------------------- plain form
def _plain_pages(c):
    page, n, lens, add, table, ring = c["page"], c["batch"], c["lens"].long(), c["add"].long(), c["table"], c["ring"]
    width, size, (head, tail) = table.shape[1], ring.numel(), c["ends"]
    held = (lens + page - 1) // page
    want = add.clamp_min(0)
    more = (lens + want + page - 1) // page
    fits = more <= width
    need = torch.where(fits, more - held, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= tail - head))
    got = torch.where(served, want, 0)
    served &= got.cumsum(0) <= c["tokens"]
    got = torch.where(served, want, 0)
    need_ok = torch.where(served, need, 0)
    starts = torch.cat((got.new_zeros(1), got.cumsum(0)))
    # pages of the ring into the table
    col = torch.arange(width, device=DEV)
    fresh = (col >= held[:, None]) & (col < (held + need_ok)[:, None])
    from_ring = ring[(head + (upto - need)[:, None] + col - held[:, None]) % size]
    table.copy_(torch.where(fresh, from_ring, table))
    # pages of ended requests back to the ring
    ended = add < 0
    back = torch.where(ended, held.clamp_max(width), 0)
    place = (tail + (back.cumsum(0) - back)[:, None] + col) % size
    spill = torch.cat((ring, ring.new_zeros(1)))
    spill[torch.where(col < back[:, None], place, size)] = table
    ring.copy_(spill[:size])
    t = torch.arange(c["tokens"], device=DEV)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp_max(n - 1)
    real = t < starts[-1]
    pos = torch.where(real, lens[b] + t - starts[b], 0)
    slot = torch.where(real, table[b, pos // page].long() * page + pos % page, -1)
    return {"lens": torch.where(ended, 0, lens + got).to(torch.int32), "ends": torch.stack((head + need_ok.sum(), tail + back.sum())),
            "starts": starts.to(torch.int32), "slots": slot, "positions": pos.to(torch.int32), "table": table, "ring": ring}


def _plain_append(c):
    out, n = {}, c["rows"] - c["pad"]
    page, place = c["slots"][:n] // c["page"], c["slots"][:n] % c["page"]
    for name in ("k", "v") if c["both"] else ("k",):
        x, cache, s = c[name].float(), c[name + "c"], c[name + "s"]
        if c["e4m3"]:
            x, scale = _rows8(x)
            s[page, :, place] = scale[:n]
            out[name + "s"] = s
            cache.view(torch.uint8).flatten(0, 1)[c["slots"][:n]] = x.view(torch.uint8)[:n]
        else:
            cache.flatten(0, 1)[c["slots"][:n]] = x.to(BF16)[:n]
        out[name] = cache
    return out


def _pages_of(c, b):
    return c["table"][b, :-(-c["host"][b] // c["page"])]


def _softmax(s):
    e = torch.exp(s - s.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_paged(c):
    kv, d, out = c["kv"], c["dim"], torch.zeros(c["batch"], c["heads"], c["dim"], device=DEV)
    for b, n in enumerate(c["host"]):
        if n == 0:
            continue
        first = max(0, n - c["window"]) if c["window"] else 0
        k, v = (t[_pages_of(c, b)].flatten(0, 1)[first:n].float() if s is None else
                (t[_pages_of(c, b)].float() * s[_pages_of(c, b)].transpose(1, 2).unsqueeze(-1)).flatten(0, 1)[first:n] for t, s in ((c["kc"], c["ks"]), (c["vc"], c["vs"])))
        q = c["q"][b].float().unflatten(0, (kv, -1))
        p = _softmax(torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(d))
        out[b] = torch.matmul(p, v.transpose(0, 1)).flatten(0, 1)
    return out.to(BF16)


def _latent_scale(c):
    return 1 / math.sqrt(c["nope"] + c["rope"])


def _plain_latent(c):
    m, r = c["nope"], c["rank"]
    w, q = c["w"].float(), c["q"].float()
    inner = torch.matmul(q[..., :m].transpose(0, 1), w[:, :m]).transpose(0, 1)  # keys' weights on the query's side
    mean = torch.zeros(c["batch"], c["heads"], r, device=DEV)
    for b, n in enumerate(c["host"]):
        if n == 0:
            continue
        rows = c["cache"][_pages_of(c, b)].flatten(0, 1)[:n].float()
        s = inner[b] @ rows[:, :r].t() + q[b, :, m:] @ rows[:, r:].t()
        mean[b] = _softmax(s * _latent_scale(c)) @ rows[:, :r]
    return torch.matmul(mean.transpose(0, 1), w[:, m:].transpose(1, 2)).transpose(0, 1).to(BF16)


def _plain_prompt(c):
    m, r, h = c["nope"], c["rank"], c["heads"]
    out = torch.empty(c["q"].shape[0], h, m, device=DEV)
    q0 = k0 = 0
    for nq, nk in zip(c["hq"], c["hk"]):
        if nq == 0:
            continue
        rows, q = c["lat"][k0:k0 + nk].float(), c["q"][q0:q0 + nq].float()
        hidden = torch.arange(nk, device=DEV) > torch.arange(nk - nq, nk, device=DEV)[:, None]
        step = max(1, min(h, (1 << 28) // max(1, nq * nk)))
        for i in range(0, h, step):
            kv = torch.matmul(rows[:, :r], c["w"][i:i + step].float().transpose(1, 2))  # [heads, keys, 2 m]
            s = torch.matmul(q[:, i:i + step, :m].transpose(0, 1), kv[..., :m].transpose(1, 2))
            s += torch.matmul(q[:, i:i + step, m:].transpose(0, 1), rows[:, r:].t())
            p = _softmax((s * _latent_scale(c)).masked_fill(hidden, -math.inf))
            out[q0:q0 + nq, i:i + step] = torch.matmul(p, kv[..., m:]).transpose(0, 1)
        q0, k0 = q0 + nq, k0 + nk
    return out.to(BF16)


def _own(c):
    from sync_protocols_amd import ops

    if c["op"] == "pages":
        r = ops.page_step(c["lens"], c["add"], c["table"], c["ring"], c["ends"], page=c["page"], tokens=c["tokens"])
        return {"lens": r.lens, "ends": r.ends, "starts": r.starts, "slots": r.slots, "positions": r.positions, "table": c["table"], "ring": c["ring"]}
    if c["op"] == "append":
        if not c["both"]:
            ops.kv_append(c["k"], c["kc"], c["slots"])
            return {"k": c["kc"]}
        ops.kv_append(c["k"], c["kc"], c["slots"], v=c["v"], v_cache=c["vc"], k_scale=c["ks"], v_scale=c["vs"])
        return {"k": c["kc"], "v": c["vc"]} | ({"ks": c["ks"], "vs": c["vs"]} if c["e4m3"] else {})
    if c["op"] == "paged":
        return ops.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], window=c["window"], k_scale=c["ks"], v_scale=c["vs"])
    if c["op"] == "latent":
        return ops.latent_attention(c["q"], c["w"], c["cache"], c["table"], c["lens"], nope=c["nope"])
    return ops.latent_prompt(c["q"], c["lat"], c["w"], c["q_starts"], k_starts=c["k_starts"], nope=c["nope"])


def run(state):
    if own:
        return _own(state)
    return {"pages": _plain_pages, "append": _plain_append, "paged": _plain_paged, "latent": _plain_latent, "prompt": _plain_prompt}[state["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "pages":
        tokens = c["batch"] * c["adds"]
        return {"bytes": 12 * c["batch"] + 12 * tokens + 8 * c["batch"] * (1 + c["adds"] // c["page"]), "flops": 4 * tokens}
    if c["op"] == "append":
        e = c["rows"] * c["heads"] * c["dim"] * (1 + c["both"])
        return {"bytes": 8 * c["rows"] + e * (3 if c["e4m3"] else 4) + (8 * c["rows"] * c["heads"] if c["e4m3"] else 0), "flops": 3 * e if c["e4m3"] else e}
    if c["op"] == "paged":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
        row = c["kv"] * (c["dim"] * (1 if c["e4m3"] else 2) + 4 * c["e4m3"])
        return {"bytes": 2 * seen * row + 4 * seen // c["page"] + 4 * c["batch"] * c["heads"] * c["dim"], "flops": 4 * seen * c["heads"] * c["dim"]}
    h, r, p, m = c["heads"], c["rank"], c["rope"], c["nope"]
    if c["op"] == "latent":
        seen, n = sum(_lengths(c)), c["batch"]
        return {"bytes": 2 * seen * (r + p) + 4 * seen // c["page"] + 4 * h * m * r + 2 * n * h * (2 * m + p),
                "flops": 2 * h * (seen * (2 * r + p) + 2 * n * m * r)}
    pairs = sum(q * k - q * (q - 1) // 2 for q, k in zip(_queries(c), _lengths(c)))
    tq, tk = sum(_queries(c)), sum(_lengths(c))
    return {"bytes": 2 * tk * (r + p) + 4 * h * m * r + 2 * tq * h * (2 * m + p), "flops": 2 * h * (pairs * (2 * m + p) + 2 * tk * m * r)}


# ----------------------------------------------------- definition, 64 bits
def _exact_pages(c):
    """The step request by request, on the host."""
    page, lens, add = c["page"], c["lens"].tolist(), c["add"].tolist()
    table, ring, (head, tail) = c["table"].tolist(), c["ring"].tolist(), c["ends"].tolist()
    asked, taken, given, wanted, left = 0, 0, 0, 0, 0
    out, starts, slots, positions = [], [0], [], []
    for b, (n, a) in enumerate(zip(lens, add)):
        if a < 0:
            for i in range(min(-(-n // page), c["width"])):
                ring[(tail + left) % len(ring)] = table[b][i]
                left += 1
            out.append(0)
        else:
            has, wants = -(-n // page), -(-(n + a) // page)
            ok = wants <= c["width"]
            if ok:
                asked += wants - has
                ok = wants == has or asked <= tail - head
                wanted += a if ok else 0
                ok = ok and wanted <= c["tokens"]
            if ok:
                for i in range(has, wants):
                    table[b][i] = ring[(head + taken) % len(ring)]
                    taken += 1
                positions += range(n, n + a)
                slots += [table[b][i // page] * page + i % page for i in range(n, n + a)]
                given += a
                n += a
            out.append(n)
        starts.append(given)
    slots += [-1] * (c["tokens"] - given)
    positions += [0] * (c["tokens"] - given)

    def whole(v, t):
        return torch.tensor(v, dtype=t, device=DEV)

    i32, i64 = torch.int32, torch.int64
    return {"lens": whole(out, i32), "ends": whole([head + taken, tail + left], i64), "starts": whole(starts, i32), "slots": whole(slots, i64),
            "positions": whole(positions, i32), "table": whole(table, i32), "ring": whole(ring, i32)}


def _weights64(scores):
    return torch.softmax(scores, -1)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "pages":
        return _exact_pages(c)
    if c["op"] == "append":
        out, n = {}, c["rows"] - c["pad"]
        for name in ("k", "v") if c["both"] else ("k",):
            x = c[name][:n].double()
            flat = c[name + "c"].double().flatten(0, 1)
            if c["e4m3"]:
                s = x.abs().max(-1).values / 448
                out[name + "s"] = c[name + "s"].double()
                for i, t in enumerate(c["slots"][:n].tolist()):
                    out[name + "s"][t // c["page"], :, t % c["page"]] = s[i]
                x = (x / torch.where(s > 0, s, 1)[..., None]).to(E4M3).double()
            out[name] = flat.index_copy(0, c["slots"][:n], x).reshape(c[name + "c"].shape)
        return out
    if c["op"] == "paged":
        out = torch.zeros(c["batch"], c["heads"], c["dim"], dtype=torch.float64, device=DEV)
        for b, n in enumerate(c["host"]):
            at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device=DEV)
            if not n:
                continue
            page, place = c["table"][b].long()[at // c["page"]], at % c["page"]
            for j in range(c["kv"]):
                k, v = (c[x + "c"][page, place, j].double() * (1 if c[x + "s"] is None else c[x + "s"][page, j, place].double()[:, None]) for x in "kv")
                for i in range(j * c["heads"] // c["kv"], (j + 1) * c["heads"] // c["kv"]):
                    out[b, i] = torch.mv(v.t(), _weights64(torch.mv(k, c["q"][b, i].double()) * c["dim"] ** -0.5))
        return out
    m, r, h = c["nope"], c["rank"], c["heads"]
    scale = (m + c["rope"]) ** -0.5
    if c["op"] == "latent":
        out = torch.zeros(c["batch"], h, m, dtype=torch.float64, device=DEV)
        up, down = c["w"][:, :m].double(), c["w"][:, m:].double()
        for b, n in enumerate(c["host"]):
            if not n:
                continue
            at = torch.arange(n, device=DEV)
            rows = c["cache"][c["table"][b].long()[at // c["page"]], at % c["page"]].double()
            q = c["q"][b].double()
            full = torch.cat((torch.stack([q[i, :m] @ up[i] for i in range(h)]), q[:, m:]), 1)
            got = torch.mm(_weights64(torch.mm(full, rows.t()) * scale), rows[:, :r])
            out[b] = torch.stack([down[i] @ got[i] for i in range(h)])
        return out
    out = torch.zeros(c["q"].shape[0], h, m, dtype=torch.float64, device=DEV)
    for i in range(h):
        kv = torch.mm(c["lat"][:, :r].double(), c["w"][i].double().t())
        keys = torch.cat((kv[:, :m], c["lat"][:, r:].double()), 1)
        q0 = k0 = 0
        for nq, nk in zip(c["hq"], c["hk"]):
            s = torch.mm(c["q"][q0:q0 + nq, i].double(), keys[k0:k0 + nk].t()) * scale
            seen = torch.ones(nq, nk, dtype=torch.bool, device=DEV).tril(nk - nq)
            out[q0:q0 + nq, i] = torch.mm(_weights64(torch.where(seen, s, -math.inf)), kv[k0:k0 + nk, m:])
            q0, k0 = q0 + nq, k0 + nk
    return out
