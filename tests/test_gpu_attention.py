"""The attention half's operators on the GPU against their plain 64-bit forms."""
import math
import random

import pytest
import torch

import attention_plain as A
from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
E4M3 = torch.float8_e4m3fn


def dev(*ts):
    r = [None if t is None else t.to(DEV) for t in ts]
    return r if len(r) > 1 else r[0]


# --------------------------------------------------------------- page_step
def check_step(lens, add, table, ring, ends, page, tokens, in_place=False, pad=0):
    i32, i64 = torch.int32, torch.int64
    width = table.shape[1]
    big = torch.full((len(lens), width + pad), -7, dtype=i32, device=DEV)
    t = big[:, :width]
    t.copy_(table)
    r, e, l = ring.clone().to(DEV), torch.tensor(ends, dtype=i64, device=DEV), torch.tensor(lens, dtype=i32, device=DEV)
    got = ops.page_step(l, torch.tensor(add, dtype=i32, device=DEV), t, r, e, page=page, tokens=tokens,
                        lens_out=l if in_place else None, ends_out=e if in_place else None)
    assert (got.lens is l) == in_place
    tw, rw = table.tolist(), ring.tolist()
    want = A.page_step(lens, add, tw, rw, ends, page, tokens)
    for name, g, w in zip(got._fields, got, want):
        assert g.tolist() == w, name
    assert t.tolist() == tw and r.tolist() == rw
    assert (big[:, width:] == -7).all()
    return got, tw, rw


def random_step(rng, batch, page, longest, adds, free, width=None, mixed=True):
    lens = [rng.randint(0, longest) for _ in range(batch)]
    add = [rng.choice([1, 1, 0, -1, rng.randint(1, adds)]) if mixed else adds for _ in range(batch)]
    width = width or -(-(longest + adds) // page)
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + free + 3
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table = torch.full((batch, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        m = min(n, width)
        table[b, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
        at += n
    head = rng.choice([0, 5, n_pages - 1, 10 ** 12 + 7])
    ring = torch.full((n_pages,), -1, dtype=torch.int32)
    for i in range(free):
        ring[(head + i) % n_pages] = ids[at + i]
    return lens, add, table, ring, [head, head + free]


@pytest.mark.parametrize("batch", [1, 2, 63, 64, 65, 255, 256, 257, 512, 513, 1100])
@pytest.mark.parametrize("page,adds,free", [(16, 1, 10000), (16, 40, 37), (48, 3, 0), (1, 7, 11), (128, 1000, 500)])
def test_page_step(batch, page, adds, free):
    rng = random.Random(batch * 31 + page)
    lens, add, table, ring, ends = random_step(rng, batch, page, 300, adds, free)
    tokens = sum(max(a, 0) for a in add) + 5
    check_step(lens, add, table, ring, ends, page, tokens, in_place=batch % 2 == 0, pad=batch % 3)


@pytest.mark.parametrize("batch", [3, 300, 700])
def test_page_step_tables_and_tokens_that_run_out(batch):
    rng = random.Random(batch)
    lens, add, table, ring, ends = random_step(rng, batch, 16, 200, 60, 40 * batch, width=11)
    for tokens in (0, 1, sum(max(a, 0) for a in add) // 2, 70 * batch):
        check_step(lens, add, table, ring, ends, 16, tokens)


def test_page_step_of_one_long_prompt_and_of_none():
    rng = random.Random(1)
    lens, add, table, ring, ends = random_step(rng, 3, 16, 100, 50000, 7000, mixed=False)
    check_step(lens, [0, 50000, 1], table, ring, ends, 16, 50011)
    check_step(lens, [0, 0, 0], table, ring, ends, 16, 0)
    check_step([-5, 0, 100], [3, 0, -1], table, ring, ends, 16, 8)
    got = ops.page_step(*dev(torch.empty(0, dtype=torch.int32), torch.empty(0, dtype=torch.int32), torch.empty(0, 4, dtype=torch.int32), ring,
                             torch.tensor(ends)), page=16, tokens=9)
    assert got.slots.tolist() == [-1] * 9 and got.starts.tolist() == [0] and got.ends.tolist() == ends


def test_page_step_of_sums_beyond_32_bits():
    """Asked tokens and pages that add up beyond any 32-bit number; only what comes before them is served."""
    page, width, n = 1 << 20, 2000, 300
    table = torch.arange(n * width, dtype=torch.int32).reshape(n, width)
    ring = torch.arange(5000, dtype=torch.int32)
    check_step([7] * n, [1, 3] + [1 << 30] * (n - 3) + [2], table, ring, [2, 5002], page, 10)
    check_step([7] * n, [1, 3] + [2 ** 31 - 1] * (n - 2), table, ring, [2, 5002], page, 10)
    check_step([2 ** 31 - 1] * n, [2 ** 31 - 1, -1, 1] * (n // 3), table, ring, [2, 2002], 1 << 20, 10)


def test_pages_go_round():
    """Many steps of requests that come and go, state on the GPU alone: no page has two owners, none is lost."""
    rng = random.Random(4)
    batch, page, width, n_pages = 20, 16, 6, 70
    lens, ends = torch.zeros(batch, dtype=torch.int32, device=DEV), torch.tensor([0, n_pages], device=DEV)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(n_pages, device=DEV).to(torch.int32)
    served = 0
    for _ in range(60):
        add = torch.tensor([rng.choice([0, 1, 1, 2, 17, 30, -1]) for _ in range(batch)], dtype=torch.int32, device=DEV)
        got = ops.page_step(lens, add, table, ring, ends, page=page, tokens=700, lens_out=lens, ends_out=ends)
        served += int(got.starts[-1])
        owned = [p for b, n in enumerate(lens.tolist()) for p in table[b, :-(-n // page)].tolist()]
        head, tail = ends.tolist()
        free = [int(ring[i % n_pages]) for i in range(head, tail)]
        assert sorted(owned + free) == list(range(n_pages))
        live = [s for s in got.slots.tolist() if s >= 0]
        assert len(set(live)) == len(live) == int(got.starts[-1]) and all(s // page in owned for s in live)
    assert served > 1000


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("rows,heads,dim,page", [(1, 1, 8, 16), (5, 3, 64, 16), (33, 8, 128, 64), (7, 2, 256, 32), (260, 1, 576, 16), (3, 1, 1024, 1), (17, 5, 40, 3)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
def test_append(rows, heads, dim, page, e4m3, layout):
    g = A.gen(rows + heads + dim)
    n_pages = rows // page + 3
    slots = torch.randperm(n_pages * page, generator=g)[:rows]
    if rows > 2:
        slots[1], slots[2] = -1, n_pages * page          # neither is a slot
    x = [torch.randn(rows, heads, dim, generator=g).bfloat16() for _ in range(2)]
    for t in x:
        t[0] = 0
    old = [torch.randn(n_pages, page, heads, dim, generator=g) for _ in range(2)]
    old = [t.to(E4M3) if e4m3 else t.bfloat16() for t in old]
    if layout == "heads":        # [n_pages, heads, page, dim] in memory
        caches = [(dev(t.view(torch.uint8).transpose(1, 2).contiguous()).view(E4M3) if e4m3 else dev(t.transpose(1, 2).contiguous())).transpose(1, 2) for t in old]
    elif layout == "both":       # keys and values of a page side by side
        both = torch.stack([t.view(torch.uint8) if e4m3 else t for t in old], 1).to(DEV)
        caches = [(both[:, i].view(E4M3) if e4m3 else both[:, i]) for i in range(2)]
    else:
        caches = [dev(t) for t in old]
    scales = [torch.full((n_pages, heads, page), -1.0, device=DEV) for _ in range(2)] if e4m3 else [None, None]
    wide = torch.zeros(rows, heads, dim + 8, dtype=BF, device=DEV)
    wide[..., :dim] = dev(x[1])
    ops.kv_append(dev(x[0]), caches[0], dev(slots), v=wide[..., :dim], v_cache=caches[1], k_scale=scales[0], v_scale=scales[1])
    for t, cache, was, s in zip(x, caches, old, scales):
        got, want = cache.float().cpu().flatten(0, 1), was.float().flatten(0, 1)
        gs, ws = s.cpu().transpose(1, 2).flatten(0, 1) if e4m3 else None, torch.full((n_pages * page, heads), -1.0)
        for i, at in enumerate(slots.tolist()):
            if not 0 <= at < n_pages * page:
                continue
            if e4m3:
                v, a = t[i].double(), t[i].double().abs().amax(-1, keepdim=True)
                # the code is half a step of 8 bits off, relative or of the smallest step 2^-9; scale, 448 / a, and
                # their products with code and row are one rounding of fp32 each
                half = torch.maximum(A.E4M3_HALF * v.abs(), 2.0 ** -10 * a / 448)
                A.close((got[at].double() * gs[at].double()[:, None]), v, half * (1 + 4 * A.U) + 4 * A.U * v.abs())
                ws[at] = (t[i].float().abs().amax(-1) / 448.0)
                want[at] = got[at]
            else:
                want[at] = t[i].float()
        assert torch.equal(got, want)
        if e4m3:
            A.close(gs, ws.double(), A.U * ws.abs().double())


def test_append_one_kind_of_rows_and_none():
    g = A.gen(3)
    x, cache, slots = torch.randn(9, 320, generator=g).bfloat16(), torch.zeros(4, 16, 320, dtype=BF), torch.randperm(64, generator=g)[:9]
    c = dev(cache)
    ops.kv_append(dev(x), c, dev(slots))
    cache.flatten(0, 1)[slots] = x
    assert torch.equal(c.cpu(), cache)
    ops.kv_append(dev(x[:0]), c, dev(slots[:0]))
    assert torch.equal(c.cpu(), cache)


def test_append_8_bit_zeros_nan_infinity_and_tiny_rows():
    x = torch.randn(6, 1, 64, generator=A.gen(1)).bfloat16()
    x[0] = 0
    x[1, 0, 5] = math.nan
    x[2, 0, 6] = -math.inf
    x[3] *= 2.0 ** -125
    x[4] = 2.0 ** -133                       # the smallest bf16 number
    x[5] = torch.finfo(BF).max
    c, s = torch.zeros(1, 16, 1, 64, dtype=E4M3, device=DEV), torch.zeros(1, 1, 16, device=DEV)
    ops.kv_append(dev(x), c, torch.arange(6, device=DEV), k_scale=s)
    s, v = s.cpu().flatten(), c.float().cpu().flatten(0, 1)[:6, 0]
    assert s[0] == 0 and (v[0] == 0).all() and s[1].isnan() and s[2].isinf()
    for i in (3, 4, 5):
        want = x[i, 0].double()
        got = v[i].double() * s[i].double()
        a = want.abs().max()
        # half a step of the code, and what fp32 loses of a scale below its smallest normal number
        assert ((got - want).abs() <= A.E4M3_HALF * want.abs() * 1.01 + a * 2.0 ** -16 + 448 * 2.0 ** -149).all(), i


# ------------------------------------------------------------------- paged
def caches_of(g, n, page, kv, dim, e4m3, layout="tokens"):
    """(device cache, device scales, float64 values) of keys or values."""
    x = torch.randn(n, page, kv, dim, generator=g).bfloat16()
    if not e4m3:
        d = dev(x) if layout == "tokens" else dev(x.transpose(1, 2).contiguous()).transpose(1, 2)
        return d, None, x.double()
    q, s = A.rows8(x)
    b = q.view(torch.uint8)
    d = dev(b).view(E4M3) if layout == "tokens" else dev(b.transpose(1, 2).contiguous()).view(E4M3).transpose(1, 2)
    return d, dev(s.transpose(1, 2).contiguous()), q.double() * s.double()[..., None]


def run_paged(lens, heads, kv, dim, page, e4m3=False, window=0, layout="tokens", scale=None, extra=0, seed=0, **kw):
    g = A.gen(seed + heads + dim + sum(lens))
    table, n = A.place(g, lens, page, max(1, -(-max(lens, default=0) // page)) + extra)
    k, ks, kd = caches_of(g, n, page, kv, dim, e4m3, layout)
    v, vs, vd = caches_of(g, n, page, kv, dim, e4m3, layout)
    q = (1.5 * torch.randn(len(lens), heads, dim, generator=g)).bfloat16()
    args = dict(scale=scale, window=window, k_scale=ks, v_scale=vs, lse=True, **kw)
    got = ops.paged_attention(dev(q), k, v, dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV), **args)
    out, tol, lse, lse_tol = A.paged(q, kd, vd, table, lens, scale or dim ** -0.5, window)
    A.close(got[0], out, tol, "out")
    A.close(got[1], lse, lse_tol, "lse")
    return got


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 8), (12, 4), (16, 1), (17, 1), (40, 1), (66, 2), (130, 1)])
def test_paged(dim, e4m3, heads, kv):
    run_paged([5, 0, 97, 300], heads, kv, dim, 16, e4m3)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_lengths(page, layout, e4m3):
    run_paged([1, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 500, 0, 513], 4, 2, 64, page, e4m3, layout=layout, extra=page % 5)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 1000, 5000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_window(window, e4m3):
    run_paged([1, 17, 100, 130, 1100, 4097], 6, 2, 64, 32, e4m3, window=window)


@pytest.mark.parametrize("lens", [[9000], [3, 12000, 700], [4096] * 5])
@pytest.mark.parametrize("e4m3,dim,heads,kv", [(False, 128, 8, 1), (True, 128, 4, 4), (False, 256, 20, 1), (True, 64, 3, 3)])
def test_paged_split(lens, e4m3, dim, heads, kv):
    run_paged(lens, heads, kv, dim, 64, e4m3)


def test_paged_many_requests():
    rng = random.Random(3)
    run_paged([rng.choice([0, 1, 20, 40, 300]) for _ in range(600)], 2, 1, 64, 16)


def test_paged_scale_and_sharp_scores():
    run_paged([700, 33], 4, 2, 128, 16, scale=0.02)
    run_paged([700, 33], 4, 2, 128, 16, scale=1.0)
    run_paged([1500], 4, 2, 64, 16, e4m3=True, scale=2.0)


def test_paged_rising_scores():
    """Every token beats the ones before it: the running maximum rises all the way."""
    g = A.gen(2)
    n, dim = 2000, 64
    k = torch.zeros(n // 16, 16, 1, dim)
    k.view(n, dim)[:, 0] = torch.arange(n) / 8.0
    k, v = k.bfloat16(), torch.randn(n // 16, 16, 1, dim, generator=g).bfloat16()
    q = torch.zeros(2, 3, dim).bfloat16()
    q[0, :, 0], q[1, :, 0] = 4.0, -4.0
    table = torch.arange(n // 16, dtype=torch.int32).expand(2, -1).contiguous()
    got = ops.paged_attention(*dev(q, k, v, table), torch.tensor([n, n], dtype=torch.int32, device=DEV), scale=1.0)
    # scores are multiples of 1/8 below 1024: exact in fp32; weights fall off within 40 tokens
    out, tol, _, _ = A.paged(q, k.double(), v.double(), table, [n, n], 1.0)
    A.close(got, out, tol)


def test_paged_nothing_outside_reaches_a_request():
    """NaN and infinities behind the last token, before the window, on other pages and in the scales there."""
    for e4m3 in (False, True):
        g = A.gen(5)
        lens, page, dim = [37, 130, 0, 300], 32, 64
        table, n = A.place(g, lens, page, 12)
        k, ks, kd = caches_of(g, n, page, 2, dim, e4m3)
        v, vs, vd = caches_of(g, n, page, 2, dim, e4m3)
        q = torch.randn(4, 4, dim, generator=g).bfloat16()
        window = 100
        seen = torch.zeros(n, page, dtype=torch.bool)
        for b, m in enumerate(lens):
            for t in range(max(0, m - window), m):
                seen[table[b, t // page], t % page] = True
        bad = dev(~seen)
        for x, s in ((k, ks), (v, vs)):
            if e4m3:
                x.view(torch.uint8)[bad] = 0x7F
                s.transpose(1, 2)[bad] = math.nan
            else:
                x[bad] = math.nan
                x[bad.nonzero()[::2, 0], bad.nonzero()[::2, 1]] = math.inf
        got = ops.paged_attention(dev(q), k, v, dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV), window=window, k_scale=ks, v_scale=vs)
        out, tol, _, _ = A.paged(q, kd, vd, table, lens, dim ** -0.5, window)
        A.close(got, out, tol)


def test_paged_pages_that_the_cache_lacks_have_no_tokens():
    g = A.gen(6)
    lens, page, dim = [100, 64, 33], 16, 128
    table, n = A.place(g, lens, page, 8)
    table[0, 2], table[0, 6], table[1, :4], table[2, 0] = -1, n, -5, 2 ** 31 - 1
    k, _, kd = caches_of(g, n, page, 1, dim, False)
    v, _, vd = caches_of(g, n, page, 1, dim, False)
    q = torch.randn(3, 2, dim, generator=g).bfloat16()
    out, tol, lse, lse_tol = A.paged(q, kd, vd, table, lens, dim ** -0.5)
    got = ops.paged_attention(dev(q), k, v, dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV), lse=True)
    A.close(got[0], out, tol)
    A.close(got[1], lse, lse_tol)
    # lengths beyond the table count as its width, below zero as none
    got = ops.paged_attention(dev(q), k, v, dev(table), torch.tensor([10 ** 6, -3, 33], dtype=torch.int32, device=DEV))
    A.close(got, *A.paged(q, kd, vd, table, [128, 0, 33], dim ** -0.5)[:2])


def test_paged_nan_and_infinity_in_a_seen_token_stay_in_their_request_and_head():
    g = A.gen(7)
    lens = [50, 60, 2000]
    table, n = A.place(g, lens, 16, 125)
    k, _, kd = caches_of(g, n, 16, 2, 64, False)
    v, _, vd = caches_of(g, n, 16, 2, 64, False)
    q = torch.randn(3, 2, 64, generator=g).bfloat16()
    k[table[0, 1], 3, 0, 7] = math.nan
    v[table[2, 70], 5, 1, 9] = math.inf
    got = ops.paged_attention(dev(q), k, v, dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV)).cpu()
    out, tol, _, _ = A.paged(q, kd, vd, table, lens, 0.125)
    assert got[0, 0].isnan().all() and got[2, 1, 9].isinf()
    out[0, 0], out[2, 1, 9] = math.nan, math.inf
    A.close(got, out, tol)


def test_paged_strided_queries_outputs_and_workspace():
    g = A.gen(8)
    lens = [700, 20]
    table, n = A.place(g, lens, 16, 50)
    both = torch.randn(n, 2, 16, 2, 64, generator=g).bfloat16().to(DEV)
    wide = torch.randn(2, 7, 192, generator=g).bfloat16().to(DEV)
    q = wide[:, :4, 64:128]
    out = torch.full((4, 3, 128), 7.0, dtype=BF, device=DEV)
    view = out.transpose(0, 1)[:2, :, :64]
    lse = torch.zeros(2, 4, device=DEV)
    need = ops.paged_attention_bytes(2, 2, 2, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    table_wide = torch.full((2, 60), 10 ** 6, dtype=torch.int32, device=DEV)
    table_wide[:, :50] = dev(table)
    got = ops.paged_attention(q, both[:, 0], both[:, 1], table_wide[:, :50], torch.tensor(lens, dtype=torch.int32, device=DEV), out=view, lse=lse,
                              workspace=ws)
    assert got[0] is view and got[1] is lse
    want, tol, wl, lt = A.paged(q.cpu(), both[:, 0].double().cpu(), both[:, 1].double().cpu(), table, lens, 0.125)
    A.close(view, want, tol)
    A.close(lse, wl, lt)
    assert (out[:, 2] == 7).all() and (out[..., 64:] == 7).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_and_paged_beyond_32_bits(e4m3):
    """Pages further apart than 32 bits of bytes."""
    g = A.gen(12)
    page, kv, dim, stride, n = 16, 2, 128, (1 << 31) + 4096, 3
    lens = [40, 16]
    table = torch.tensor([[2, 0, 1], [2, -1, -1]], dtype=torch.int32)
    typ = E4M3 if e4m3 else BF
    caches = []
    for _ in range(2):
        room = torch.empty((n - 1) * stride + page * kv * dim, dtype=torch.uint8 if e4m3 else BF, device=DEV).view(typ)
        caches.append(room.as_strided((n, page, kv, dim), (stride, kv * dim, dim, 1)))
    k, v = (torch.randn(n * page, kv, dim, generator=g).bfloat16() for _ in range(2))
    scales = [torch.zeros(n, kv, page, device=DEV) if e4m3 else None for _ in range(2)]
    ops.kv_append(dev(k), caches[0], torch.arange(n * page, device=DEV), v=dev(v), v_cache=caches[1], k_scale=scales[0], v_scale=scales[1])

    def seen(x, c, s):
        if not e4m3:
            assert torch.equal(c.cpu(), x.reshape(n, page, kv, dim))
            return x.double().reshape(n, page, kv, dim)
        return c.cpu().double() * s.transpose(1, 2).cpu().double()[..., None]

    q = torch.randn(2, 4, dim, generator=g).bfloat16()
    got = ops.paged_attention(dev(q), *caches, dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV), k_scale=scales[0], v_scale=scales[1])
    want = A.paged(q, seen(k, caches[0], scales[0]), seen(v, caches[1], scales[1]), table, lens, dim ** -0.5)
    A.close(got, *want[:2])


@pytest.mark.parametrize("kind", ["paged", "latent"])
def test_as_many_tokens_as_a_length_counts(kind):
    """2^31 - 16 tokens, of which only the first and the last page are there."""
    g = A.gen(14)
    width = 2 ** 27 - 1
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    table[0, 0], table[0, -1] = 1, 0
    lens = torch.tensor([16 * width], dtype=torch.int32, device=DEV)
    small = torch.tensor([[1, 0]], dtype=torch.int32)
    if kind == "paged":
        q = torch.randn(1, 2, 64, generator=g).bfloat16()
        k, _, kd = caches_of(g, 2, 16, 1, 64, False)
        v, _, vd = caches_of(g, 2, 16, 1, 64, False)
        A.close(ops.paged_attention(dev(q), k, v, table, lens), *A.paged(q, kd, vd, small, [32], 0.125)[:2])
        A.close(ops.paged_attention(dev(q), k, v, table, lens, window=20), *A.paged(q, kd, vd, small[:, 1:], [16], 0.125)[:2])
    else:
        q, w, cache, _ = latent_inputs([32], 2, 256, 32, 64, 16)
        A.close(ops.latent_attention(*dev(q, w, cache[:2]), table, lens, nope=64), *A.latent(q, w, cache[:2], small, [32], 64, 96 ** -0.5)[:2])


def test_parts_of_a_cache_are_joined_by_lse():
    g = A.gen(9)
    table, n = A.place(g, [640], 16, 40)
    k, _, kd = caches_of(g, n, 16, 1, 128, False)
    v, _, vd = caches_of(g, n, 16, 1, 128, False)
    q = dev(torch.randn(1, 4, 128, generator=g).bfloat16())
    whole, lse = ops.paged_attention(q, k, v, dev(table), torch.tensor([640], dtype=torch.int32, device=DEV), lse=True)
    a, la = ops.paged_attention(q, k, v, dev(table[:, :25].contiguous()), torch.tensor([400], dtype=torch.int32, device=DEV), lse=True)
    b, lb = ops.paged_attention(q, k, v, dev(table[:, 25:].contiguous()), torch.tensor([240], dtype=torch.int32, device=DEV), lse=True)
    l = torch.logaddexp(la.double(), lb.double())
    joined = a.double() * (la - l).exp()[..., None] + b.double() * (lb - l).exp()[..., None]
    # three results, each with its weights' and its own rounding
    assert ((joined - whole.double()).abs() <= 6 * A.BF16_HALF * vd.abs().max()).all()
    assert ((l - lse.double()).abs() < 1e-4).all()


# ------------------------------------------------------------------ latent
def latent_inputs(lens, heads, rank, rope, nope, page, extra=0, seed=0):
    g = A.gen(seed + heads + rank + sum(lens))
    table, n = A.place(g, lens, page, max(1, -(-max(lens, default=0) // page)) + extra)
    cache = torch.randn(n, page, rank + rope, generator=g).bfloat16()
    w = (torch.randn(heads, 2 * nope, rank, generator=g) / math.sqrt(rank)).bfloat16()
    q = torch.randn(len(lens), heads, nope + rope, generator=g).bfloat16()
    return q, w, cache, table


def run_latent(lens, heads, rank, rope, nope, page, scale=None, **kw):
    q, w, cache, table = latent_inputs(lens, heads, rank, rope, nope, page, **kw)
    got = ops.latent_attention(*dev(q, w, cache, table), torch.tensor(lens, dtype=torch.int32, device=DEV), nope=nope, scale=scale, lse=True)
    out, tol, lse, lse_tol = A.latent(q, w, cache, table, lens, nope, scale or (nope + rope) ** -0.5)
    A.close(got[0], out, tol, "out")
    A.close(got[1], lse, lse_tol, "lse")


@pytest.mark.parametrize("rank,rope,nope", [(512, 64, 128), (512, 32, 64), (256, 64, 64), (256, 32, 128)])
@pytest.mark.parametrize("heads", [1, 12, 16, 17, 40, 64, 128])
def test_latent(rank, rope, nope, heads):
    run_latent([70, 0, 1, 333], heads, rank, rope, nope, 16)


@pytest.mark.parametrize("page", [16, 48, 64, 512])
@pytest.mark.parametrize("heads", [3, 30, 50, 100])
def test_latent_lengths(page, heads):
    run_latent([1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 0], heads, 256, 32, 64, page, extra=page % 7)


@pytest.mark.parametrize("heads", [2, 20, 64, 70])
def test_latent_split(heads):
    run_latent([9100, 30], heads, 512, 64, 64, 64)
    run_latent([3000] * 3, heads, 256, 64, 128, 16)


def test_latent_piece_longer_than_its_table_of_blocks():
    """More than 8192 tokens in one piece: enough requests that each has one."""
    run_latent([8200 + i for i in range(2)] + [20] * 300, 130, 256, 32, 64, 16)


def test_latent_many_requests_and_scale():
    rng = random.Random(5)
    run_latent([rng.choice([0, 1, 30, 100]) for _ in range(400)], 2, 256, 32, 64, 16, scale=0.5)


def test_latent_nothing_outside_reaches_a_request():
    lens, page = [37, 130, 0, 700], 32
    q, w, cache, table = latent_inputs(lens, 20, 512, 64, 128, page, extra=2)
    table[1, 1] = -1
    seen = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for b, m in enumerate(lens):
        for t in range(m):
            if table[b, t // page] >= 0:
                seen[table[b, t // page], t % page] = True
    want = A.latent(q, w, cache, table, lens, 128, 192 ** -0.5)
    cache[~seen] = math.nan
    at = (~seen).nonzero()[::2]
    cache[at[:, 0], at[:, 1]] = math.inf
    got = ops.latent_attention(*dev(q, w, cache, table), torch.tensor(lens, dtype=torch.int32, device=DEV), nope=128)
    A.close(got, *want[:2])


def test_latent_strided_rows_outputs_and_workspace():
    lens = [300, 40]
    q, w, cache, table = latent_inputs(lens, 5, 256, 64, 64, 16)
    wide = torch.zeros(cache.shape[0], 16, 400, dtype=BF, device=DEV)
    wide[..., 40:360] = dev(cache)
    qw = torch.zeros(5, 2, 200, dtype=BF, device=DEV).transpose(0, 1)
    qw[..., 8:136] = dev(q)
    out = torch.full((2, 6, 80), 3.0, dtype=BF, device=DEV)
    ws = torch.full((ops.latent_attention_bytes(2, 5, 256),), 255, dtype=torch.uint8, device=DEV)
    ops.latent_attention(qw[..., 8:136], dev(w), wide[..., 40:360], dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV), nope=64,
                         out=out[:, :5, 16:], workspace=ws)
    want = A.latent(q, w, cache, table, lens, 64, 128 ** -0.5)
    A.close(out[:, :5, 16:], *want[:2])
    assert (out[:, 5] == 3).all() and (out[..., :16] == 3).all()


def test_latent_pages_beyond_32_bits():
    lens = [40, 16]
    q, w, cache, table = latent_inputs(lens, 5, 256, 32, 64, 16)
    n, stride = cache.shape[0], (1 << 30) + 4096
    far = torch.empty((n - 1) * stride + 16 * 288, dtype=BF, device=DEV).as_strided((n, 16, 288), (stride, 288, 1))
    far.copy_(dev(cache))
    got = ops.latent_attention(*dev(q, w), far, dev(table), torch.tensor(lens, dtype=torch.int32, device=DEV), nope=64)
    A.close(got, *A.latent(q, w, cache, table, lens, 64, 96 ** -0.5)[:2])


# ------------------------------------------------------------------ prompt
def starts_of(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def prompt_inputs(nq, nk, heads, rank, rope, nope, seed=0):
    g = A.gen(seed + heads + sum(nq) + sum(nk))
    lat = torch.randn(sum(nk), rank + rope, generator=g).bfloat16()
    w = (torch.randn(heads, 2 * nope, rank, generator=g) / math.sqrt(rank)).bfloat16()
    q = torch.randn(sum(nq), heads, nope + rope, generator=g).bfloat16()
    return q, lat, w


def run_prompt(nq, nk, heads, rank, rope, nope, scale=None):
    q, lat, w = prompt_inputs(nq, nk, heads, rank, rope, nope)
    qs, ks = starts_of(nq), starts_of(nk)
    got = ops.latent_prompt(*dev(q, lat, w, torch.tensor(qs, dtype=torch.int32)), k_starts=torch.tensor(ks, dtype=torch.int32, device=DEV), nope=nope,
                            scale=scale, lse=True)
    out, tol, lse, lse_tol = A.prompt(q, lat, w, qs, ks, nope, scale or (nope + rope) ** -0.5)
    A.close(got[0], out, tol, "out")
    A.close(got[1], lse, lse_tol, "lse")


@pytest.mark.parametrize("rank,rope,nope", [(512, 64, 128), (512, 32, 64), (256, 64, 64), (256, 32, 128)])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_prompt(rank, rope, nope, heads):
    run_prompt([70, 0, 1, 150], [70, 0, 1, 150], heads, rank, rope, nope)


@pytest.mark.parametrize("nq,nk", [([1, 2, 3], [1, 200, 64]), ([31, 32, 33], [31, 95, 97]), ([127, 128, 129], [127, 128, 129]), ([260], [333]),
                                   ([5, 0, 7], [0, 9, 7]), ([70], [20]), ([63, 64, 65], [64, 64, 64])])
def test_prompt_lengths(nq, nk):
    run_prompt(nq, nk, 2, 256, 32, 64)


def test_prompt_tiles_of_256_queries():
    """Enough rows and heads for the larger tiles."""
    run_prompt([300, 257, 700], [300, 400, 700], 64, 256, 32, 64)


def test_prompt_scale():
    run_prompt([100], [130], 2, 512, 64, 128, scale=1.0)
    run_prompt([100], [130], 2, 512, 64, 128, scale=0.01)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_prompt_hidden_rows_do_not_reach_a_query(bad):
    nq, nk = [150, 90], [180, 90]
    q, lat, w = prompt_inputs(nq, nk, 2, 256, 32, 64)
    qs, ks = starts_of(nq), starts_of(nk)
    out, tol, _, _ = A.prompt(q, lat, w, qs, ks, 64, 96 ** -0.5)
    lat[100, 5] = bad                        # of the first request: queries 70.. see it
    lat[ks[1] + 40, 3] = bad                 # of the second: queries 40.. see it
    got = ops.latent_prompt(*dev(q, lat, w, torch.tensor(qs, dtype=torch.int32)), k_starts=torch.tensor(ks, dtype=torch.int32, device=DEV), nope=64).cpu()
    clean = list(range(70)) + list(range(150, 190))
    A.close(got[clean], out[clean], tol[clean])
    assert not got[70:150].isfinite().all(-1).any() and not got[190:].isfinite().all(-1).any()


def test_prompt_strides_and_rows_of_no_request():
    nq, nk = [40, 33], [60, 33]
    q, lat, w = prompt_inputs(nq, nk, 3, 256, 64, 64)
    wide_q = torch.zeros(100, 4, 136, dtype=BF, device=DEV)
    wide_q[10:83, :3, 8:] = dev(q)
    wide_l = torch.full((120, 336), math.nan, dtype=BF, device=DEV)
    wide_l[5:98, 8:328] = dev(lat)
    out = torch.full((100, 3, 72), 5.0, dtype=BF, device=DEV)
    lse = torch.full((100, 3), 5.0, device=DEV)
    qs, ks = [10, 50, 83], [5, 65, 98]
    i32 = dict(dtype=torch.int32, device=DEV)
    ops.latent_prompt(wide_q[:, :3, 8:], wide_l[:, 8:328], dev(w), torch.tensor(qs, **i32), k_starts=torch.tensor(ks, **i32), nope=64, out=out[..., 8:],
                      lse=lse)
    want, tol, wl, lt = A.prompt(q, lat, w, starts_of(nq), starts_of(nk), 64, 128 ** -0.5)
    A.close(out[10:83, :, 8:], want, tol)
    A.close(lse[10:83], wl, lt)
    assert (out[:10] == 5).all() and (out[83:] == 5).all() and (out[..., :8] == 5).all() and (lse[83:] == 5).all()


def test_prompt_starts_beyond_the_rows_are_left_out():
    nq = [50, 40]
    q, lat, w = prompt_inputs(nq, nq, 2, 256, 32, 64)
    want, tol, _, _ = A.prompt(q, lat, w, [0, 50, 90], [0, 50, 90], 64, 96 ** -0.5)
    got = ops.latent_prompt(*dev(q, lat, w, torch.tensor([0, 50, 90, 400, 500], dtype=torch.int32)), nope=64)
    A.close(got, want, tol)
    out = torch.full((90, 2, 64), 2.0, dtype=BF, device=DEV)
    ops.latent_prompt(*dev(q, lat, w, torch.tensor([95, 300], dtype=torch.int32)), nope=64, out=out)
    assert (out == 2).all()


def test_prompt_rows_beyond_32_bits():
    """A workspace and inputs of more than 4 GiB: the last of 70 requests, and the first."""
    heads, rank, rope, nope, n, each = 128, 256, 32, 128, 70, 1000
    g = torch.Generator(device=DEV).manual_seed(13)
    lat = torch.randn(n * each, rank + rope, generator=g, device=DEV).bfloat16()
    w = (torch.randn(heads, 2 * nope, rank, generator=g, device=DEV) / math.sqrt(rank)).bfloat16()
    q = torch.randn(n, heads, nope + rope, generator=g, device=DEV).bfloat16()
    far = torch.empty((n - 1) * (1 << 26) + heads * (nope + rope), dtype=BF, device=DEV).as_strided(q.shape, (1 << 26, nope + rope, 1))
    far.copy_(q)
    out = torch.empty((n - 1) * (1 << 26) + heads * nope, dtype=BF, device=DEV).as_strided((n, heads, nope), (1 << 26, nope, 1))
    ks = torch.arange(0, n * each + 1, each, dtype=torch.int32, device=DEV)
    ops.latent_prompt(far, lat, w, torch.arange(n + 1, dtype=torch.int32, device=DEV), k_starts=ks, nope=nope, out=out)
    for b in (0, n - 1):
        h = [0, 77, 127]
        want = A.prompt(q[b:b + 1, h].cpu(), lat[b * each:(b + 1) * each].cpu(), w[h].cpu(), [0, 1], [0, each], nope, (nope + rope) ** -0.5)
        A.close(out[b:b + 1, h], *want[:2])


def test_both_forms_agree():
    """One request, token by token over its cache, and as a prompt."""
    g = A.gen(11)
    n, heads, rank, rope, nope = 40, 6, 512, 64, 128
    q, lat, w = prompt_inputs([n], [n], heads, rank, rope, nope)
    whole = ops.latent_prompt(*dev(q, lat, w, torch.tensor([0, n], dtype=torch.int32)), nope=nope)
    table, pages = A.place(g, [n], 16, 3)
    cache = torch.zeros(pages, 16, rank + rope, dtype=BF, device=DEV)
    t = torch.arange(n)
    ops.kv_append(dev(lat), cache, dev(table[0].long()[t // 16] * 16 + t % 16))
    step = ops.latent_attention(*dev(q, w), cache, dev(table.expand(n, -1).contiguous()), torch.arange(1, n + 1, dtype=torch.int32, device=DEV), nope=nope)
    a = A.prompt(q, lat, w, [0, n], [0, n], nope, 192 ** -0.5)
    b = A.latent(q, w, cache.cpu(), table.expand(n, -1), list(range(1, n + 1)), nope, 192 ** -0.5)
    # each within its bound of its own formula, and the formulas differ by the roundings that the bounds' first terms count
    A.close(whole, *a[:2])
    A.close(step, *b[:2])
    assert ((whole - step).float().norm() / step.float().norm()) < 4 * A.BF16_HALF
