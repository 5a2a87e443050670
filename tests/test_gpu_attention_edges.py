"""The attention half's operators on the GPU in calls that are empty, ragged, tied or far out."""
import gc
import weakref

import pytest
import torch

import attention_plain as A
from sync_protocols_amd import attention_layer as L
from sync_protocols_amd import decode_layer as D
from sync_protocols_amd import fg, ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
E4M3 = torch.float8_e4m3fn


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# --------------------------------------------------------------- page_step
@pytest.mark.parametrize("in_place", [False, True])
def test_page_step_of_no_request_and_no_token(in_place):
    """The ring's ends and the one entry of starts are outputs all the same."""
    ends = torch.tensor([7, 12], device=DEV)
    starts = torch.full((1,), 99, dtype=torch.int32, device=DEV)
    out = ends if in_place else torch.full((2,), -1, device=DEV)
    got = ops.page_step(i32(), i32(), torch.empty(0, 4, dtype=torch.int32, device=DEV), i32(*range(20)), ends, page=16, tokens=0, ends_out=out, starts=starts)
    assert got.ends.tolist() == [7, 12] and got.starts.tolist() == [0]
    assert got.slots.shape == got.positions.shape == got.lens.shape == (0,)


# ------------------------------------------------------------------ prompt
def prompt_inputs(nq, nk, heads, seed):
    g = A.gen(seed)
    lat = torch.randn(nk, 288, generator=g).bfloat16()
    w = (torch.randn(heads, 128, 256, generator=g) / 16).bfloat16()
    return torch.randn(nq, heads, 96, generator=g).bfloat16(), lat, w


@pytest.mark.parametrize("q_starts,k_starts", [
    ([-1000, 50, 90], [-1000, 50, 90]), ([-1000, -500, -3, 0, 40, 90], [-9, -9, -3, 0, 40, 90]), ([-70000, 0, 90], [0, 0, 90]),
    ([-2 ** 31, -2 ** 31, 90], [-2 ** 31, -2 ** 31, 90]), ([-2 ** 31, 30, 2 ** 31 - 1], [-2 ** 31, 30, 2 ** 31 - 1]), ([-5, 60, 5000], [-800, 60, 100]),
    ([0, 90, 2 ** 31 - 1], [0, 90, 2 ** 31 - 1]), ([10, 20, 80], [500, 600, 700])])
def test_prompt_starts_outside_the_rows_count_as_the_nearest_row(q_starts, k_starts):
    nq, nk, heads = 90, 100, 2
    q, lat, w = prompt_inputs(nq, nk, heads, 21)
    out, lse = torch.full((nq, heads, 64), 5.0, dtype=BF, device=DEV), torch.full((nq, heads), 5.0, device=DEV)
    ops.latent_prompt(q.to(DEV), lat.to(DEV), w.to(DEV), i32(*q_starts), k_starts=i32(*k_starts), nope=64, out=out, lse=lse)
    qs, ks = ([min(max(s, 0), n) for s in v] for v, n in ((q_starts, nq), (k_starts, nk)))
    want, tol, wl, lt = A.prompt(q, lat, w, qs, ks, 64, 96 ** -0.5)
    A.close(out[qs[0]:qs[-1]], want[qs[0]:qs[-1]], tol[qs[0]:qs[-1]], "out")
    A.close(lse[qs[0]:qs[-1]], wl[qs[0]:qs[-1]], lt[qs[0]:qs[-1]], "lse")
    assert (out[:qs[0]] == 5).all() and (out[qs[-1]:] == 5).all() and (lse[:qs[0]] == 5).all() and (lse[qs[-1]:] == 5).all()


def test_prompt_of_as_many_requests_and_heads_as_fill_a_grid():
    """65535 requests with 256 heads: 2^24 workgroups, more than one dimension of a grid holds. The first and the last request have rows."""
    heads = 256
    q, lat, w = prompt_inputs(130, 130, heads, 23)
    starts = torch.full((65536,), 60, dtype=torch.int32, device=DEV)
    starts[0], starts[-1] = 0, 130
    got, lse = ops.latent_prompt(q.to(DEV), lat.to(DEV), w.to(DEV), starts, nope=64, lse=True)
    for h in ([0, 1], [127, 255]):
        want, tol, wl, lt = A.prompt(q[:, h], lat, w[h], [0, 60, 130], [0, 60, 130], 64, 96 ** -0.5)
        A.close(got[:, h], want, tol)
        A.close(lse[:, h], wl, lt)


# ------------------------------------------------------------------ append
def codes(x):
    """e4m3 codes of x * 448 / max |x|. The quotient of bf16 numbers lies on a border between two codes or at least 2^-13 of itself away
    from one (x 448 has 11 bits, max |x| 8, the border 5), so a quotient in 64 bits decides like an exact one; a border goes to the even code."""
    a = x.double().abs().amax(-1, keepdim=True)
    v = (x.double() * 448 / torch.where(a > 0, a, 1)).abs()
    step = torch.exp2(torch.floor(torch.log2(v.clamp_min(2.0 ** -6))) - 3)
    return torch.copysign(torch.round(v / step) * step, x.double())          # torch.round: ties to even


@pytest.mark.parametrize("dim", [64, 128, 256, 576])
def test_append_8_bit_codes_are_those_of_the_exact_quotient(dim):
    """Every code of many rows, quotients on the border between two codes among them."""
    g = A.gen(dim)
    rows = 2048
    x = torch.randn(rows, 1, dim, generator=g).bfloat16()
    # x = T a / 448 for borders T: a = 7 2^k b makes them numbers of 8 bits
    a = 7 * torch.randint(16, 19, (rows // 2, 1), generator=g) * torch.exp2(torch.randint(-90, 90, (rows // 2, 1), generator=g).double())
    border = torch.tensor([17, 19, 21, 23, 25, 27, 29, 31, 1, 3, 5, 7, 9, 11, 13, 15]) * torch.tensor([2.0 ** -4] * 8 + [2.0 ** -10] * 8)
    pick = border[torch.randint(0, 16, (rows // 2, dim), generator=g)] * torch.exp2(torch.randint(0, 4, (rows // 2, dim), generator=g).double())
    tied = pick.double() * a / 448
    tied = torch.where(tied.bfloat16().double() == tied, tied, torch.zeros_like(tied))
    tied[:, 0] = a[:, 0]
    x[rows // 2:, 0] = tied.bfloat16()
    x[5] *= 2.0 ** -120
    cache, scale = torch.zeros(rows // 16, 16, 1, dim, dtype=E4M3, device=DEV), torch.zeros(rows // 16, 1, 16, device=DEV)
    ops.kv_append(x.to(DEV), cache, torch.arange(rows, device=DEV), k_scale=scale)
    assert torch.equal(cache.cpu().double().flatten(0, 1), codes(x))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kind", ["page", "token", "head", "columns", "pages"])
def test_append_into_caches_that_lie_within_each_other(kind, e4m3):
    """Keys and values of a page, a token or a head side by side in one buffer, and two caches of other strides page beside page."""
    n, page, kv, dim = 4, 16, 3, 64
    g = A.gen(41)
    x = [torch.randn(20, kv, dim, generator=g).bfloat16() for _ in range(2)]
    slots = torch.randperm(n * page, generator=g)[:20]
    room = torch.zeros(n * page * kv * dim * 2, dtype=torch.uint8 if e4m3 else BF, device=DEV)
    if kind == "page":
        k, v = room.view(n, 2, page, kv, dim).unbind(1)
    elif kind == "token":
        k, v = room.view(n, page, 2, kv, dim).unbind(2)
    elif kind == "head":
        k, v = room.view(n, page, kv, 2, dim).unbind(3)
    elif kind == "columns":
        k, v = room.view(n, page, kv, 2 * dim).split(dim, -1)
    else:                    # keys by token, values by head, in the two halves of a page
        both = room.view(n, 2, page * kv * dim)
        k, v = both[:, 0].unflatten(1, (page, kv, dim)), both[:, 1].unflatten(1, (kv, page, dim)).transpose(1, 2)
    typ = E4M3 if e4m3 else BF
    scales = [torch.zeros(n, kv, page, device=DEV) if e4m3 else None for _ in range(2)]
    ops.kv_append(x[0].to(DEV), k.view(typ), slots.to(DEV), v=x[1].to(DEV), v_cache=v.view(typ), k_scale=scales[0], v_scale=scales[1])
    for t, c in zip(x, (k, v)):
        want = torch.zeros(n * page, kv, dim, dtype=torch.float64)
        want[slots] = codes(t) if e4m3 else t.double()
        assert torch.equal(c.view(typ).cpu().double().reshape(n * page, kv, dim), want)


# --------------------------------------------------------------- broadcasts
def test_broadcast_inputs():
    """Inputs with strides of zero, as expand() makes them, their row in the gap between two rows of the output where that is possible."""
    g = A.gen(31)
    lens, table = [20, 33], torch.tensor([[0, 1, -1], [2, 1, 0]], dtype=torch.int32)
    row = torch.randn(4, 64, generator=g).bfloat16()
    k, v = torch.randn(3, 16, 2, 64, generator=g).bfloat16(), torch.randn(3, 16, 1, 64, generator=g).bfloat16().expand(3, 16, 2, 64)
    room = torch.zeros(2, 1024, dtype=BF, device=DEV)
    room[0, 512:768] = row.flatten().to(DEV)
    q = room[0, 512:768].view(1, 4, 64).expand(2, 4, 64)
    out = room[:, :256].unflatten(1, (4, 64))
    ops.paged_attention(q, k.to(DEV), v[:, :, :1].to(DEV).expand(3, 16, 2, 64), table.to(DEV), i32(*lens), out=out)
    A.close(out, *A.paged(row.expand(2, 4, 64), k.double(), v.double(), table, lens, 0.125)[:2])
    cache = torch.zeros(3, 16, 2, 64, dtype=BF, device=DEV)
    ops.kv_append(row[:1].to(DEV).expand(7, 2, 64), cache, torch.arange(7, device=DEV) * 5)
    assert (cache.flatten(0, 1)[:35:5].cpu() == row[0]).all() and (cache.flatten(0, 1)[1:35:5] == 0).all()
    # one row of queries at all positions of a prompt
    qp, lat, w = prompt_inputs(1, 40, 2, 32)
    got = ops.latent_prompt(qp.to(DEV).expand(40, 2, 96), lat.to(DEV), w.to(DEV), i32(0, 40), nope=64)
    A.close(got, *A.prompt(qp.expand(40, 2, 96), lat, w, [0, 40], [0, 40], 64, 96 ** -0.5)[:2])


# ------------------------------------------------------------------ graphs
@pytest.mark.parametrize("kind", ["paged", "latent"])
def test_captured_step_keeps_what_its_graph_addresses(kind):
    """Tables, lengths, ring, caches and weights stay when the program puts others in their place."""
    pages = L.Pages(2, 4, 8, 16, DEV)
    attention = L.random_paged(256, 4, 2, 64, pages, group=64) if kind == "paged" else L.random_latent(256, 4, 256, 32, 64, pages, group=64)
    captured = L.CapturedDecode(attention, D.random_layer(256, 128, 256, 8, 8, 2, group=32, device=DEV), 2)
    held = {f"{type(o).__name__}.{k}": weakref.ref(v) for o in (attention, pages) for k, v in vars(o).items() if isinstance(v, torch.Tensor)}
    assert len(held) > 6
    for o in (attention, pages):
        for k, v in list(vars(o).items()):
            if isinstance(v, torch.Tensor):
                setattr(o, k, v.clone())
    del v
    gc.collect()
    assert [k for k, r in held.items() if r() is None] == []
    captured.add.fill_(1)
    captured.replay()
    torch.cuda.synchronize()
    assert captured.weights and pages.lens.tolist() == [0, 0]


# ------------------------------------------------------------------ layers
def test_step_of_other_rows_than_requests_leaves_the_pages():
    pages = L.Pages(3, 4, 12, 16, DEV)
    attention, experts = L.random_paged(256, 4, 2, 64, pages, group=64), D.random_layer(256, 128, 256, 8, 8, 2, group=32, device=DEV)
    for rows in (0, 2, 4):
        with pytest.raises(fg.FgError):
            L.decode_step(attention, experts, torch.zeros(rows, 256, dtype=BF, device=DEV), i32(1, 1, 1))
        assert pages.lens.tolist() == [0, 0, 0] and pages.ends.tolist() == [0, 12]


def test_layers_that_share_their_pages():
    """One step of the pages, every layer's step with its slots, against layers with pages of their own; a request without a slot is told by its length."""
    shared = L.Pages(3, 2, 4, 16, DEV)
    layers = [L.random_paged(256, 4, 2, 64, shared, group=64, seed=1), L.random_latent(256, 4, 256, 32, 64, shared, group=64, seed=2)]
    alone = [L.random_paged(256, 4, 2, 64, L.Pages(3, 2, 4, 16, DEV), group=64, seed=1), L.random_latent(256, 4, 256, 32, 64, L.Pages(3, 2, 4, 16, DEV), group=64, seed=2)]
    g = torch.Generator(device=DEV).manual_seed(9)
    for step in range(20):
        x = torch.randn(3, 256, device=DEV, generator=g).to(BF)
        before = shared.lens.clone()
        p = shared.step(i32(1, 1, 1), 3)
        served = p.starts[1:] > p.starts[:-1]
        assert torch.equal(shared.lens - before, served.int())
        at = p.starts[:-1].long().clamp_max(2)
        slots, positions = torch.where(served, p.slots[at], -1), torch.where(served, p.positions[at], 0)
        for a, b in zip(layers, alone):
            q = b.pages.step(i32(1, 1, 1), 3)
            assert torch.equal(q.slots, p.slots)
            assert torch.equal(a.step(x, slots, positions), b.step(x, slots, positions))
    assert sorted(shared.lens.tolist()) == [16, 16, 20]
