"""Attention over a paged cache where a workgroup's piece is longer than the list of pages that it holds at a time, and where
tokens that are seen hold NaN or infinities, one piece of many. Requests share pages, so that long ones need little memory."""
import math

import pytest
import torch

import attention_plain as A
from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def dev(*ts):
    r = [t.to(DEV) for t in ts]
    return r if len(r) > 1 else r[0]


def lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


def longest_piece(lens, unit, target):
    """Tokens of the longest piece of one request, when `target` workgroups take equal shares of all requests' units."""
    units = [max(1, -(-n // unit)) for n in lens]
    total = sum(units)
    n = min(target, total)
    share, more = total // n, total % n
    ends = [w * share + min(w, more) for w in range(n + 1)]
    best = at = 0
    for u in units:
        best = max([best] + [min(e, at + u) - max(s, at) for s, e in zip(ends, ends[1:])])
        at += u
    return best * unit


def shared_pages(g, lens, page, n):
    """A table of n pages that all requests use, each in an order of its own."""
    table = torch.full((len(lens), -(-max(lens) // page)), -1, dtype=torch.int32)
    for b, m in enumerate(lens):
        k = -(-m // page)
        table[b, :k] = torch.randint(0, n, (k,), generator=g)
    return table


LIST = 1024          # tokens of the 64 blocks whose pages a wave holds


@pytest.mark.parametrize("heads,requests,length,page", [(128, 64, 4000, 64), (40, 140, 9000, 16), (20, 128, 5000, 16), (5, 130, 5000, 48)])
def test_latent_pieces_longer_than_the_list_of_pages(heads, requests, length, page):
    g = A.gen(heads)
    lens = [length - 7 * b for b in range(requests)]
    # workgroups: one a compute unit and 64 heads, or two for up to 32 heads
    target, unit = (256 // -(-heads // 64), 64) if heads > 32 else (512, 32)
    assert longest_piece(lens, unit, target) > LIST + 2 * unit
    n = 70
    table = shared_pages(g, lens, page, n)
    cache = torch.randn(n, page, 288, generator=g).bfloat16()
    w = (torch.randn(heads, 128, 256, generator=g) / 16).bfloat16()
    q = torch.randn(requests, heads, 96, generator=g).bfloat16()
    got, lse = ops.latent_attention(*dev(q, w, cache, table), lengths(lens), nope=64, lse=True)
    some = [0, requests // 2, requests - 1]
    out, tol, wl, lt = A.latent(q[some], w, cache, table[some], [lens[b] for b in some], 64, 96 ** -0.5)
    A.close(got[some], out, tol, "out")
    A.close(lse[some], wl, lt, "lse")


@pytest.mark.parametrize("dim,window", [(64, 0), (64, 35000), (128, 0), (256, 0)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_pieces_longer_than_the_list_of_pages(dim, window, e4m3):
    g = A.gen(dim + window)
    kv, page, n, lens = 64, 16, 50, [41000, 30001]
    # 512 workgroups over 64 key heads; a piece's four waves share its tiles of 32 tokens
    assert longest_piece([min(m, window or m) for m in lens], 128, 8) > 4 * (LIST + 64)
    table = shared_pages(g, lens, page, n)
    k, v = (torch.randn(n, page, kv, dim, generator=g).bfloat16() for _ in range(2))
    q = (1.5 * torch.randn(2, kv, dim, generator=g)).bfloat16()
    scales, kd, vd = {}, k.double(), v.double()
    if e4m3:
        (k, ks), (v, vs) = A.rows8(k), A.rows8(v)
        kd, vd = k.double() * ks.double()[..., None], v.double() * vs.double()[..., None]
        scales = dict(k_scale=dev(ks.transpose(1, 2).contiguous()), v_scale=dev(vs.transpose(1, 2).contiguous()))
    got, lse = ops.paged_attention(*dev(q, k, v, table), lengths(lens), window=window, lse=True, **scales)
    h = [0, 29, 63]
    out, tol, wl, lt = A.paged(q[:, h], kd[:, :, h], vd[:, :, h], table, lens, dim ** -0.5, window)
    A.close(got[:, h], out, tol, "out")
    A.close(lse[:, h], wl, lt, "lse")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [2, 20, 70])
def test_latent_bad_numbers_in_a_seen_token_stay_in_their_request(heads, bad):
    """In the latent part every score of the request is NaN or infinite, or its value is; one piece of many, and a request of one piece."""
    g = A.gen(heads + 1)
    lens, page = [9100, 40, 333, 30], 16
    table, n = A.place(g, lens, page, 569)
    cache = torch.randn(n, page, 288, generator=g).bfloat16()
    w = (torch.randn(heads, 128, 256, generator=g) / 16).bfloat16()
    q = torch.randn(4, heads, 96, generator=g).bfloat16()
    out, tol, wl, lt = A.latent(q, w, cache, table, lens, 64, 96 ** -0.5)
    for b, t in ((0, 4567), (3, 12)):
        cache[table[b, t // page].item(), t % page, 77] = bad
    got, lse = (x.cpu() for x in ops.latent_attention(*dev(q, w, cache, table), lengths(lens), nope=64, lse=True))
    A.close(got[1:3], out[1:3], tol[1:3], "out")
    A.close(lse[1:3], wl[1:3], lt[1:3], "lse")
    # the mean has a NaN (0 times an infinity where the weight is zero), and every result takes part of it
    assert got[0].isnan().all() and got[3].isnan().all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("heads", [2, 20, 70])
def test_latent_infinite_scores(heads, sign):
    """An infinity in the rotary key of the last token: heads whose query turns it to minus infinity are as without the token, the others NaN."""
    g = A.gen(heads + 2)
    lens, page = [9100, 40, 333], 16
    table, n = A.place(g, lens, page, 569)
    cache = torch.randn(n, page, 288, generator=g).bfloat16()
    w = (torch.randn(heads, 128, 256, generator=g) / 16).bfloat16()
    q = torch.randn(3, heads, 96, generator=g).bfloat16()
    without = [lens[0] - 1, lens[1] - 1, lens[2]]
    out, tol, wl, lt = A.latent(q, w, cache, table, without, 64, 96 ** -0.5)
    for b in (0, 1):
        t = lens[b] - 1
        cache[table[b, t // page].item(), t % page, 256 + 9] = sign * math.inf
    got, lse = (x.cpu() for x in ops.latent_attention(*dev(q, w, cache, table), lengths(lens), nope=64, lse=True))
    away = q[:, :, 64 + 9].double() * sign < 0
    away[2] = True
    assert (away[:2].any() or heads == 2) and not away[:2].all()
    A.close(got[away], out[away], tol[away], "out")
    A.close(lse[away], wl[away], lt[away], "lse")
    assert got[~away].isnan().all() and lse[~away].isnan().all()
