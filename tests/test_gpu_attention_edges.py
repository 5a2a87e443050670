"""The attention half's operators on the GPU in calls that are empty, ragged, tied or far out."""
import pytest
import torch

import attention_plain as A
from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


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
