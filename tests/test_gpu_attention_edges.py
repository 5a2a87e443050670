"""The attention half's operators on the GPU in calls that are empty, ragged, tied or far out."""
import pytest
import torch

from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


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
