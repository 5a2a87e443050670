"""Refusals of outputs that lie on inputs, of gradients, and of sizes no grid holds, without a GPU: nothing is launched."""
import pytest
import torch

from sync_protocols_amd import fg, ops
from test_ops_refusals import P, _moe, _route, _w4

FAR = P + (1 << 30)      # the outputs, away from everything that lies at P


@pytest.mark.parametrize("kw", [
    dict(out=P), dict(out=P, n=256, ldo=256), dict(out=P + 2, n=1, ldo=1), dict(x=FAR + 112), dict(x=FAR + 48, rows=1), dict(w=FAR),
    dict(w=FAR - 32 * 128 + 16), dict(s=FAR + 62), dict(s=FAR - 62), dict(z=FAR + 127), dict(b=FAR + 2), dict(t=1, xs=FAR + 4),
    dict(t=1, xs=FAR + 120, xg=128), dict(x=FAR - 512 * 3 + 16, ldx=768, rows=2), dict(x=FAR, ldx=64, k=64, g=32, n=32, ldo=40, rows=20)])
def test_w4_refuses_out_on_an_input(kw):
    a = dict(out=FAR)
    a.update(kw)
    assert _w4(**a) == fg.EINVAL


@pytest.mark.parametrize("kw", [dict(topk=P), dict(w=P), dict(topk=P + 63 * 4), dict(w=P + 4 * 64 + 4), dict(topk=FAR, w=FAR + 4), dict(l=FAR + 32, w=P)])
def test_route_refuses_outputs_on_its_logits_or_each_other(kw):
    a = dict(topk=FAR, w=FAR + 4096)
    a.update(kw)
    assert _route(**a) == fg.EINVAL


@pytest.mark.parametrize("kw", [
    dict(ws=P), dict(y=P + (1 << 24), ws=P + (1 << 24)), dict(y=FAR + 16 + 4 * 2 * 2 * 64 - 2, ws=FAR + 16), dict(topk=FAR + 8), dict(topk=FAR - 12), dict(w2=FAR),
    dict(w=FAR + (1 << 20) + 4), dict(x=FAR + (1 << 20) + 16), dict(w1=FAR + (1 << 20)), dict(g=32, s1=FAR + (1 << 20), s2=P), dict(g=32, s1=P, s2=FAR),
    dict(g=32, s1=P, s2=P, z2=FAR + 7), dict(g=32, s1=P, s2=P, z1=FAR + (1 << 20)), dict(t=1, xs=FAR + (1 << 20))])
def test_moe_refuses_outputs_on_what_it_still_reads(kw):
    """y may lie on x: the first kernel has read it."""
    a = dict(y=FAR, ws=FAR + (1 << 20))
    a.update(kw)
    assert _moe(**a) == fg.EINVAL


# ------------------------------------------------------------------ autograd

def _grad(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, requires_grad=True)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


W = ops.W4Weight(torch.zeros(32, 128, dtype=torch.uint8), _bf(32, 2))
PICKS = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
CALLS = [
    lambda: ops.add_rmsnorm(_grad(2, 8), _bf(8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _grad(8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), residual=_grad(2, 8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), y=_grad(2, 8)),
    lambda: ops.add_rmsnorm(_grad(2, 8) * 2, _bf(8)),
    lambda: ops.moe_route(_grad(2, 8), 2),
    lambda: ops.w4_linear(_grad(2, 256), W),
    lambda: ops.w4_linear(_bf(2, 256), ops.W4Weight(W.q, _grad(32, 2))),
    lambda: ops.w4_linear(_bf(2, 256), W, bias=_grad(32)),
    lambda: ops.w4_linear(_bf(2, 256), W, out=_grad(2, 32)),
    lambda: ops.moe_few(_grad(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), *PICKS),
    lambda: ops.moe_few(_bf(2, 64), _grad(4, 64, 64), _bf(4, 64, 32), *PICKS),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), PICKS[0], PICKS[1].clone().requires_grad_()),
]


@pytest.mark.parametrize("call", CALLS)
def test_tensors_that_require_gradients_are_refused(call):
    """There is no backward pass: a result cut off from its inputs would be a silent loss."""
    with pytest.raises(fg.FgError, match="no backward pass") as e:
        call()
    assert e.value.code == fg.EINVAL
    with torch.no_grad(), pytest.raises(fg.FgError, match="on the GPU"):      # the next refusal, of these CPU tensors
        call()


# --------------------------------------------------------------------- grids
def test_moe_refuses_the_first_grid_of_eight_waves_that_does_not_fit():
    """2^23 workgroups of 512 threads are 2^32 threads: 8 experts of 2^24 columns, more than 16 tokens each."""
    far = 1 << 45
    many = dict(tokens=64, k=4, e=8, K=32, ldx=32, F=1 << 24, g=32, s1=P, s2=P, ldy=32, wsb=1 << 45, ws=far, y=far - 65536)
    assert _moe(**many) == fg.EINVAL
