"""The half decoder layer built from the decoding operators, against its float32 form."""
import pytest
import torch

from sync_protocols_amd import decode_layer as D
from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(tokens, heads, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, heads, generator=g).bfloat16().to(DEV), torch.randn(tokens, hidden, generator=g).bfloat16().to(DEV))


def _picks(layer, a, residual):
    n = ops.add_rmsnorm(ops.w4_linear(a, layer.wo), layer.gamma, residual=residual, eps=layer.eps)
    return ops.moe_route(torch.nn.functional.linear(n.y, layer.router), layer.top_k, score=layer.score)


# Relative to the norm of y. bf16 roundings (2^-8 / sqrt(3) each at most, in the mean): o, the experts' input and y, all
# multiplied by about 3 through SiLU's product; e4m3 adds 2^-4 / sqrt(3) and int8 6 / 127 / sqrt(12) of an element.
@pytest.mark.parametrize("norm_out,tol", [("bf16", 0.02), ("i8", 0.06), ("e4m3", 0.12)])
@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_step(tokens, norm_out, tol):
    layer = D.random_layer(512, 256, 384, 16, 16, 4, group=64, norm_out=norm_out, device=DEV, seed=tokens)
    a, residual = _inputs(tokens, 384, 512, tokens)
    got, want = layer.step(a, residual), D.plain_step(layer, a, residual, *_picks(layer, a, residual))
    assert (got.y.float() - want.y).norm() <= tol * want.y.norm()
    assert (got.residual.float() - want.residual).norm() <= 2.0 ** -7 * want.residual.norm()


def test_shares_of_experts_add_up():
    layer = D.random_layer(256, 128, 256, 12, 12, 3, group=32, device=DEV)
    a, residual = _inputs(9, 256, 256, 3)
    whole = layer.step(a, residual).y.float()
    part = torch.zeros_like(whole)
    for base in (0, 4, 8):
        w1, w2 = (ops.W4Weight(w.q[base:base + 4], w.scale[base:base + 4]) for w in (layer.w1, layer.w2))
        share = D.ExpertLayer(layer.wo, layer.gamma, layer.router, w1, w2, 3, expert_base=base)
        part += share.step(a, residual).y.float()
    assert (part - whole).abs().max() <= 4 * 2.0 ** -8 * whole.abs().max()


def test_captured_step_replays():
    layer = D.random_layer(384, 192, 256, 8, 8, 2, group=32, device=DEV)
    captured = D.CapturedStep(layer, 5, 256)
    for seed in range(4):
        a, residual = _inputs(5, 256, 384, seed)
        captured.a.copy_(a)
        captured.residual.copy_(residual)
        want = layer.step(a, residual)
        torch.cuda.synchronize()
        got = captured.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.y, want.y) and torch.equal(got.residual, want.residual), seed


def test_command(capsys):
    D.main(["--tokens", "3", "--hidden", "256", "--width", "128", "--heads", "128", "--experts", "8", "--local", "8", "--top-k", "2", "--repeat", "2"])
    assert "graph equals calls: True" in capsys.readouterr().out
