"""The decoding operators together: one decoder layer's half from the attention
output to the expert layer's result, for a step of 1 to 64 tokens.

    o      = wo a                              4-bit output projection   (w4_linear)
    h      = o + residual
    n      = rms_norm(h) * gamma               8-bit codes and bf16      (add_rmsnorm)
    p      = top-k of router n                                           (moe_route)
    y      = sum_j p_j expert_j(n)             this GPU's experts        (moe_few)

With the experts spread over GPUs every one runs the same step on its share
(`expert_base`, the leading size of w1) and the results y are added.

    python -m sync_protocols_amd.decode_layer [--tokens N] [--hidden ..] [--width ..]

runs it on random weights, call by call and as a graph, and prints the time of each
and how far the results are from the same step in float32. With --attention paged
or latent a step starts at the layer's input instead: attention_layer's half, over a
paged cache of --context tokens a request, in front of this one.
"""
from __future__ import annotations

import argparse
import math
from typing import NamedTuple, Optional

import torch

from . import ops


class StepResult(NamedTuple):
    y: torch.Tensor             # bf16 [tokens, hidden]: this GPU's experts' part
    residual: torch.Tensor      # bf16 [tokens, hidden]: o + residual


class ExpertLayer:
    """Weights of the half layer. `wo` [hidden, heads] 4-bit; gamma bf16 [hidden];
    router bf16 [experts, hidden]; w1 [n_local, 2 width, hidden] and w2 [n_local,
    hidden, width], both 4-bit or both bf16. `norm_out` is the type of the experts'
    input: "e4m3" and "i8" (scales per 128 columns where hidden allows) or "bf16".
    Parameters serve as weights under torch.no_grad(): a step has no backward pass."""

    def __init__(self, wo: ops.W4Weight, gamma: torch.Tensor, router: torch.Tensor, w1, w2, top_k: int, *, expert_base: int = 0,
                 score: str = "softmax", eps: float = 1e-6, norm_out: str = "e4m3"):
        self.wo, self.gamma, self.router, self.w1, self.w2 = wo, gamma, router, w1, w2
        self.top_k, self.expert_base, self.score, self.eps, self.norm_out = top_k, expert_base, score, eps, norm_out
        self.group = 128 if norm_out != "bf16" and gamma.numel() % 128 == 0 else 0
        first = w2.q if isinstance(w2, ops.W4Weight) else w2
        self.width = first.shape[2] * (2 if isinstance(w2, ops.W4Weight) else 1)

    def workspace(self, tokens: int) -> torch.Tensor:
        """Scratch memory of a step; a program keeps one for its steps, which follow each other on one stream."""
        return torch.empty(ops.moe_few_bytes(tokens, self.top_k, self.width), dtype=torch.uint8, device=self.gamma.device)

    def step(self, a: torch.Tensor, residual: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> StepResult:
        """a bf16 [tokens, heads], residual bf16 [tokens, hidden]."""
        o = ops.w4_linear(a, self.wo)
        n = ops.add_rmsnorm(o, self.gamma, residual=residual, eps=self.eps, out=self.norm_out, group=self.group, keep_bf16=True)
        topk, weights = ops.moe_route(torch.nn.functional.linear(n.y, self.router), self.top_k, score=self.score)
        x = n.y if self.norm_out == "bf16" else n.q
        y = ops.moe_few(x, self.w1, self.w2, topk, weights, expert_base=self.expert_base, x_scale=n.scale, workspace=workspace)
        return StepResult(y, n.sum)


class CapturedStep:
    """A step of a fixed number of tokens as one graph launch: fill `a` and
    `residual`, call replay(), read `result`. The graph holds the addresses of the
    layer's weights as they were, so those tensors are kept with it."""

    def __init__(self, layer: ExpertLayer, tokens: int, heads: int):
        hidden, device = layer.gamma.numel(), layer.gamma.device
        self.a = torch.zeros(tokens, heads, dtype=torch.bfloat16, device=device)
        self.residual = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device=device)
        self.workspace = layer.workspace(tokens)
        self.weights = (layer.wo, layer.gamma, layer.router, layer.w1, layer.w2)
        side = torch.cuda.Stream(device)
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):          # the library product's own setup happens here, outside the graph
            layer.step(self.a, self.residual, self.workspace)
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.result = layer.step(self.a, self.residual, self.workspace)

    def replay(self) -> StepResult:
        self.graph.replay()
        return self.result


def random_weight4(n: int, k: int, group: int, lead=(), device="cuda", generator=None) -> ops.W4Weight:
    """4-bit weights of standard deviation about 1 / sqrt(k)."""
    q = torch.randint(0, 256, (*lead, n, k // 2), dtype=torch.uint8, device=device, generator=generator)
    scale = torch.rand(*lead, n, k // group, device=device, generator=generator) + 0.5
    return ops.W4Weight(q, (scale * (0.22 / math.sqrt(k))).bfloat16(), None)


def dequantise(w: ops.W4Weight) -> torch.Tensor:
    """float32 [.., n, k]."""
    v = torch.stack((w.q & 15, w.q >> 4), -1).flatten(-2).float().unflatten(-1, (w.scale.shape[-1], -1))
    return ((v - (8.0 if w.zero is None else w.zero.float().unsqueeze(-1))) * w.scale.float().unsqueeze(-1)).flatten(-2)


def plain_step(layer: ExpertLayer, a: torch.Tensor, residual: torch.Tensor, topk: torch.Tensor, weights: torch.Tensor) -> StepResult:
    """The same step in float32, unquantised between the operators, for given picks."""
    h = a.float() @ dequantise(layer.wo).t() + residual.float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + layer.eps) * layer.gamma.float()
    quant = isinstance(layer.w1, ops.W4Weight)
    y = torch.zeros_like(n)
    for e in range((layer.w1.q if quant else layer.w1).shape[0]):
        t, j = torch.nonzero(topk == e + layer.expert_base, as_tuple=True)
        if not t.numel():
            continue
        w1, w2 = (dequantise(ops.W4Weight(*(None if v is None else v[e] for v in w))) if quant else w[e].float() for w in (layer.w1, layer.w2))
        gate, up = (n[t] @ w1.t()).chunk(2, 1)
        y.index_add_(0, t, (gate * torch.sigmoid(gate) * up) @ w2.t() * weights[t, j].unsqueeze(1))
    return StepResult(y, h)


def random_layer(hidden: int, width: int, heads: int, experts: int, n_local: int, top_k: int, *, group: int = 128, norm_out: str = "e4m3",
                 device="cuda", seed: int = 0) -> ExpertLayer:
    g = torch.Generator(device=device).manual_seed(seed)
    gamma = (1 + 0.1 * torch.randn(hidden, device=device, generator=g)).bfloat16()
    router = (torch.randn(experts, hidden, device=device, generator=g) / math.sqrt(hidden)).bfloat16()
    return ExpertLayer(random_weight4(hidden, heads, group, (), device, g), gamma, router,
                       random_weight4(2 * width, hidden, group, (n_local,), device, g),
                       random_weight4(hidden, width, group, (n_local,), device, g), top_k, norm_out=norm_out)


def _time_us(f, repeat: int) -> float:
    for _ in range(3):
        f()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(repeat):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / repeat * 1e3


def _whole_layer(c) -> None:
    from . import attention_layer as A
    page, new = 64, 3 * c.repeat + 16
    width = -(-(c.context + new) // page)
    pages = A.Pages(c.tokens, width, c.tokens * width, page)
    if c.attention == "paged":
        attention = A.random_paged(c.hidden, c.heads // 128, max(1, c.heads // 512), 128, pages)
    else:
        attention = A.random_latent(c.hidden, c.heads // 128, 512, 64, 128, pages)
    experts = random_layer(c.hidden, c.width, c.heads, c.experts, c.local, c.top_k, norm_out=c.norm_out)
    g = torch.Generator(device="cuda").manual_seed(1)
    for cache in (attention.k, attention.v) if c.attention == "paged" else (attention.cache,):
        cache.normal_(generator=g)
    pages.step(torch.full_like(pages.lens, c.context), 0 if c.context == 0 else c.tokens * c.context)
    captured = A.CapturedDecode(attention, experts, c.tokens)
    captured.x.normal_(generator=g)
    captured.add.fill_(1)
    before = pages.lens.clone(), pages.ends.clone()
    want = A.decode_step(attention, experts, captured.x, captured.add)
    pages.lens.copy_(before[0])
    pages.ends.copy_(before[1])
    got = captured.replay()
    torch.cuda.synchronize()
    print(f"{c.tokens} requests of {c.context} tokens, {c.attention} attention: graph equals calls: {torch.equal(got.y, want.y)}")
    print(f"call by call {_time_us(lambda: A.decode_step(attention, experts, captured.x, captured.add, *captured.workspace), c.repeat):.1f} us, "
          f"as a graph {_time_us(captured.replay, c.repeat):.1f} us a step")


def main(argv=None) -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--hidden", type=int, default=7168)
    p.add_argument("--width", type=int, default=2048)
    p.add_argument("--heads", type=int, default=4096, help="columns of the attention output")
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--local", type=int, default=8, help="experts on this GPU")
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--norm-out", choices=("bf16", "i8", "e4m3"), default="e4m3")
    p.add_argument("--repeat", type=int, default=50)
    p.add_argument("--attention", choices=("none", "paged", "latent"), default="none")
    p.add_argument("--context", type=int, default=4096, help="tokens that a request has in the cache")
    c = p.parse_args(argv)
    if c.attention != "none":
        return _whole_layer(c)
    layer = random_layer(c.hidden, c.width, c.heads, c.experts, c.local, c.top_k, norm_out=c.norm_out)
    captured = CapturedStep(layer, c.tokens, c.heads)
    g = torch.Generator(device="cuda").manual_seed(1)
    captured.a.copy_(torch.randn(c.tokens, c.heads, device="cuda", generator=g))
    captured.residual.copy_(torch.randn(c.tokens, c.hidden, device="cuda", generator=g))
    got = layer.step(captured.a, captured.residual)
    again = captured.replay()
    torch.cuda.synchronize()
    o = ops.w4_linear(captured.a, layer.wo)
    n = ops.add_rmsnorm(o, layer.gamma, residual=captured.residual, eps=layer.eps)
    topk, weights = ops.moe_route(torch.nn.functional.linear(n.y, layer.router), layer.top_k, score=layer.score)
    want = plain_step(layer, captured.a, captured.residual, topk, weights)
    off = (got.y.float() - want.y).norm() / want.y.norm()
    print(f"{c.tokens} tokens, {c.local} of {c.experts} experts of {c.hidden} x {c.width}: graph equals calls: {torch.equal(got.y, again.y)}, "
          f"relative distance to float32 {float(off):.4f} ({c.norm_out} expert inputs)")
    print(f"call by call {_time_us(lambda: layer.step(captured.a, captured.residual, captured.workspace), c.repeat):.1f} us, "
          f"as a graph {_time_us(captured.replay, c.repeat):.1f} us a step")


if __name__ == "__main__":
    main()
