"""The attention half of a decoder layer from the attention operators: one step of
1 to 64 requests, whose output goes to decode_layer.ExpertLayer.

    slots, positions, lengths            pages of the step, once for all layers      (page_step)
    n      = rms_norm(x) * gamma                                                     (add_rmsnorm)
    q, k, v = wqkv n                      4-bit projection, q and k turned            (w4_linear)
    cache[slots] = k, v                                                              (kv_append)
    a      = attention of q over the request's pages                                 (paged_attention)

LatentAttention keeps one row [latent | rotary key] a token instead of keys and
values of every head:

    q, c, r = wq n, wc n                  c normed, q's last columns and r turned     (w4_linear, add_rmsnorm)
    cache[slots] = [c | r]                                                           (kv_append)
    a      = attention over the request's pages, keys and values W_k c, W_v c         (latent_attention)

and takes prompts too (prompt: latent_prompt over the new rows)."""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import decode_layer, fg, ops


class Pages:
    """Pages of up to `batch` requests of up to `width` pages each, all on the GPU. step()
    takes the new tokens' counts (negative: the request has ended) and returns their slots and
    positions; `table` and `lens` are what the attention reads. Layers may share one: step() is then called once for all of them."""

    def __init__(self, batch: int, width: int, n_pages: int, page: int, device="cuda"):
        self.page, self.n_pages = page, n_pages
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.ring = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.ends = torch.tensor([0, n_pages], dtype=torch.int64, device=device)

    def step(self, add: torch.Tensor, tokens: int) -> ops.PageStep:
        return ops.page_step(self.lens, add, self.table, self.ring, self.ends, page=self.page, tokens=tokens, lens_out=self.lens, ends_out=self.ends)


def turn(x: torch.Tensor, positions: torch.Tensor, base: float = 10000.0) -> torch.Tensor:
    """Rotary embedding of x [rows, heads, columns] (halves turned against each other) at int32 positions [rows]."""
    half = x.shape[-1] // 2
    freq = torch.exp(torch.arange(half, dtype=torch.float64, device=x.device) * (-math.log(base) / half))
    angle = (positions.double()[:, None] * freq)[:, None]
    c, s = angle.cos().float(), angle.sin().float()
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat((a * c - b * s, b * c + a * s), -1).to(x.dtype)


class PagedAttention:
    """gamma bf16 [hidden]; wqkv 4-bit [(heads + 2 kv) * dim, hidden], queries' rows first, then keys', then
    values'. `e4m3` keeps the cache as 8-bit rows with a scale a token and head."""

    def __init__(self, gamma: torch.Tensor, wqkv: ops.W4Weight, heads: int, kv: int, dim: int, pages: Pages, *, e4m3: bool = False, window: int = 0,
                 eps: float = 1e-6):
        self.gamma, self.wqkv, self.heads, self.kv, self.dim, self.pages, self.window, self.eps = gamma, wqkv, heads, kv, dim, pages, window, eps
        shape = (pages.n_pages, pages.page, kv, dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=gamma.device) for _ in range(2))
        self.k_scale, self.v_scale = ((torch.zeros(pages.n_pages, kv, pages.page, device=gamma.device) if e4m3 else None) for _ in range(2))

    def workspace(self, tokens: int) -> torch.Tensor:
        return torch.empty(ops.paged_attention_bytes(tokens, self.kv, self.heads // self.kv, self.dim), dtype=torch.uint8, device=self.gamma.device)

    def step(self, x: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x bf16 [requests, hidden], one new token of each: bf16 [requests, heads * dim]."""
        n = ops.add_rmsnorm(x, self.gamma, eps=self.eps).y
        qkv = ops.w4_linear(n, self.wqkv).unflatten(1, (-1, self.dim))
        qk = turn(qkv[:, :self.heads + self.kv], positions)
        ops.kv_append(qk[:, self.heads:], self.k, slots, v=qkv[:, self.heads + self.kv:], v_cache=self.v, k_scale=self.k_scale, v_scale=self.v_scale)
        return ops.paged_attention(qk[:, :self.heads], self.k, self.v, self.pages.table, self.pages.lens, window=self.window, k_scale=self.k_scale,
                                   v_scale=self.v_scale, workspace=workspace).flatten(1)


class LatentAttention:
    """gamma bf16 [hidden]; wq 4-bit [heads * (nope + rope), hidden]; wc 4-bit [rank + rope, hidden]; latent_gamma bf16
    [rank]; w bf16 [heads, 2 nope, rank]."""

    def __init__(self, gamma: torch.Tensor, wq: ops.W4Weight, wc: ops.W4Weight, latent_gamma: torch.Tensor, w: torch.Tensor, rope: int, pages: Pages, *,
                 eps: float = 1e-6):
        self.gamma, self.wq, self.wc, self.latent_gamma, self.w, self.rope, self.pages, self.eps = gamma, wq, wc, latent_gamma, w, rope, pages, eps
        self.heads, self.nope, self.rank = w.shape[0], w.shape[1] // 2, w.shape[2]
        self.cache = torch.zeros(pages.n_pages, pages.page, self.rank + rope, dtype=torch.bfloat16, device=gamma.device)

    def workspace(self, tokens: int) -> torch.Tensor:
        return torch.empty(ops.latent_attention_bytes(tokens, self.heads, self.rank), dtype=torch.uint8, device=self.gamma.device)

    def _rows(self, x, positions):
        n = ops.add_rmsnorm(x, self.gamma, eps=self.eps).y
        q = ops.w4_linear(n, self.wq).unflatten(1, (self.heads, -1))
        row = ops.w4_linear(n, self.wc)
        c, r = row[:, :self.rank], row[:, self.rank:]
        ops.add_rmsnorm(c, self.latent_gamma, eps=self.eps, y=c)
        r.copy_(turn(r[:, None], positions)[:, 0])
        return torch.cat((q[..., :self.nope], turn(q[..., self.nope:], positions)), -1), row

    def step(self, x: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x bf16 [requests, hidden], one new token of each: bf16 [requests, heads * nope]."""
        q, row = self._rows(x, positions)
        ops.kv_append(row, self.cache, slots)
        return ops.latent_attention(q, self.w, self.cache, self.pages.table, self.pages.lens, nope=self.nope, workspace=workspace).flatten(1)

    def prompt(self, x: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor, starts: torch.Tensor) -> torch.Tensor:
        """x bf16 [rows, hidden]: whole prompts, request b's rows starts[b]..starts[b + 1]-1."""
        q, row = self._rows(x, positions)
        ops.kv_append(row, self.cache, slots)
        return ops.latent_prompt(q, row, self.w, starts, nope=self.nope).flatten(1)


class CapturedDecode:
    """One decoding step of `tokens` requests through the attention and expert halves as one graph launch:
    pages, projections, cache, attention, experts. Fill `x` and `add` (1: a new token, 0: none, negative: ended),
    call replay(), read `result`; the pages move on by themselves, so no other layer shares them. A request that
    gets no slot keeps its length in attention.pages.lens and gives a row that means nothing."""

    def __init__(self, attention, experts: decode_layer.ExpertLayer, tokens: int):
        hidden, device = experts.gamma.numel(), experts.gamma.device
        self.attention, self.experts = attention, experts
        self.x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device=device)
        self.add = torch.zeros(tokens, dtype=torch.int32, device=device)
        self.workspace = attention.workspace(tokens), experts.workspace(tokens)
        self.weights = [v for o in (attention, experts, attention.pages) for v in vars(o).values()]          # the graph holds their addresses
        side = torch.cuda.Stream(device)
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):          # without new tokens: nothing moves on; the library product's own setup happens here
            self._step()
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.result = self._step()

    def _step(self):
        return decode_step(self.attention, self.experts, self.x, self.add, *self.workspace)

    def replay(self) -> decode_layer.StepResult:
        self.graph.replay()
        return self.result


def decode_step(attention, experts: decode_layer.ExpertLayer, x: torch.Tensor, add: torch.Tensor, attention_workspace=None, expert_workspace=None):
    """x bf16 [requests, hidden]; add int32 [requests], 1 for those that have a new token. Both halves of a layer that
    has its pages to itself, as it moves them on: where layers share their pages, call pages.step once and every
    layer's step with its slots and positions. A request that got its slot has a length one higher than before."""
    if x.shape[0] != attention.pages.lens.numel():
        raise fg.FgError(fg.EINVAL, "x must have one row a request of the pages")
    p = attention.pages.step(add, x.shape[0])
    # tokens are numbered over the served requests; here every request has a row, so its slot is looked up
    at = p.starts[:-1].long().clamp_max(x.shape[0] - 1)
    served = p.starts[1:] > p.starts[:-1]
    slots, positions = torch.where(served, p.slots[at], -1), torch.where(served, p.positions[at], 0)
    a = attention.step(x, slots, positions, attention_workspace)
    return experts.step(a, x, expert_workspace)


def random_paged(hidden: int, heads: int, kv: int, dim: int, pages: Pages, *, group: int = 128, e4m3: bool = False, seed: int = 0) -> PagedAttention:
    device = pages.lens.device
    g = torch.Generator(device=device).manual_seed(seed)
    gamma = (1 + 0.1 * torch.randn(hidden, device=device, generator=g)).bfloat16()
    return PagedAttention(gamma, decode_layer.random_weight4((heads + 2 * kv) * dim, hidden, group, (), device, g), heads, kv, dim, pages, e4m3=e4m3)


def random_latent(hidden: int, heads: int, rank: int, rope: int, nope: int, pages: Pages, *, group: int = 128, seed: int = 0) -> LatentAttention:
    device = pages.lens.device
    g = torch.Generator(device=device).manual_seed(seed)
    gamma, latent_gamma = ((1 + 0.1 * torch.randn(n, device=device, generator=g)).bfloat16() for n in (hidden, rank))
    w = (torch.randn(heads, 2 * nope, rank, device=device, generator=g) / math.sqrt(rank)).bfloat16()
    return LatentAttention(gamma, decode_layer.random_weight4(heads * (nope + rope), hidden, group, (), device, g),
                           decode_layer.random_weight4(rank + rope, hidden, group, (), device, g), latent_gamma, w, rope, pages)
