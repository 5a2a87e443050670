"""The attention operators as they are used together: pages, projections, cache, attention
and the expert half, step after step, against float32; graphs; streams."""
import math
import random

import pytest
import torch

from sync_protocols_amd import attention_layer as L
from sync_protocols_amd import decode_layer as D
from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def norm(x, gamma, eps=1e-6):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.float()


def plain_paged(layer, history):
    """Attention output of the last token of one request, whose inputs so far are `history` [n, hidden], in float32."""
    n = history.shape[0]
    qkv = (norm(history, layer.gamma) @ D.dequantise(layer.wqkv).t()).unflatten(1, (-1, layer.dim))
    qk = L.turn(qkv[:, :layer.heads + layer.kv], torch.arange(n, device=DEV))
    q, k, v = qk[-1, :layer.heads], qk[:, layer.heads:], qkv[:, layer.heads + layer.kv:]
    group = layer.heads // layer.kv
    s = torch.stack([k[:, h // group] @ q[h] for h in range(layer.heads)]) / math.sqrt(layer.dim)
    p = torch.softmax(s, -1)
    return torch.stack([p[h] @ v[:, h // group] for h in range(layer.heads)]).flatten()


def plain_latent(layer, history):
    n = history.shape[0]
    x = norm(history, layer.gamma)
    q = (x @ D.dequantise(layer.wq).t()).unflatten(1, (layer.heads, -1))
    row = x @ D.dequantise(layer.wc).t()
    c = norm(row[:, :layer.rank], layer.latent_gamma)
    r = L.turn(row[:, None, layer.rank:], torch.arange(n, device=DEV))[:, 0]
    rot = L.turn(q[..., layer.nope:], torch.arange(n, device=DEV))
    w = layer.w.float()
    out = []
    for h in range(layer.heads):
        s = ((c @ w[h, :layer.nope].t()) @ q[-1, h, :layer.nope] + r @ rot[-1, h]) / math.sqrt(layer.nope + layer.rope)
        out.append(torch.softmax(s, -1) @ (c @ w[h, layer.nope:].t()))
    return torch.cat(out)


# Relative to the norm of the output, in the mean: bf16 roundings (2^-8 / sqrt(3) each) of the normed input, q, k, v, weights and
# result, 8-bit rows 2^-4 / sqrt(3) of keys (a score's error times the spread of the values) and of values.
@pytest.mark.parametrize("kind,tol", [("paged", 0.02), ("paged8", 0.10), ("latent", 0.02)])
def test_steps(kind, tol):
    rng = random.Random(1)
    hidden, batch, page = 256, 6, 16
    pages = L.Pages(batch, 4, 18, page, DEV)
    layer = (L.random_latent(hidden, 4, 256, 32, 64, pages, group=64) if kind == "latent" else
             L.random_paged(hidden, 4, 2, 64, pages, group=64, e4m3=kind == "paged8"))
    plain = plain_latent if kind == "latent" else plain_paged
    g = torch.Generator(device=DEV).manual_seed(3)
    history = [torch.zeros(0, hidden, dtype=BF, device=DEV) for _ in range(batch)]
    checked = 0
    for step in range(45):
        add = [rng.choice([1, 1, 1, 1, 0, -1]) if step % 9 == 8 else 1 for _ in range(batch)]
        before = pages.lens.tolist()
        x = torch.randn(batch, hidden, device=DEV, generator=g).to(BF)
        p = pages.step(torch.tensor(add, dtype=torch.int32, device=DEV), batch)
        starts, lens = p.starts.tolist(), pages.lens.tolist()
        at = torch.tensor([min(s, batch - 1) for s in starts[:-1]], device=DEV)
        served = torch.tensor([b > a for a, b in zip(starts, starts[1:])], device=DEV)
        got = layer.step(x, torch.where(served, p.slots[at], -1), torch.where(served, p.positions[at], 0))
        for b in range(batch):
            if add[b] < 0:
                history[b] = history[b][:0]
            elif lens[b] > before[b]:
                history[b] = torch.cat((history[b], x[b:b + 1]))
                want = plain(layer, history[b])
                assert (got[b].float() - want).norm() <= tol * want.norm(), (step, b)
                checked += 1
            assert lens[b] == history[b].shape[0]
    assert checked > 150


def test_prompt_then_steps():
    hidden, counts, page = 256, [37, 0, 80], 16
    pages = L.Pages(3, 8, 30, page, DEV)
    layer = L.random_latent(hidden, 4, 512, 64, 128, pages, group=64)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(sum(counts), hidden, device=DEV, generator=g).to(BF)
    p = pages.step(torch.tensor(counts, dtype=torch.int32, device=DEV), sum(counts))
    got = layer.prompt(x, p.slots, p.positions, p.starts)
    history = list(x.split(counts))
    for i in (0, 1, 36, 37, 60, 116):
        own = history[0][:i + 1] if i < 37 else history[2][:i - 37 + 1]
        want = plain_latent(layer, own)
        assert (got[i].float() - want).norm() <= 0.02 * want.norm(), i
    for _ in range(3):
        y = torch.randn(3, hidden, device=DEV, generator=g).to(BF)
        p = pages.step(torch.ones(3, dtype=torch.int32, device=DEV), 3)
        got = layer.step(y, p.slots, p.positions)
        for b in range(3):
            history[b] = torch.cat((history[b], y[b:b + 1]))
            want = plain_latent(layer, history[b])
            assert (got[b].float() - want).norm() <= 0.02 * want.norm()


@pytest.mark.parametrize("kind", ["paged", "latent"])
def test_captured_steps_replay(kind):
    """The whole layer as a graph, pages moving on by themselves, against the same steps call by call."""
    hidden, batch = 256, 5

    def build():
        pages = L.Pages(batch, 4, 14, 16, DEV)
        attention = (L.random_paged(hidden, 4, 2, 64, pages, group=64, e4m3=True, seed=2) if kind == "paged" else
                     L.random_latent(hidden, 4, 256, 32, 64, pages, group=64, seed=2))
        return attention, D.random_layer(hidden, 128, 256, 8, 8, 2, group=32, device=DEV, seed=4)

    attention, experts = build()
    captured = L.CapturedDecode(*build(), batch)
    rng = random.Random(2)
    g = torch.Generator(device=DEV).manual_seed(7)
    for step in range(40):
        add = torch.tensor([rng.choice([1, 1, 1, 0, -1]) if step % 7 == 6 else 1 for _ in range(batch)], dtype=torch.int32, device=DEV)
        x = torch.randn(batch, hidden, device=DEV, generator=g).to(BF)
        want = L.decode_step(attention, experts, x, add)
        captured.x.copy_(x)
        captured.add.copy_(add)
        got = captured.replay()
        torch.cuda.synchronize()
        assert torch.equal(attention.pages.lens, captured.attention.pages.lens) and torch.equal(attention.pages.ends, captured.attention.pages.ends)
        live = attention.pages.lens > 0
        assert torch.equal(got.y[live], want.y[live]), step


@pytest.mark.parametrize("kind", ["paged", "latent"])
def test_command(kind, capsys):
    D.main(["--attention", kind, "--context", "100", "--tokens", "3", "--hidden", "256", "--width", "128", "--heads", "512", "--experts", "8", "--local", "8",
            "--top-k", "2", "--repeat", "2"])
    assert "graph equals calls: True" in capsys.readouterr().out


# ------------------------------------------------------------------ streams
def attention_calls(seed):
    """One call of every operator, with its inputs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, page = 40, 16
    k, v = (torch.randn(n, page, 2, 128, generator=g, device=DEV).to(BF) for _ in range(2))
    cache = torch.randn(n, page, 576, generator=g, device=DEV).to(BF)
    table = torch.randperm(n, generator=g, device=DEV).to(torch.int32).view(2, 20)
    lens = torch.tensor([320, 290], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 8, 128, generator=g, device=DEV).to(BF)
    ql = torch.randn(2, 20, 192, generator=g, device=DEV).to(BF)
    w = (torch.randn(20, 256, 512, generator=g, device=DEV) / 22).to(BF)
    qp = torch.randn(300, 20, 192, generator=g, device=DEV).to(BF)
    lat = torch.randn(300, 576, generator=g, device=DEV).to(BF)
    starts = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    ring, ends, add = torch.arange(64, dtype=torch.int32, device=DEV), torch.tensor([3, 60], device=DEV), torch.tensor([5, 40], dtype=torch.int32, device=DEV)
    wide = torch.full((2, 32), -1, dtype=torch.int32, device=DEV)
    wide[:, :20] = table
    return [lambda **kw: ops.paged_attention(q, k, v, table, lens, lse=True, **kw), lambda **kw: ops.latent_attention(ql, w, cache, table, lens, nope=128, lse=True, **kw),
            lambda **kw: ops.latent_prompt(qp, lat, w, starts, nope=128, lse=True, **kw),
            lambda **kw: tuple(ops.page_step(lens, add, wide.clone(), ring, ends, page=page, tokens=50, **kw))]


def test_two_streams_at_once():
    """Their workspaces are the calls' own: the first one's is freed on return, while its kernels have yet to run."""
    s = torch.cuda.Stream()
    first, second = attention_calls(1), attention_calls(2)
    want = [(f(), h()) for f, h in zip(first[:3], second[:3])]
    torch.cuda.synchronize()
    for _ in range(5):
        for (a, b), f, h in zip(want, first, second):
            torch.cuda._sleep(1_000_000)
            x, y = f(), h(stream=s)
            torch.cuda.synchronize()
            assert all(torch.equal(i, j) for i, j in zip((*x, *y), (*a, *b)))


def test_graphs_that_share_a_workspace_and_runs_that_repeat():
    calls = attention_calls(3)
    need = max(ops.paged_attention_bytes(2, 2, 4, 128), ops.latent_attention_bytes(2, 20, 512), ops.latent_prompt_bytes(300, 20, 128))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    want = [f() for f in calls]
    side = torch.cuda.Stream()
    graphs = []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f in calls:
            f()
    torch.cuda.current_stream().wait_stream(side)
    for f, kw in zip(calls, [dict(workspace=ws)] * 3 + [{}]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f(**kw)
        graphs.append((graph, out))
    for _ in range(4):
        for (graph, out), w in zip(graphs, want):
            for t in out:
                t.fill_(3)
            graph.replay()
            again = calls[0]()                       # the program's own work between replays
            torch.cuda.synchronize()
            assert all(torch.equal(i, j) for i, j in zip(out, w))
            assert torch.equal(again[0], want[0][0])


def test_append_on_another_stream_marks_what_it_writes():
    s = torch.cuda.Stream()
    cache = torch.zeros(4, 16, 2, 64, dtype=BF, device=DEV)
    x, slots = torch.randn(9, 2, 64, device=DEV).to(BF), torch.randperm(64, device=DEV)[:9]
    torch.cuda.synchronize()
    version = cache._version
    ops.kv_append(x, cache, slots, stream=s)
    s.synchronize()
    assert cache._version > version and torch.equal(cache.flatten(0, 1)[slots], x)
