"""The decoding operators at the ends of their ranges, against their plain 64-bit forms."""
import math

import pytest
import torch

import ops_plain as R
from sync_protocols_amd import ops
from test_gpu_ops import check_norm, check_route, dev, run_moe, run_w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


# ----------------------------------------------------------------- products
# Every sum of a group is at most 15 sum |x| s and is rounded once an element, the one of x as often; then the groups'.
@pytest.mark.parametrize("rows", [1, 5, 20, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_group", [0, 128])
def test_w4_small_elements_beside_a_large_one(rows, group, x_group):
    """One element of 448 where the weight is its zero point, 2^-5 elsewhere: what is left is the small elements' sum."""
    k, n = 256, 48
    x = torch.full((rows, k), 2.0 ** -5)
    q = torch.full((n, k), 1, dtype=torch.uint8)
    for t in range(rows):
        x[t, 17 + t % 3] = 448.0
        x[t, 140 + t % 3] = -448.0
    q[:, 17:20] = q[:, 140:143] = 15
    packed = q[:, 0::2] | q[:, 1::2] << 4
    s, z = torch.ones(n, k // group).bfloat16(), torch.full((n, k // group), 15, dtype=torch.uint8)
    x = x.to(torch.float8_e4m3fn)
    xs = torch.ones((rows, k // 128) if x_group else rows)
    got = ops.w4_linear(dev(x), ops.W4Weight(*dev(packed, s, z)), x_scale=dev(xs))
    want = x.double() @ R.w4_values(packed, s, z).t()
    tol = (2 * group + 8) * R.U * 15 * x.double().abs().sum(1, keepdim=True)
    R.close(got, want, tol + R.BF16_HALF * (want.abs() + tol), "out")


# ------------------------------------------------------------------ streams
def _fresh(nbytes):
    """The address of a block of that size that the current stream has just freed."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    at = t.data_ptr()
    del t
    return at


def test_outputs_on_another_stream_are_not_memory_that_this_one_freed():
    s = torch.cuda.Stream()
    g = R.gen(21)
    x, gamma = torch.randn(2048, 4096, generator=g).bfloat16(), torch.ones(4096).bfloat16()
    logits = torch.randn(1 << 17, 64, generator=g)
    w = ops.W4Weight(*dev(*R.make_w4(g, (), 65536, 128, 64, False)))
    x, gamma, logits = dev(x, gamma, logits)
    rows = torch.randn(64, 128, generator=g).bfloat16().to(DEV)
    torch.cuda.synchronize()
    at = _fresh(2048 * 4096 * 2)
    r = ops.add_rmsnorm(x, gamma, stream=s)
    assert r.y.data_ptr() != at and _fresh(2048 * 4096 * 2) == at
    at = _fresh(2048 * 4096)
    r8 = ops.add_rmsnorm(x, gamma, out="i8", stream=s)
    assert r8.q.data_ptr() != at
    at = _fresh((1 << 17) * 32)
    topk, weights = ops.moe_route(logits, 8, stream=s)
    assert topk.data_ptr() != at and weights.data_ptr() != at
    at = _fresh(64 * 65536 * 2)
    out = ops.w4_linear(rows, w, stream=s)
    assert out.data_ptr() != at
    s.synchronize()
    assert torch.equal(r.y, ops.add_rmsnorm(x, gamma).y) and torch.equal(out, ops.w4_linear(rows, w))


def test_outputs_of_another_stream_stay_while_this_one_uses_them():
    s = torch.cuda.Stream()
    x, gamma = torch.randn(2048, 2048, generator=R.gen(22)).bfloat16().to(DEV), torch.ones(2048, dtype=BF, device=DEV)
    want = ops.add_rmsnorm(x, gamma).y
    torch.cuda.synchronize()
    r = ops.add_rmsnorm(x, gamma, stream=s)
    at = r.y.data_ptr()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    copy = r.y.clone()
    del r                                                     # this stream has yet to read it
    with torch.cuda.stream(s):
        other = torch.zeros(2048, 2048, dtype=BF, device=DEV)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_expert_layers_of_two_streams_at_once():
    """Their workspaces are the calls' own: the first one's is freed on return, while its kernels have yet to run."""
    s = torch.cuda.Stream()
    args = [run_moe(24, 512, 384, 12, 0, 5, 64, seed=i)[1] for i in range(2)]
    want = [ops.moe_few(*a) for a in args]
    torch.cuda.synchronize()
    for _ in range(10):
        torch.cuda._sleep(1_000_000)
        a, b = ops.moe_few(*args[0]), ops.moe_few(*args[1], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_captured_step_outlives_its_layer():
    from sync_protocols_amd import decode_layer as D
    g = R.gen(31)
    a, residual = torch.randn(5, 256, generator=g).bfloat16().to(DEV), torch.randn(5, 384, generator=g).bfloat16().to(DEV)
    want = D.random_layer(384, 192, 256, 8, 8, 2, group=32, device=DEV, seed=7).step(a, residual)
    captured = D.CapturedStep(D.random_layer(384, 192, 256, 8, 8, 2, group=32, device=DEV, seed=7), 5, 256)
    captured.a.copy_(a)
    captured.residual.copy_(residual)
    for _ in range(3):
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (1 << 12, 1 << 16, 1 << 18, 1 << 20) for _ in range(8)]
        got = captured.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.y, want.y) and torch.equal(got.residual, want.residual)
        del junk


# ------------------------------------------- tiles of the expert layer's large cases
def check_moe_large(tokens, K, F, local, k, group, zero, kind, x_group, seed):
    """As run_moe, an expert at a time and with the 64-bit form on the GPU."""
    g = R.gen(seed)
    x, xs, xv = R.make_rows(g, tokens, K, kind, x_group)
    topk = torch.stack([torch.randperm(local, generator=g)[:k] for _ in range(tokens)]).int()
    weights = torch.rand(tokens, k, generator=g)
    if group:
        p1, p2 = (dev(*R.make_w4(g, (local,), a, b, group, zero)) for a, b in ((2 * F, K), (K, F)))
        w1, w2 = ops.W4Weight(*p1), ops.W4Weight(*p2)
        of = lambda p, e: R.w4_values(*(None if v is None else v[e].cpu() for v in p)).to(DEV)
        error = lambda v, p, e, w: R.w4_error(v, p[1][e], group)
    else:
        w1, w2 = p1, p2 = [(torch.randn(local, a, b, generator=g) / math.sqrt(b)).bfloat16().to(DEV) for a, b in ((2 * F, K), (K, F))]
        of = lambda p, e: p[e].double()
        error = lambda v, p, e, w: R.dense_error(v, w)
    got = ops.moe_few(dev(x), w1, w2, dev(topk), dev(weights), x_scale=dev(xs))
    topk, weights, xv = topk.to(DEV), weights.to(DEV), xv.to(DEV)
    y, tol = torch.zeros(tokens, K, dtype=torch.float64, device=DEV), torch.zeros(tokens, K, dtype=torch.float64, device=DEV)
    for e in range(local):
        t, j = torch.nonzero(topk == e, as_tuple=True)
        if not t.numel():
            continue
        a, b = of(p1, e), of(p2, e)
        gu, d, c = xv[t] @ a.t(), error(xv[t], p1, e, a), weights[t, j].double()[:, None]
        (gate, up), (dg, du) = gu.chunk(2, 1), d.chunk(2, 1)
        silu = gate * torch.sigmoid(gate)
        h = c * silu * up
        dh = c.abs() * (1.1 * dg * (up.abs() + du) + silu.abs() * du) + (2.0 ** -16 + (8 + 2 * gate.abs()) * R.U) * h.abs()      # as in R.moe
        y.index_add_(0, t, h @ b.t())
        tol.index_add_(0, t, dh @ b.abs().t() + error(h, p2, e, b))
    R.close(got, y.cpu(), (tol + R.BF16_HALF * (y.abs() + tol) + 2.0 ** -133).cpu(), "y")


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("kind,x_group", [("bf16", 0), ("i8", 0), ("i8", 128), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("tokens,k", [(16, 4), (40, 3)])
def test_moe_two_column_tiles_of_the_first_product(tokens, k, group, kind, x_group):
    """64 experts of width 2048: 4096 pairs of column tiles."""
    check_moe_large(tokens, 640, 2048, 64, k, group, group == 64, kind, x_group, tokens + group)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("tokens,F,local,k", [(64, 256, 8, 2), (64, 128, 64, 8), (63, 384, 5, 5)])
def test_moe_many_tokens_and_columns_of_the_second_product(tokens, F, local, k, group):
    """Two column tiles over 64 tokens: 64 KB of sums beside the plan."""
    check_moe_large(tokens, 4096, F, local, k, group, True, "bf16", 0, tokens + F)


# --------------------------------------------------------------------- norm
@pytest.mark.parametrize("out", ["i8", "e4m3"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("n", [256, 2048, 20096])
@pytest.mark.parametrize("top", [2.0 ** -118, 2.0 ** -121, 2.0 ** -126, 2.0 ** -133, 2.0 ** -143])
def test_norm_tiny_rows(n, out, group, top):
    """Zeros and numbers whose maximum, about 2^10 x, is too small for its reciprocal; the last are below what gamma leaves of them."""
    g = R.gen(n)
    down = 100 if top < 2.0 ** -123 else 0   # bf16's smallest numbers are 2^-133: the rest by gamma
    x = (torch.randn(4, n, generator=g).double().clamp(-2, 2) * top * 2.0 ** (down - 10)).bfloat16()
    x[:, ::3] = 0
    x[1, n // 2:] = 0
    gamma = torch.full((n,), 2.0 ** -down).bfloat16()
    got = ops.add_rmsnorm(dev(x), dev(gamma), eps=2.0 ** -20, out=out, group=group, keep_bf16=True)
    assert got.scale.isfinite().all() and got.q.float().isfinite().all()
    assert (got.q[:, ::3].float() == 0).all() and (got.q[1, n // 2:].float() == 0).all()
    check_norm(got, x, gamma, None, 2.0 ** -20, out, group)
    if top == 2.0 ** -118:                   # scales that fp32 holds in full: codes that use their range
        v = R.groups_of(got.q.float(), group).abs().amax(-1)
        assert ((v == 0) == (got.scale == 0)).all() and (v[got.scale > 0] >= 0.99 * R.TOP[out]).all()


# ------------------------------------------------------------- zero points
@pytest.mark.parametrize("zero", [16, 127, 128, 129, 200, 255])
@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 3, 33])
def test_w4_every_zero_point(rows, group, kind, zero):
    """Zero points a byte holds, 16 and more among them; the tolerance is that of sums of up to 255 |x| s instead of 15.
    int8 rows take them up to 128: a column with a larger one is NaN, the others are what they are without it."""
    k, n = 384, 40
    g = R.gen(zero + rows)
    q, s, z = R.make_w4(g, (), n, k, group, True)
    z[::2] = zero                                                     # and ordinary ones beside them
    x, xs, xv = R.make_rows(g, rows, k, kind, 0)
    got = ops.w4_linear(dev(x), ops.W4Weight(*dev(q, s, z)), x_scale=dev(xs))
    want = xv @ R.w4_values(q, s, z).t()
    if kind == "i8" and zero > 128:
        want[:, ::2] = math.nan
    tol = 255 / 15 * R.w4_error(xv, s, group)
    R.close(got, want, tol + R.BF16_HALF * (want.abs() + tol), "out")


def test_w4_int8_zero_points_are_exact():
    """Whole numbers below 2^24 throughout: only the result's rounding is left."""
    k, n = 128, 129
    q = torch.full((n, k // 2), 0xF0, dtype=torch.uint8)
    z = torch.arange(129, dtype=torch.uint8)[:, None].expand(n, 2).contiguous()      # all that int8 rows take
    x = torch.tensor([[127] * k, [-127] * k, [127, -127] * (k // 2), [-127, 126] * (k // 2)], dtype=torch.int8)
    w = ops.W4Weight(*dev(q, torch.ones(n, 2).bfloat16(), z))
    got = ops.w4_linear(dev(x), w, x_scale=torch.ones(4, device=DEV))
    assert torch.equal(got.cpu(), (x.double() @ R.w4_values(q, torch.ones(n, 2).bfloat16(), z).t()).bfloat16())


# ------------------------------------------------------------ shared memory
def test_outputs_beside_their_inputs_in_one_buffer():
    """Rows that interleave without sharing a byte are taken; moe_few may write over its own x."""
    g = R.gen(41)
    w = ops.W4Weight(*dev(*R.make_w4(g, (), 64, 128, 64, True)))
    x = torch.randn(20, 128, generator=g).bfloat16().to(DEV)
    want = ops.w4_linear(x, w)
    for first, gap in ((0, 0), (0, 8), (64, 0), (72, 8)):             # x before out in each row, or after it
        big = torch.zeros(20, 128 + 64 + gap + 8, dtype=BF, device=DEV)
        xv = big[:, first:first + 128]
        out = big[:, 128 + gap:192 + gap] if first == 0 else big[:, :64]
        xv.copy_(x)
        assert torch.equal(ops.w4_linear(xv, w, out=out), want) and torch.equal(xv, x)
    logits = torch.randn(9, 24, generator=g).to(DEV)
    topk, weights = ops.moe_route(logits, 4)
    big = torch.empty(3 * 9 * 24, device=DEV)
    big[:216] = logits.flatten()
    got = ops.moe_route(big[:216].view(9, 24), 4, topk=big[216:252].view(torch.int32).view(9, 4), weights=big[252:288].view(9, 4))
    assert torch.equal(got[0], topk) and torch.equal(got[1], weights)
    want, args = run_moe(6, 128, 64, 4, 0, 2)
    x = args[0]
    assert torch.equal(ops.moe_few(*args, out=x), want)


@pytest.mark.parametrize("shift", [0, 8, 127])
def test_w4_refuses_to_write_over_its_own_input(shift):
    from sync_protocols_amd import fg
    w = ops.W4Weight(*dev(*R.make_w4(R.gen(1), (), 128, 128, 64, False)))
    big = torch.randn(8, 256, device=DEV).bfloat16()
    before = big.clone()
    with pytest.raises(fg.FgError):
        ops.w4_linear(big[:, :128], w, out=big[:, shift:shift + 128])
    assert torch.equal(big, before)


# ------------------------------------------------------------------ autograd
def test_given_outputs_count_as_written():
    """What autograd has saved and a call then overwrites is noticed; without gradients parameters are taken."""
    g = R.gen(51)
    x, gamma = torch.randn(4, 128, generator=g).bfloat16().to(DEV), torch.nn.Parameter(torch.ones(128, dtype=BF, device=DEV))
    w = ops.W4Weight(*dev(*R.make_w4(g, (), 128, 128, 64, True)))
    buffers = dict(sum=torch.empty_like(x), y=torch.empty_like(x), q=torch.empty_like(x, dtype=torch.int8), scale=torch.empty(4, 1, device=DEV))
    before = {k: t._version for k, t in buffers.items()}
    with torch.no_grad():
        ops.add_rmsnorm(x, gamma, residual=x, out="i8", **buffers)
    assert all(t._version > before[k] for k, t in buffers.items())
    leaf = torch.randn(4, 128, device=DEV, requires_grad=True)
    held = torch.randn(4, 128, device=DEV).bfloat16()
    loss = (leaf * held).sum()
    ops.w4_linear(x, w, out=held)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        out = torch.empty(4, 128, dtype=BF, device=DEV)
    ops.w4_linear(x, w, out=out)                                      # has no version to raise
    assert torch.equal(out, held)


# --------------------------------------------------------------------- route
@pytest.mark.parametrize("experts", [2, 7, 64, 300])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_nan_comes_after_minus_infinity(experts, dtype, score):
    logits = torch.full((6, experts), -math.inf)
    logits[0, 0] = math.nan                                              # of [NaN, -inf, ..] the second is first
    logits[1, ::2] = math.nan
    logits[2, -1] = 1.0
    logits[2, 0] = math.nan
    logits[3, :-1] = math.nan
    logits[4] = math.nan
    logits[5, 1] = math.inf                                              # softmax: NaN weights
    logits = logits.to(dtype)
    k = min(experts, 6)
    for renorm in (True, False):
        check_route(ops.moe_route(dev(logits), k, score=score, renorm=renorm), logits, k, score, renorm, 1.0)
    assert ops.moe_route(dev(logits), k)[0][0, 0] == 1


# ---------------------------------------------------------- infinities and NaN
@pytest.mark.parametrize("group", [0, 32, 128])
def test_moe_an_infinity_in_x_stays_in_its_token(group):
    """With bf16 rows of 4-bit weights it gives NaN: its product and its sum are both infinite."""
    tokens = 20
    g = R.gen(61)
    x = torch.randn(tokens, 128, generator=g).bfloat16()
    topk = torch.stack([torch.randperm(6, generator=g)[:2] for _ in range(tokens)]).int()
    tw = torch.rand(tokens, 2, generator=g)
    if group:
        w1, w2 = (ops.W4Weight(*dev(*R.make_w4(g, (6,), a, b, group, True))) for a, b in ((256, 128), (128, 128)))
    else:
        w1, w2 = (torch.randn(6, a, b, generator=g).bfloat16().to(DEV) for a, b in ((256, 128), (128, 128)))
    clean = ops.moe_few(dev(x), w1, w2, *dev(topk, tw))
    x[4, 7], x[11, 100] = math.inf, math.nan
    got = ops.moe_few(dev(x), w1, w2, *dev(topk, tw))
    rest = torch.ones(tokens, dtype=torch.bool, device=DEV)
    rest[4] = rest[11] = False
    assert torch.equal(got[rest], clean[rest]) and got[11].isnan().all()
    assert got[4].isnan().all() if group else not got[4].isfinite().any()


# ---------------------------------------------------------------- largest sizes
@pytest.mark.parametrize("group", [32, 64])
def test_w4_most_rows(group):
    """FG_W4_MAX_ROWS rows: up to 65536 workgroups in the grid's second dimension."""
    rows, n, k = ops.W4_MAX_ROWS, 16, 64
    g = R.gen(71)
    q, s, z = R.make_w4(g, (), n, k, group, True)
    x = torch.randn(rows, k, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).bfloat16()
    got = ops.w4_linear(x, ops.W4Weight(*dev(q, s, z)))
    w, s = R.w4_values(q, s, z).to(DEV), s.to(DEV)
    for part, rest in zip(x.split(1 << 17), got.split(1 << 17)):
        want, tol = part.double() @ w.t(), R.w4_error(part.double(), s, group)
        assert ((rest.double() - want).abs() <= tol + R.BF16_HALF * (want.abs() + tol) + 2.0 ** -133).all()


# ---------------------------------------------------------------- e4m3 rows
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_group", [0, 128])
def test_w4_e4m3_nan_stays_in_its_row(group, x_group):
    g = R.gen(81)
    w = ops.W4Weight(*dev(*R.make_w4(g, (), 48, 384, group, True)))
    x, xs, _ = R.make_rows(g, 20, 384, "e4m3", x_group)
    clean = ops.w4_linear(dev(x), w, x_scale=dev(xs))
    x.view(torch.uint8)[3, 100], x.view(torch.uint8)[18, 383] = 0x7F, 0xFF
    got = ops.w4_linear(dev(x), w, x_scale=dev(xs))
    rest = torch.ones(20, dtype=torch.bool, device=DEV)
    rest[3] = rest[18] = False
    assert got[~rest].isnan().all() and torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("tokens", [1, 20, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_group", [0, 128])
def test_moe_small_elements_beside_a_large_one(tokens, group, x_group):
    """As the product's test of that name, through both products; the first one's tolerance is taken through the formula."""
    K, F = 256, 128
    g = R.gen(group + tokens)
    x = torch.full((tokens, K), 2.0 ** -5)
    q = torch.full((1, 2 * F, K), 1, dtype=torch.uint8)
    for t in range(tokens):
        x[t, 17 + t % 3], x[t, 140 + t % 3] = 448.0, -448.0
    q[..., 17:20] = q[..., 140:143] = 15
    w1 = q[..., 0::2] | q[..., 1::2] << 4, torch.full((1, 2 * F, K // group), 2.0 ** -6).bfloat16(), torch.full((1, 2 * F, K // group), 15, dtype=torch.uint8)
    w1[1][:, :F] *= -1                                                # gates of about +1.7, up values of -1.7
    w2 = R.make_w4(g, (1,), K, F, group, True)
    x = x.to(torch.float8_e4m3fn)
    xs = torch.ones((tokens, K // 128) if x_group else tokens)
    got = ops.moe_few(dev(x), ops.W4Weight(*dev(*w1)), ops.W4Weight(*dev(*w2)), torch.zeros(tokens, 1, dtype=torch.int32, device=DEV),
                      torch.ones(tokens, 1, device=DEV), x_scale=dev(xs))
    a, b = R.w4_values(*(v[0] for v in w1)), R.w4_values(*(v[0] for v in w2))
    gate, up = (x.double() @ a.t()).chunk(2, 1)
    d = (2 * group + 8) * R.U * 15 * x.double().abs().sum(1, keepdim=True) * 2.0 ** -6
    silu = gate * torch.sigmoid(gate)
    h = silu * up
    dh = 1.1 * d * (up.abs() + d) + silu.abs() * d + (2.0 ** -16 + (8 + 2 * gate.abs()) * R.U) * h.abs()
    y, tol = h @ b.t(), dh @ b.abs().t() + R.w4_error(h, w2[1][0], group)
    R.close(got, y, tol + R.BF16_HALF * (y.abs() + tol) + 2.0 ** -133, "y")
