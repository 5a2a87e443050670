"""The decoding operators on the GPU against their plain 64-bit forms."""
import math

import pytest
import torch

import ops_plain as R
from sync_protocols_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def dev(*ts):
    r = [None if t is None else t.to(DEV) for t in ts]
    return r if len(r) > 1 else r[0]


def wide(t, pad, shift):
    """t on the GPU as a slice of a wider tensor: rows `pad` elements longer, the first `shift` elements in."""
    big = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=DEV)
    v = big[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


# --------------------------------------------------------------------- norm
# fp32: 64 squares a thread and 24 partial sums, each rounded; mean, root, two products
NORM_U = (64 + 24 + 8) * R.U


def check_norm(r, x, gamma, res, eps, out, group):
    h, y = R.norm(x, gamma, res, eps)
    if r.sum is not None:
        R.close(r.sum, h, (R.BF16_HALF + R.U) * h.abs() * (1 + R.U) + 2.0 ** -133, "sum")
    if r.y is not None:
        R.close(r.y, y, (R.BF16_HALF * (1 + NORM_U) + NORM_U) * y.abs() + 2.0 ** -133, "y")
    if out != "bf16":
        v = R.groups_of(y, group)
        a = v.abs().amax(-1)
        R.close(r.scale, a / R.TOP[out], NORM_U * a / R.TOP[out] + 2.0 ** -149, "scale")
        s = r.scale.double().cpu()[..., None]
        got = (R.groups_of(r.q.float().double().cpu(), group) * s).flatten(1)
        step = 0.5 * s * torch.ones_like(v) if out == "i8" else torch.maximum(R.E4M3_HALF * v.abs(), 2.0 ** -10 * s)
        R.close(got, y, (step * (1 + NORM_U) + 2 * NORM_U * v.abs() + 2.0 ** -133).flatten(1), "codes")
        assert r.q.float().abs().max() <= R.TOP[out]


@pytest.mark.parametrize("rows,n", [(1, 1), (1, 7), (3, 64), (5, 127), (2, 128), (17, 5003), (4, 7168), (1030, 264), (1025, 7168), (2, 16384),
                                    (1, 65536), (2, 60001), (1024, 8)])
@pytest.mark.parametrize("out", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("res", [False, True])
def test_norm(rows, n, out, res):
    g = R.gen(rows * 7 + n)
    x, gamma = torch.randn(rows, n, generator=g).bfloat16(), (1 + 0.3 * torch.randn(n, generator=g)).bfloat16()
    r = (2 * torch.randn(rows, n, generator=g)).bfloat16() if res else None
    got = ops.add_rmsnorm(dev(x), dev(gamma), residual=dev(r), eps=1e-5, out=out, keep_bf16=res)
    assert (got.sum is not None) == res
    check_norm(got, x, gamma, r, 1e-5, out, 0)


@pytest.mark.parametrize("rows,n", [(1, 128), (3, 7168), (1100, 384), (2, 65536 - 128), (1, 2048)])
@pytest.mark.parametrize("out", ["i8", "e4m3"])
def test_norm_groups(rows, n, out):
    g = R.gen(n + rows)
    x, gamma = torch.randn(rows, n, generator=g).bfloat16(), torch.randn(n, generator=g).bfloat16()
    x[:, :128] *= 1e-3                       # a group whose numbers are much smaller
    gamma[n // 128 * 128 - 128:] = 0         # and one of zeros: scale and codes 0
    got = ops.add_rmsnorm(dev(x), dev(gamma), out=out, group=128)
    check_norm(got, x, gamma, None, 1e-6, out, 128)
    if n > 128:
        assert (got.scale[:, -1] == 0).all() and (got.q[:, -128:].float() == 0).all()


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 1), (5, 2), (16, 8)])
@pytest.mark.parametrize("n", [24, 1001, 640])
def test_norm_strides_and_alignment(pad, shift, n):
    g = R.gen(pad + n)
    x, res, gamma = (torch.randn(6, n, generator=g).bfloat16() for _ in range(3))
    gamma = gamma[0].contiguous()
    sum_, y, q = (wide(torch.zeros(6, n, dtype=t), pad, shift) for t in (BF, BF, torch.int8))
    got = ops.add_rmsnorm(wide(x, pad, shift), wide(gamma[None], pad, shift)[0], residual=wide(res, pad + 1, shift), eps=0.1, out="i8",
                          sum=sum_, y=y, q=q)
    check_norm(got, x, gamma, res, 0.1, "i8", 0)
    for t in (sum_, y, q):                   # nothing beside the rows is written
        base = t._base
        assert (base[:, :shift].float() == 0).all() and (base[:, shift + n:].float() == 0).all()


def test_norm_in_place_and_no_rows():
    g = R.gen(5)
    x, res, gamma = torch.randn(9, 512, generator=g).bfloat16(), torch.randn(9, 512, generator=g).bfloat16(), torch.ones(512).bfloat16()
    dx, dr = dev(x, res)
    got = ops.add_rmsnorm(dx, dev(gamma), residual=dr, sum=dr, y=dx)
    assert got.sum is dr and got.y is dx
    check_norm(got, x, gamma, res, 1e-6, "bf16", 0)
    none = ops.add_rmsnorm(torch.empty(0, 512, dtype=BF, device=DEV), dev(gamma), out="i8")
    assert none.q.shape == (0, 512) and none.scale.shape == (0, 1)


def test_norm_zeros_nan_and_infinity():
    x = torch.randn(5, 300, generator=R.gen(1)).bfloat16()
    x[0] = 0
    x[1, 17] = math.nan
    x[2, 299] = math.inf
    x[3, 0] = 3e38                           # its square leaves fp32: the row becomes zeros
    gamma = torch.ones(300).bfloat16()
    for out in ("i8", "e4m3"):
        got = ops.add_rmsnorm(dev(x), dev(gamma), out=out, keep_bf16=True)
        s, y = got.scale[:, 0].cpu(), got.y.cpu()
        assert s[0] == 0 and (got.q[0].float() == 0).all() and (y[0] == 0).all()
        assert y[1].isnan().all() and s[1].isnan()
        assert y[2, 299].isnan() and (y[2, :299] == 0).all() and s[2].isnan()
        assert (y[3] == 0).all() and s[3] == 0
        check_norm(ops.NormResult(None, got.y[4:], got.q[4:], got.scale[4:]), x[4:], gamma, None, 1e-6, out, 0)


# -------------------------------------------------------------------- route
def check_route(got, logits, k, score, renorm, scale):
    topk, w = R.route(logits, k, score, renorm, scale)
    assert torch.equal(got[0].cpu(), topk)
    l = torch.where(logits.isfinite(), logits.double(), 0.0)
    # exponent's argument and exponential, sums over lanes and picks, two divisions
    tol = (2 * (l.amax(1) - l.amin(1)).clamp_min(l.abs().amax(1)) + 32) * R.U
    R.close(got[1], w, tol[:, None] * w + 1e-37, "weights")


@pytest.mark.parametrize("rows,experts,k", [(1, 1, 1), (1, 64, 8), (5, 8, 8), (67, 60, 4), (3, 64, 64), (130, 256, 8), (9, 257, 6), (4, 1000, 33),
                                            (2, 1024, 64), (16, 128, 1), (7, 512, 16)])
@pytest.mark.parametrize("score,renorm,dtype", [("softmax", True, torch.float32), ("softmax", False, BF), ("sigmoid", True, BF),
                                                ("sigmoid", False, torch.float32)])
def test_route(rows, experts, k, score, renorm, dtype):
    logits = (3 * torch.randn(rows, experts, generator=R.gen(rows + experts))).to(dtype)
    check_route(ops.moe_route(dev(logits), k, score=score, renorm=renorm, scale=2.5), logits, k, score, renorm, 2.5)


@pytest.mark.parametrize("experts", [6, 64, 200])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_masks_and_nan(experts, score):
    g = R.gen(experts)
    logits = torch.randint(-2, 3, (8, experts), generator=g).float()      # mostly ties
    logits[0] = -math.inf                                                # nothing left
    logits[1, 1:] = -math.inf
    logits[2, ::2] = -math.inf
    logits[3, ::3] = math.nan
    logits[4] = 0.0
    logits[4, 1::2] = -0.0                                               # equal to +0
    logits[5] = torch.finfo(torch.float32).min
    logits[6] = math.nan
    for renorm in (True, False):
        check_route(ops.moe_route(dev(logits), 5, score=score, renorm=renorm), logits, 5, score, renorm, 1.0)


def test_route_strided_rows():
    logits = torch.randn(33, 50, generator=R.gen(2))
    check_route(ops.moe_route(wide(logits, 7, 3), 6), logits, 6, "softmax", True, 1.0)
    topk, w = ops.moe_route(torch.empty(0, 8, device=DEV), 2)
    assert topk.shape == (0, 2) and w.shape == (0, 2)


# ----------------------------------------------------------------- products
def run_w4(rows, n, k, group, zero, kind, x_group, bias=False, seed=0, pad=0):
    g = R.gen(seed + 1000 * rows + n + k)
    q, s, z = R.make_w4(g, (), n, k, group, zero)
    x, xs, xv = R.make_rows(g, rows, k, kind, x_group)
    b = torch.randn(n, generator=g).bfloat16() if bias else None
    out = wide(torch.zeros(rows, n, dtype=BF), pad, pad // 2) if pad else None
    xd = wide(x, 8 * pad, 8 * (pad // 2)) if pad else dev(x)
    got = ops.w4_linear(xd, ops.W4Weight(*dev(q, s, z)), x_scale=dev(xs), bias=dev(b), out=out)
    want = xv @ R.w4_values(q, s, z).t() + (b.double() if bias else 0.0)
    tol = R.w4_error(xv, s, group)
    R.close(got, want, tol + R.BF16_HALF * (want.abs() + tol) + 2.0 ** -133, "out")
    if pad:
        assert (out._base[:, :pad // 2] == 0).all() and (out._base[:, pad // 2 + n:] == 0).all()


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 150])
@pytest.mark.parametrize("group,kind,x_group,zero", [(128, "bf16", 0, False), (64, "i8", 0, True), (32, "e4m3", 128, True), (32, "bf16", 0, False),
                                                     (128, "i8", 128, True), (64, "e4m3", 0, False)])
def test_w4_rows(rows, group, kind, x_group, zero):
    run_w4(rows, 80, 1280, group, zero, kind, x_group)


@pytest.mark.parametrize("n", [1, 15, 16, 31, 33, 250])
@pytest.mark.parametrize("k", [32, 96, 128, 160, 1024, 4128, 10240])
def test_w4_sizes(n, k):
    for group in (32, 64, 128):
        if k % group == 0:
            run_w4(3, n, k, group, n % 2 == 0, "bf16", 0, bias=True)
            run_w4(20, n, k, group, n % 2 == 1, "i8", 0)


def test_w4_strides():
    run_w4(5, 40, 384, 64, True, "bf16", 0, pad=6)
    run_w4(18, 40, 384, 128, False, "e4m3", 128, pad=3)


def test_w4_same_bits_for_any_batch_of_the_same_tile():
    """A token's result does not depend on its neighbours, and runs repeat bit for bit."""
    g = R.gen(3)
    w = ops.W4Weight(*dev(*R.make_w4(g, (), 96, 2048, 64, True)))
    x = dev(torch.randn(16, 2048, generator=g).bfloat16())
    a = ops.w4_linear(x, w)
    assert torch.equal(a, ops.w4_linear(x, w))
    for t in (0, 7, 15):
        assert torch.equal(a[t], ops.w4_linear(x[t:t + 1], w)[0])


def test_w4_infinity_and_nan_stay_in_their_row():
    g = R.gen(4)
    w = ops.W4Weight(*dev(*R.make_w4(g, (), 48, 512, 128, False)))
    x = torch.randn(20, 512, generator=g).bfloat16()
    clean = ops.w4_linear(dev(x), w)
    x[3, 100], x[18, 511] = math.nan, math.inf
    got = ops.w4_linear(dev(x), w)
    bad = torch.zeros(20, dtype=torch.bool)
    bad[3] = bad[18] = True
    assert got[bad.to(DEV)].isnan().all() and torch.equal(got[~bad.to(DEV)], clean[~bad.to(DEV)])


# ------------------------------------------------------------- expert layer
def run_moe(tokens, K, F, local, base, k, group=0, zero=False, kind="bf16", x_group=0, topk=None, weights=None, seed=0, experts=None, pad=0):
    g = R.gen(seed + tokens + K + F + local)
    x, xs, xv = R.make_rows(g, tokens, K, kind, x_group)
    if topk is None:
        topk = torch.stack([torch.randperm(experts or local, generator=g)[:k] for _ in range(tokens)]).int()
    if weights is None:
        weights = torch.rand(tokens, k, generator=g)
    if group:
        p1, p2 = R.make_w4(g, (local,), 2 * F, K, group, zero), R.make_w4(g, (local,), K, F, group, zero)
        v1, v2, w4 = R.w4_values(*p1), R.w4_values(*p2), (p1[1], p2[1], group)
        w1, w2 = ops.W4Weight(*dev(*p1)), ops.W4Weight(*dev(*p2))
    else:
        w1, w2 = ((torch.randn(local, a, b, generator=g) / math.sqrt(b)).bfloat16() for a, b in ((2 * F, K), (K, F)))
        v1, v2, w4 = w1.double(), w2.double(), None
        w1, w2 = dev(w1, w2)
    ws = torch.full((4 * tokens * k * F,), 255, dtype=torch.uint8, device=DEV)      # NaN patterns
    out = wide(torch.zeros(tokens, K, dtype=BF), pad, pad // 2) if pad else torch.full((tokens, K), math.nan, dtype=BF, device=DEV)
    xd = wide(x, 8 * pad, 8 * (pad // 2)) if pad else dev(x)
    got = ops.moe_few(xd, w1, w2, dev(topk), dev(weights), expert_base=base, x_scale=dev(xs), out=out, workspace=ws)
    y, tol = R.moe(xv, v1, v2, topk, weights, base, w4)
    R.close(got, y, tol, "y")
    if pad:
        assert (out._base[:, :pad // 2] == 0).all() and (out._base[:, pad // 2 + K:] == 0).all()
    return got, (xd, w1, w2, dev(topk), dev(weights))


@pytest.mark.parametrize("tokens,k", [(1, 1), (1, 4), (2, 8), (16, 2), (17, 4), (40, 8), (64, 3)])
@pytest.mark.parametrize("group,kind,x_group,zero", [(0, "bf16", 0, False), (0, "e4m3", 128, False), (0, "i8", 0, False), (128, "bf16", 0, True),
                                                     (64, "i8", 0, False), (32, "e4m3", 128, True)])
def test_moe(tokens, k, group, kind, x_group, zero):
    run_moe(tokens, 384, 256, 8, 0, k, group, zero, kind, x_group)


@pytest.mark.parametrize("K,F", [(32, 32), (96, 160), (160, 96), (1056, 544), (2048, 1024)])
@pytest.mark.parametrize("group", [0, 32])
def test_moe_sizes(K, F, group):
    run_moe(5, K, F, 4, 0, 2, group, True)
    run_moe(19, K, F, 3, 0, 3, group, False, "i8")


@pytest.mark.parametrize("tokens", [1, 9, 50])
@pytest.mark.parametrize("group", [0, 64])
def test_moe_local_share(tokens, group):
    """This GPU owns 3 of 40 experts; tokens without a local pick get zeros."""
    run_moe(tokens, 192, 128, 3, 20, 6, group, experts=40)


def test_moe_no_local_pick_and_negative_picks():
    topk = torch.tensor([[-1, 9], [0, -1], [4, 5], [2147483647, -2147483648], [3, 7]], dtype=torch.int32)
    got, _ = run_moe(5, 64, 96, 4, 4, 2, topk=topk)
    assert (got[:2] == 0).all() and (got[3] == 0).all()
    got, _ = run_moe(5, 64, 96, 4, 4, 2, topk=torch.full((5, 2), -1, dtype=torch.int32))
    assert (got == 0).all()


@pytest.mark.parametrize("tokens", [16, 33, 64])
@pytest.mark.parametrize("group", [0, 128])
def test_moe_all_tokens_on_one_expert(tokens, group):
    topk = torch.full((tokens, 1), 2, dtype=torch.int32)
    run_moe(tokens, 256, 128, 5, 0, 1, group, topk=topk)


def test_moe_many_experts_and_most_picks():
    run_moe(64, 64, 32, 1024, 0, 16)
    run_moe(3, 64, 32, 700, 300, 16, experts=1024)


def test_moe_strides():
    run_moe(6, 128, 64, 4, 0, 2, pad=4)


def test_moe_same_expert_twice():
    """Picks are meant to be distinct; a repeated one counts twice, no term is lost."""
    run_moe(4, 64, 64, 4, 0, 3, topk=torch.tensor([[1, 1, 2], [0, 0, 0], [3, 2, 3], [1, 2, 3]], dtype=torch.int32))


@pytest.mark.parametrize("group", [0, 64])
def test_moe_repeats_bit_for_bit(group):
    got, args = run_moe(30, 512, 384, 12, 0, 5, group)
    first = got.clone()
    for _ in range(5):
        assert torch.equal(first, ops.moe_few(*args))


# ------------------------------------------------------- streams and graphs
def _layer(x, res, gamma, wr, w1, w2, wo, scale, out):
    r = ops.add_rmsnorm(x, gamma, residual=res, out="e4m3", group=128, keep_bf16=True)
    topk, w = ops.moe_route(r.y.float() @ wr, 3)
    y = ops.moe_few(r.q, w1, w2, topk, w, x_scale=r.scale)
    out.copy_(ops.w4_linear(y, wo))
    return out


def _layer_inputs(seed):
    g = R.gen(seed)
    T, K, F, E = 7, 256, 128, 6
    x, res = torch.randn(T, K, generator=g).bfloat16(), torch.randn(T, K, generator=g).bfloat16()
    gamma, wr = torch.ones(K).bfloat16(), torch.randn(K, E, generator=g)
    w1, w2, wo = (ops.W4Weight(*dev(*R.make_w4(g, lead, n, k, 64, True))) for lead, n, k in (((E,), 2 * F, K), ((E,), K, F), ((), 96, K)))
    return (*dev(x, res, gamma, wr), w1, w2, wo, None, torch.zeros(T, 96, dtype=BF, device=DEV))


def test_layer_on_another_stream():
    args = _layer_inputs(1)
    want = _layer(*args).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _layer(*args)
    s.synchronize()
    assert torch.equal(got, want)
    # the stream given by argument: tensors of this stream, used on that one
    x, res, gamma = args[:3]
    s.wait_stream(torch.cuda.current_stream())
    r = ops.add_rmsnorm(x, gamma, residual=res, stream=s)
    s.synchronize()
    assert torch.equal(r.y, ops.add_rmsnorm(x, gamma, residual=res).y)


def test_layer_in_a_graph():
    args = _layer_inputs(2)
    x, out = args[0], args[-1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _layer(*args)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _layer(*args)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=R.gen(50 + i)).bfloat16())
        want = _layer(*args).clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


# ------------------------------------------------ tiles, grids and distances
# Every tile of the products: rows and columns that pick it, with the types, groups and zero points.
@pytest.mark.parametrize("rows,n", [(1, 4096), (16, 4096), (9, 8192), (31, 8192), (32, 6001), (64, 8192), (63, 8177), (50, 4111), (129, 4096), (3, 8199)])
@pytest.mark.parametrize("group,kind,x_group,zero", [(128, "bf16", 0, True), (64, "i8", 0, False), (32, "e4m3", 128, True), (32, "bf16", 0, True),
                                                     (128, "i8", 128, False), (64, "e4m3", 0, True), (64, "bf16", 0, False)])
def test_w4_tiles(rows, n, group, kind, x_group, zero):
    run_w4(rows, n, 384, group, zero, kind, x_group, bias=True)


@pytest.mark.parametrize("k", [6144, 6272, 8064])
def test_w4_long_rows(k):
    """Steps in every remainder of four and of the waves, rows that share cache lines."""
    run_w4(4, 100, k + 32, 32, True, "bf16", 0)
    run_w4(16, 100, k + 64, 64, False, "i8", 0)
    run_w4(40, 100, k, 128, True, "e4m3", 128)


@pytest.mark.parametrize("zero", [0, 15])
def test_w4_extreme_codes(zero):
    """Every code against every 8-bit activation code, by exact values: no product or sum is out of its type's range."""
    k, n = 256, 32
    q = torch.full((n, k // 2), 0xFF, dtype=torch.uint8)
    q[::2] = 0
    s, z = torch.ones(n, k // 64).bfloat16(), torch.full((n, k // 64), zero, dtype=torch.uint8)
    for kind, top in (("i8", -127), ("e4m3", 448)):
        x = torch.full((17, k), top, dtype=torch.float32).to(torch.int8 if kind == "i8" else torch.float8_e4m3fn)
        got = ops.w4_linear(dev(x), ops.W4Weight(*dev(q, s, z)), x_scale=torch.ones(17, device=DEV))
        want = x.double() @ R.w4_values(q, s, z).t()
        R.close(got, want, R.BF16_HALF * want.abs(), kind)


def test_w4_rows_far_apart():
    """Rows a little less than 64 MiB apart, 40 of them: distances beyond 31 bits."""
    g = R.gen(8)
    w = R.make_w4(g, (), 48, 256, 64, True)
    x = torch.randn(40, 256, generator=g).bfloat16()
    big = torch.empty(40 * ((1 << 25) - 8), dtype=BF, device=DEV).view(40, -1)
    big[:, :256] = x.to(DEV)
    want = ops.w4_linear(dev(x), ops.W4Weight(*dev(*w)))
    assert torch.equal(ops.w4_linear(big[:, :256], ops.W4Weight(*dev(*w))), want)


def test_norm_and_route_with_grids_of_two_dimensions():
    rows = 5_000_003
    x = torch.randn(rows, 8, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    gamma = torch.ones(8, dtype=BF, device=DEV)
    y = ops.add_rmsnorm(x, gamma).y
    for at in (0, 4 << 20, (4 << 20) - 1, rows - 1):
        check_norm(ops.NormResult(None, y[at:at + 1], None, None), x[at:at + 1].cpu(), gamma.cpu(), None, 1e-6, "bf16", 0)
    h = x.float()
    want = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    assert ((y.float() - want).abs() <= (R.BF16_HALF + 2 * NORM_U) * want.abs()).all()
    rows = 17_000_001
    l = torch.randint(-9, 10, (rows, 4), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV, dtype=torch.int8).to(BF)
    topk, w = ops.moe_route(l, 1, score="sigmoid", renorm=True)
    want = 4 * l.float() - torch.arange(4, device=DEV)                   # ties: lowest index
    assert torch.equal(topk[:, 0].long(), want.argmax(1)) and (w == 1).all()


@pytest.mark.parametrize("n", [64, 130, 512])
def test_norm_many_short_rows(n):
    """A wave a row, four rows a workgroup, the last one not full; and outputs larger than the caches."""
    for rows in (1, 3, 1025, 40_001):
        g = R.gen(rows)
        x, res, gamma = torch.randn(rows, n, generator=g).bfloat16(), torch.randn(rows, n, generator=g).bfloat16(), torch.randn(n, generator=g).bfloat16()
        check_norm(ops.add_rmsnorm(dev(x), dev(gamma), residual=dev(res), out="i8", keep_bf16=True), x, gamma, res, 1e-6, "i8", 0)


def test_norm_infinite_group_leaves_the_others():
    x = torch.randn(3, 384, generator=R.gen(3)).bfloat16()
    gamma = torch.ones(384).bfloat16()
    gamma[130] = math.inf                                                # its group alone has an infinite scale
    got = ops.add_rmsnorm(dev(x), dev(gamma), out="e4m3", group=128)
    assert got.scale[:, 1].isinf().all()
    gamma[130] = 1
    want = ops.add_rmsnorm(dev(x), dev(gamma), out="e4m3", group=128)
    for c in (0, 2):
        assert torch.equal(got.scale[:, c], want.scale[:, c])
        assert torch.equal(got.q[:, 128 * c:128 * c + 128].float(), want.q[:, 128 * c:128 * c + 128].float())


@pytest.mark.parametrize("experts", [16, 17, 32, 33, 129, 256, 512, 513])
def test_route_lane_shapes(experts):
    for dtype in (torch.float32, BF):
        logits = (4 * torch.randn(19, experts, generator=R.gen(experts))).to(dtype)
        logits[::3] = logits[::3].round()                                # equal ones
        k = min(experts, 40)
        check_route(ops.moe_route(dev(logits), k), logits, k, "softmax", True, 1.0)
        check_route(ops.moe_route(wide(logits, 3, 1), k, score="sigmoid"), logits, k, "sigmoid", True, 1.0)


# Entries of every size in the second product: 1 to 64 picks of an expert, first rows at odd and even places.
@pytest.mark.parametrize("tokens", [8, 9, 16, 17, 64])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_moe_uneven_experts(tokens, group):
    topk = torch.stack([torch.tensor([0, 1 + t % 3, 4 + t % 5]) for t in range(tokens)]).int()
    topk[::4, 2] = -1
    run_moe(tokens, 256, 384, 9, 0, 3, group, True, "bf16" if group % 64 else "i8", topk=topk)


def test_moe_wide():
    """Two column tiles in both products, 16 and more tokens."""
    run_moe(16, 4096, 128, 3, 0, 2, 0)
    run_moe(33, 4128, 96, 3, 0, 1, 32, True)
    run_moe(2, 4224, 256, 3, 0, 2, 128, False, "e4m3", 128)
    run_moe(20, 256, 4096, 8, 0, 2, 64, True, "i8")


def test_moe_weights_of_zero_infinity_and_nan():
    g = R.gen(11)
    x = torch.randn(6, 64, generator=g).bfloat16()
    w1, w2 = torch.randn(4, 64, 64, generator=g).bfloat16(), torch.randn(4, 64, 32, generator=g).bfloat16()
    topk = torch.tensor([[0, 1], [1, 2], [2, 3], [3, 0], [0, 2], [1, 3]], dtype=torch.int32)
    tw = torch.rand(6, 2, generator=g)
    clean = ops.moe_few(*dev(x, w1, w2, topk, tw))
    tw[1, 0] = 0
    x[3, 5], tw[4, 1] = math.inf, math.nan
    got = ops.moe_few(*dev(x, w1, w2, topk, tw))
    for t in (0, 2, 5):
        assert torch.equal(got[t], clean[t])
    assert got[4].isnan().all() and not got[3].isfinite().any() and got[1].isfinite().all()


@pytest.mark.parametrize("group", [0, 64])
def test_moe_more_than_32_picks_repeat_bit_for_bit(group):
    topk = torch.stack([torch.tensor([2, t % 2, 3 + t % 4]) for t in range(64)]).int()
    got, args = run_moe(64, 320, 192, 8, 0, 3, group, topk=topk)
    first = got.clone()
    for _ in range(5):
        assert torch.equal(first, ops.moe_few(*args))


@pytest.mark.parametrize("k", [32, 96, 128, 480, 2048, 6176, 8192, 16384, 16416])
@pytest.mark.parametrize("n", [1, 47, 4500])
def test_w4_one_row(n, k):
    """One bf16 row, in LDS up to 16384 elements; both tiles, ends of rows inside a step."""
    for group in (32, 64, 128):
        if k % group == 0:
            run_w4(1, n, k, group, n % 2 == 1, "bf16", 0, bias=n == 47, pad=8 if k == 480 else 0)


def test_w4_one_row_has_the_bits_it_has_among_others():
    g = R.gen(11)
    for n, k, group in ((48, 480, 32), (4500, 1088, 64), (80, 8192, 128)):
        w = ops.W4Weight(*dev(*R.make_w4(g, (), n, k, group, True)))
        x = torch.randn(5, k, generator=g).bfloat16()
        x[4, k - 1] = math.inf
        x = dev(x)
        many = ops.w4_linear(x, w)
        for t in range(4):
            assert torch.equal(ops.w4_linear(x[t:t + 1], w), many[t:t + 1])
        assert not ops.w4_linear(x[4:], w).isfinite().any()
