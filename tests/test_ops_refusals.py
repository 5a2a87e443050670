"""Refusals of the decoding operators, without a GPU: the C entries return
FG_EINVAL before they launch anything, and the binding raises fg.FgError."""
import ctypes as C

import pytest
import torch

from sync_protocols_amd import fg, ops

P = 4096      # stands for an aligned device pointer; no call here gets as far as using it


def _norm(**kw):
    a = dict(x=P, ldx=64, res=None, ldr=0, gamma=P, eps=1e-6, sum=None, lds=0, y=P, ldy=64, q=None, ldq=0, qt=0, qg=0, qs=None,
             rows=2, n=64)
    a.update(kw)
    return fg.load_library().fg_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(gamma=None), dict(y=None), dict(ldx=63), dict(ldy=63), dict(res=P, ldr=8), dict(sum=P, lds=63), dict(rows=-1),
    dict(n=0), dict(n=65537, ldx=65537, ldy=65537), dict(eps=-1.0), dict(eps=float("nan")), dict(x=P + 1), dict(gamma=P + 1),
    dict(q=P, ldq=64, qt=1), dict(q=P, ldq=64, qt=0, qs=P), dict(q=P, ldq=63, qt=1, qs=P), dict(q=P, ldq=64, qt=1, qs=P, qg=64),
    dict(q=P, ldq=64, qt=1, qs=P, qg=128), dict(q=P, ldq=64, qt=2, qs=P + 2), dict(rows=1 << 31)])
def test_norm_refuses(kw):
    assert _norm(**kw) == fg.EINVAL


def _route(**kw):
    a = dict(l=P, ld=64, t=ops.F32, rows=2, e=64, k=8, score=0, renorm=1, scale=1.0, topk=P, w=P)
    a.update(kw)
    return fg.load_library().fg_moe_route(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(l=None), dict(topk=None), dict(w=None), dict(ld=63), dict(t=1), dict(rows=-1), dict(e=0), dict(e=1025, ld=1025),
                                dict(k=0), dict(k=65, e=128, ld=128), dict(k=9, e=8), dict(score=2), dict(l=P + 2), dict(topk=P + 2)])
def test_route_refuses(kw):
    assert _route(**kw) == fg.EINVAL


def _w4(**kw):
    a = dict(x=P, ldx=256, t=0, xs=None, xg=0, w=P, s=P, z=None, g=128, b=None, out=P, ldo=32, rows=2, n=32, k=256)
    a.update(kw)
    return fg.load_library().fg_w4_linear(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(s=None), dict(out=None), dict(ldx=255), dict(ldx=257), dict(ldo=31), dict(g=16), dict(g=96), dict(k=192),
    dict(k=0), dict(n=0), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(x=P + 2), dict(w=P + 8), dict(out=P + 1), dict(b=P + 1), dict(t=3), dict(t=1),
    dict(xs=P), dict(t=1, xs=P, xg=64), dict(t=1, xs=P, xg=128, k=192, g=64, ldx=192), dict(t=1, xs=P, x=P + 4)])
def test_w4_refuses(kw):
    assert _w4(**kw) == fg.EINVAL


def _moe(**kw):
    a = dict(x=P, ldx=256, t=0, xs=None, xg=0, w1=P, s1=None, z1=None, w2=P, s2=None, z2=None, g=0, topk=P, w=P, tokens=2, k=2, base=0,
             e=4, K=256, F=64, ws=P, wsb=4 * 2 * 2 * 64, y=P, ldy=256)
    a.update(kw)
    return fg.load_library().fg_moe_few(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w1=None), dict(w2=None), dict(topk=None), dict(w=None), dict(ws=None), dict(y=None), dict(tokens=65), dict(tokens=-1),
    dict(k=0), dict(k=17), dict(base=-1), dict(e=0), dict(e=1025), dict(K=240), dict(F=40), dict(ldy=255), dict(wsb=4 * 2 * 2 * 64 - 1),
    dict(s1=P), dict(z2=P), dict(g=128, s1=P, s2=P), dict(g=64, s1=P), dict(g=16, s1=P, s2=P), dict(w1=P + 8), dict(ws=P + 8), dict(topk=P + 2),
    dict(t=2), dict(t=2, xs=P, xg=32)])
def test_moe_refuses(kw):
    assert _moe(**kw) == fg.EINVAL


def test_moe_workspace_size():
    out = C.c_int64(0)
    f = fg.load_library().fg_moe_few_bytes
    assert f(64, 16, 2048, C.byref(out)) == fg.OK and out.value == 4 * 64 * 16 * 2048
    assert ops.moe_few_bytes(3, 2, 96) == 4 * 3 * 2 * 96
    for bad in ((65, 1, 32), (-1, 1, 32), (1, 0, 32), (1, 17, 32), (1, 1, 0)):
        assert f(*bad, C.byref(out)) == fg.EINVAL
    assert f(1, 1, 32, None) == fg.EINVAL


def test_no_rows_launch_nothing():
    assert _norm(rows=0, x=None, y=P) == fg.OK
    assert _route(rows=0, l=None) == fg.OK
    assert _w4(rows=0, x=None) == fg.OK
    assert _moe(tokens=0, x=None) == fg.OK


def test_limits_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fg.h")).read()
    defs = {k: int(v) for k, v in re.findall(r"^#define FG_(\w+) (\d+)", src, re.M)}
    for name in ("NORM_MAX_N", "W4_MAX_ROWS", "MOE_FEW_TOKENS", "MOE_FEW_TOPK", "MOE_FEW_EXPERTS"):
        assert getattr(ops, name) == defs[name], name
    for name, val in re.findall(r"FG_(BF16|I8|E4M3|F32|SCORE_SOFTMAX|SCORE_SIGMOID) = (\d+)", src):
        assert getattr(ops, name) == int(val), name


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


W = ops.W4Weight(_u8(32, 128), _bf(32, 2))


@pytest.mark.parametrize("call", [
    lambda: ops.add_rmsnorm(_bf(2, 8).float(), _bf(8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(7)),
    lambda: ops.add_rmsnorm(_bf(8), _bf(8)),
    lambda: ops.add_rmsnorm(_bf(8, 2).t(), _bf(8)),
    lambda: ops.add_rmsnorm(_bf(1, 8).expand(2, 8), _bf(8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), residual=_bf(1, 8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), out="fp4"),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), out="i8", group=128),
    lambda: ops.add_rmsnorm(_bf(2, 128), _bf(128), group=128),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), q=_bf(2, 8)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8), y=_bf(2, 7)),
    lambda: ops.add_rmsnorm(_bf(2, 8), _bf(8)),                       # not on a GPU
    lambda: ops.moe_route(_bf(2, 8).half(), 2),
    lambda: ops.moe_route(_bf(2, 8), 9),
    lambda: ops.moe_route(_bf(2, 8), 2, score="relu"),
    lambda: ops.moe_route(_bf(2, 8), 2, topk=torch.zeros(2, 2, dtype=torch.int64)),
    lambda: ops.moe_route(_bf(2, 8), 2),
    lambda: ops.w4_linear(_bf(2, 128), W),
    lambda: ops.w4_linear(_bf(2, 256), W, x_scale=torch.ones(2)),
    lambda: ops.w4_linear(_bf(2, 256).to(torch.int8), W),
    lambda: ops.w4_linear(_bf(2, 256).to(torch.int8), W, x_scale=torch.ones(3)),
    lambda: ops.w4_linear(_bf(2, 256), ops.W4Weight(W.q, _bf(32, 3))),
    lambda: ops.w4_linear(_bf(2, 256), ops.W4Weight(W.q, W.scale, _u8(32, 1))),
    lambda: ops.w4_linear(_bf(2, 256), ops.W4Weight(W.q[:, ::2], W.scale)),
    lambda: ops.w4_linear(_bf(2, 256), W, bias=_bf(31)),
    lambda: ops.w4_linear(_bf(2, 256), W),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), W, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 32, 64), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), torch.zeros(2, 2, dtype=torch.int64), torch.zeros(2, 2)),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 3)),
    lambda: ops.moe_few(_bf(65, 64), _bf(4, 64, 64), _bf(4, 64, 32), torch.zeros(65, 2, dtype=torch.int32), torch.zeros(65, 2)),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)),
])
def test_binding_refuses(call):
    with pytest.raises(fg.FgError) as e:
        call()
    assert e.value.code == fg.EINVAL


@pytest.mark.parametrize("kw", [dict(n=(1 << 24) + 1, ldo=(1 << 24) + 1), dict(k=(1 << 24) + 128, ldx=(1 << 24) + 128), dict(ldx=1 << 25),
                                dict(ldx=1 << 26, t=1, xs=P)])
def test_w4_refuses_what_its_distances_do_not_reach(kw):
    assert _w4(**kw) == fg.EINVAL


@pytest.mark.parametrize("kw", [dict(K=(1 << 24) + 32, ldx=(1 << 24) + 32, ldy=(1 << 24) + 32), dict(F=(1 << 24) + 32, wsb=1 << 40), dict(ldx=1 << 25),
                                dict(K=32768, ldx=32768, ldy=32768, F=65536, wsb=1 << 40),
                                dict(K=65536, ldx=65536, ldy=65536, F=1 << 17, wsb=1 << 40, g=64, s1=P, s2=P),
                                dict(F=1 << 20, e=1024, wsb=1 << 40)])
def test_moe_refuses_what_its_distances_and_grid_do_not_reach(kw):
    assert _moe(**kw) == fg.EINVAL


def test_limits_of_sizes_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fg.h")).read()
    defs = {k: int(v) for k, v in re.findall(r"^#define FG_(\w+) (\d+)", src, re.M)}
    assert ops.FEW_MAX_SIZE == defs["FEW_MAX_SIZE"] and ops.FEW_MAX_ROW_BYTES == defs["FEW_MAX_ROW_BYTES"]


@pytest.mark.parametrize("call", [
    lambda: ops.add_rmsnorm(None, _bf(8)),
    lambda: ops.add_rmsnorm([1.0], _bf(8)),
    lambda: ops.moe_route(_bf(2, 8), "2"),
    lambda: ops.moe_route(_bf(2, 8), 2.5),
    lambda: ops.w4_linear(_bf(2, 256), W, out=3),
    lambda: ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), torch.zeros(2, 2, dtype=torch.int32), None),
])
def test_binding_refuses_other_types(call):
    with pytest.raises(TypeError):
        call()


def test_binding_refuses_a_base_beyond_int32():
    with pytest.raises(fg.FgError):
        ops.moe_few(_bf(2, 64), _bf(4, 64, 64), _bf(4, 64, 32), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), expert_base=1 << 40)
