"""Refusals of the attention half's operators, without a GPU: the C entries return
FG_EINVAL before they launch anything, and the binding raises fg.FgError."""
import ctypes as C
import os
import re

import pytest
import torch

from sync_protocols_amd import fg, ops

P = 1 << 20                 # stands for an aligned device pointer; no call here gets as far as using it
GAP = 1 << 30
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_and_library_agree():
    src = open(os.path.join(ROOT, "include", "fg_attention.h")).read()
    names = re.findall(r"^fg_status\s+(fg_\w+)\(", src, re.M)
    assert sorted(names) == sorted(fg.ATTENTION_EXPORTS)
    lib = fg.load_library()
    for n in names:
        assert hasattr(lib, n), n
    defs = {k: int(v) for k, v in re.findall(r"^#define FG_(\w+) (\d+)", src, re.M)}
    assert (ops.ATTN_MAX_BATCH, ops.ATTN_MAX_HEADS, ops.APPEND_MAX_DIM) == (defs["ATTN_MAX_BATCH"], defs["ATTN_MAX_HEADS"], defs["APPEND_MAX_DIM"])


def test_structures_match_the_header(tmp_path):
    import subprocess
    lines = []
    for c, py in (("fg_append_t", fg.FgAppend), ("fg_pages_t", fg.FgPages), ("fg_cache_t", fg.FgCache)):
        lines.append(f'printf("%zu ", sizeof({c}));')
        lines += [f'printf("%zu ", offsetof({c}, {n}));' for n, _ in py._fields_]
    src = tmp_path / "l.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include <fg_attention.h>\nint main() {" + "\n".join(lines) + "}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src), "-o", str(exe)], check=True, capture_output=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for py in (fg.FgAppend, fg.FgPages, fg.FgCache):
        want += [C.sizeof(py)] + [getattr(py, n).offset for n, _ in py._fields_]
    assert got == want


# --------------------------------------------------------------- page_step
def _pages(**kw):
    a = dict(lens=P, add=P + GAP, batch=4, table=P + 2 * GAP, ldt=8, width=8, ring=P + 3 * GAP, ends=P + 4 * GAP, n_pages=32, page=16, lens_out=P + 5 * GAP,
             ends_out=P + 6 * GAP, starts=P + 7 * GAP, slots=P + 8 * GAP, positions=P + 9 * GAP, tokens=9)
    a.update(kw)
    return fg.load_library().fg_page_step(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(lens=None), dict(add=None), dict(table=None), dict(ring=None), dict(ends=None), dict(lens_out=None), dict(ends_out=None), dict(starts=None),
    dict(slots=None), dict(positions=None), dict(batch=-1), dict(ldt=7), dict(width=0), dict(n_pages=0), dict(page=0), dict(tokens=-1), dict(lens=P + 2),
    dict(ends=P + 4 * GAP + 4), dict(slots=P + 8 * GAP + 4), dict(width=1 << 27, ldt=1 << 27), dict(lens_out=P + 4), dict(starts=P), dict(slots=P - 64),
    dict(ring=P + 2 * GAP + 4 * 31), dict(positions=P + 8 * GAP + 64), dict(ends_out=P + 4 * GAP + 8), dict(table=P + GAP), dict(lens_out=P + GAP)])
def test_page_step_refuses(kw):
    assert _pages(**kw) == fg.EINVAL


# ------------------------------------------------------------------ append
def _append(keys=None, values=None, **kw):
    k = dict(x=P, x_row=256, x_head=64, cache=P + GAP, page_stride=16 * 256, row_stride=256, head_stride=64, scale=None)
    v = dict(k, x=P + 2 * GAP, cache=P + 3 * GAP)
    k.update(keys or {})
    v.update(values or {})
    a = dict(t=ops.BF16, slots=P + 4 * GAP, rows=3, heads=4, dim=64, n_pages=8, page=16)
    a.update(kw)
    return fg.load_library().fg_kv_append(C.byref(fg.FgAppend(*k.values())), None if values is False else C.byref(fg.FgAppend(*v.values())), *a.values(), None)


@pytest.mark.parametrize("keys,values,kw", [
    (dict(x=None), {}, {}), (dict(cache=None), {}, {}), ({}, dict(x=None), {}), ({}, {}, dict(slots=None)), ({}, {}, dict(t=1)), ({}, {}, dict(t=2)),
    (dict(scale=P + 5 * GAP), {}, {}), ({}, {}, dict(rows=-1)), ({}, {}, dict(heads=0)), ({}, {}, dict(dim=63)), ({}, {}, dict(dim=0)),
    ({}, {}, dict(n_pages=0)), ({}, {}, dict(page=0)), (dict(x=P + 8), {}, {}), (dict(cache=P + GAP + 8), {}, {}), (dict(x_row=4), {}, {}),
    (dict(row_stride=252), {}, {}), (dict(head_stride=56), {}, {}), (dict(row_stride=248), {}, {}), (dict(page_stride=256), {}, {}),
    (dict(page_stride=-4096), {}, {}), (dict(x=P + GAP), {}, {}), ({}, dict(x=P + GAP + 64), {}), ({}, {}, dict(slots=P + GAP)), ({}, dict(cache=P + GAP), {}),
    (dict(scale=P + 5 * GAP), dict(scale=P + 5 * GAP), dict(t=2)), (dict(scale=P), dict(scale=P + 5 * GAP), dict(t=2)), ({}, {}, dict(slots=P + 4 * GAP + 4))])
def test_append_refuses(keys, values, kw):
    assert _append(keys, values, **kw) == fg.EINVAL


# --------------------------------------------------------------- attention
def _cache(at, **kw):
    a = dict(data=at, page_stride=16 * 256, row_stride=256, head_stride=64, scale=None)
    a.update(kw)
    return fg.FgCache(*a.values())


def _table(**kw):
    a = dict(table=P + 3 * GAP, ldt=8, width=8, lens=P + 4 * GAP, batch=2, n_pages=8, page=16)
    a.update(kw)
    return fg.FgPages(*a.values())


def _paged(**kw):
    a = dict(q=P, q_b=8 * 64, q_h=64, k=C.byref(_cache(P + GAP)), v=C.byref(_cache(P + 2 * GAP)), t=ops.BF16, pages=C.byref(_table()), kv=4, group=2,
             dim=64, window=0, scale=0.1, ws=P + 5 * GAP, wsb=1 << 28, out=P + 6 * GAP, out_b=8 * 64, out_h=64, lse=None, lse_b=0)
    a.update(kw)
    return fg.load_library().fg_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(ws=None), dict(pages=None), dict(k=None), dict(t=1), dict(t=2), dict(kv=0), dict(group=0), dict(dim=96), dict(dim=32),
    dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(wsb=64), dict(q=P + 8), dict(q_h=60),
    dict(q_b=-8), dict(out=P + 6 * GAP + 1), dict(out_h=63), dict(out_b=100), dict(ws=P + 5 * GAP + 8), dict(lse=P + 7 * GAP, lse_b=7), dict(lse=P + 7 * GAP + 2, lse_b=8),
    dict(out=P), dict(out=P + GAP), dict(out=P + 2 * GAP + 64), dict(out=P + 3 * GAP), dict(out=P + 4 * GAP), dict(out=P + 5 * GAP + 16), dict(ws=P),
    dict(ws=P + GAP), dict(lse=P + 6 * GAP, lse_b=8), dict(lse=P + GAP, lse_b=8), dict(k=C.byref(_cache(None))), dict(k=C.byref(_cache(P + GAP + 8))),
    dict(k=C.byref(_cache(P + GAP, row_stride=252))), dict(k=C.byref(_cache(P + GAP, row_stride=1 << 27))), dict(v=C.byref(_cache(P + 2 * GAP, scale=P))),
    dict(pages=C.byref(_table(page=8))), dict(pages=C.byref(_table(page=24))), dict(pages=C.byref(_table(n_pages=0))), dict(pages=C.byref(_table(width=0))),
    dict(pages=C.byref(_table(ldt=7))), dict(pages=C.byref(_table(table=None))), dict(pages=C.byref(_table(lens=None))), dict(pages=C.byref(_table(batch=-1))),
    dict(pages=C.byref(_table(batch=65536))), dict(pages=C.byref(_table(width=1 << 27, ldt=1 << 27))), dict(pages=C.byref(_table(batch=65535, width=1 << 26, ldt=1 << 26)))])
def test_paged_refuses(kw):
    assert _paged(**kw) == fg.EINVAL


def _latent(**kw):
    a = dict(q=P, q_b=4 * 192, q_h=192, w=P + GAP, cache=P + 2 * GAP, page_stride=16 * 576, row_stride=576, pages=C.byref(_table()), heads=4, rank=512, rope=64,
             nope=128, scale=0.1, ws=P + 5 * GAP, wsb=1 << 28, out=P + 6 * GAP, out_b=4 * 128, out_h=128, lse=None, lse_b=0)
    a.update(kw)
    return fg.load_library().fg_latent_attention(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(w=None), dict(cache=None), dict(pages=None), dict(out=None), dict(ws=None), dict(heads=0), dict(rank=128), dict(rank=384), dict(rope=0),
    dict(rope=48), dict(nope=96), dict(scale=0.0), dict(scale=float("nan")), dict(wsb=100), dict(q=P + 8), dict(w=P + GAP + 8), dict(cache=P + 2 * GAP + 8),
    dict(q_h=191), dict(page_stride=100), dict(row_stride=570), dict(row_stride=1 << 26), dict(out_h=127), dict(out_b=300), dict(lse=P + 7 * GAP, lse_b=3), dict(out=P),
    dict(out=P + GAP), dict(out=P + 2 * GAP), dict(out=P + 3 * GAP), dict(ws=P + 2 * GAP + 16), dict(lse=P + 4 * GAP, lse_b=4), dict(pages=C.byref(_table(page=8))),
    dict(pages=C.byref(_table(n_pages=0))), dict(pages=C.byref(_table(batch=1025, width=1 << 22, ldt=1 << 22)))])
def test_latent_refuses(kw):
    assert _latent(**kw) == fg.EINVAL


def _prompt(**kw):
    a = dict(q=P, q_t=4 * 192, q_h=192, qs=P + 3 * GAP, q_rows=20, lat=P + 2 * GAP, ld=576, ks=P + 4 * GAP, k_rows=30, batch=2, w=P + GAP, heads=4, rank=512, rope=64,
             nope=128, scale=0.1, ws=P + 5 * GAP, wsb=1 << 28, out=P + 6 * GAP, out_t=4 * 128, out_h=128, lse=None, lse_t=0)
    a.update(kw)
    return fg.load_library().fg_latent_prompt(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(qs=None), dict(ks=None), dict(lat=None), dict(w=None), dict(ws=None), dict(out=None), dict(q_rows=-1), dict(k_rows=-1), dict(batch=-1),
    dict(batch=65536), dict(heads=0), dict(rank=100), dict(rope=16), dict(nope=32), dict(scale=-0.5), dict(wsb=1000), dict(q=P + 2), dict(q_t=4), dict(ld=568),
    dict(ld=579), dict(ld=1 << 23), dict(k_rows=65535 * 128 + 1, wsb=1 << 40), dict(q_rows=2 ** 31 - 1), dict(batch=60000, heads=40000, wsb=1 << 40), dict(lat=P + 2 * GAP + 2), dict(out=P + 6 * GAP + 4), dict(out_h=130), dict(out_h=64), dict(lse=P + 7 * GAP, lse_t=2), dict(out=P), dict(out=P + GAP),
    dict(out=P + 2 * GAP), dict(out=P + 3 * GAP), dict(out=P + 5 * GAP), dict(ws=P + 2 * GAP), dict(lse=P + 6 * GAP, lse_t=4)])
def test_prompt_refuses(kw):
    assert _prompt(**kw) == fg.EINVAL


def test_workspaces():
    assert ops.paged_attention_bytes(4, 8, 4, 128) > 0 and ops.latent_attention_bytes(4, 16, 512) > 0 and ops.latent_prompt_bytes(100, 16, 128) == 4 * 100 * 16 * 128
    for f, sizes in ((ops.paged_attention_bytes, (4, 8, 4, 100)), (ops.paged_attention_bytes, (-1, 8, 4, 64)), (ops.latent_attention_bytes, (4, 0, 512)),
                     (ops.latent_attention_bytes, (4, 4, 500)), (ops.latent_prompt_bytes, (-1, 4, 64)), (ops.latent_prompt_bytes, (1, 4, 65))):
        with pytest.raises(fg.FgError):
            f(*sizes)


# ----------------------------------------------------------------- binding
def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _e4(*s):
    return torch.zeros(*s, dtype=torch.float8_e4m3fn)


ENDS, SLOTS = torch.zeros(2, dtype=torch.int64), torch.zeros(3, dtype=torch.int64)
KC, LAT, W = _bf(8, 16, 2, 64), _bf(8, 16, 576), _bf(4, 256, 512)


def paged(q=_bf(2, 4, 64), k=KC, v=KC, table=_i(2, 4), lens=_i(2), **kw):
    return ops.paged_attention(q, k, v, table, lens, **kw)


def latent(q=_bf(2, 4, 192), w=W, cache=LAT, table=_i(2, 4), lens=_i(2), nope=128, **kw):
    return ops.latent_attention(q, w, cache, table, lens, nope=nope, **kw)


def prompt(q=_bf(9, 4, 192), lat=_bf(9, 576), w=W, starts=_i(3), nope=128, **kw):
    return ops.latent_prompt(q, lat, w, starts, nope=nope, **kw)


@pytest.mark.parametrize("call", [
    lambda: ops.page_step(_i(2), _i(3), _i(2, 4), _i(8), ENDS, page=16, tokens=4),
    lambda: ops.page_step(_i(2), _i(2), _i(3, 4), _i(8), ENDS, page=16, tokens=4),
    lambda: ops.page_step(_i(2).long(), _i(2), _i(2, 4), _i(8), ENDS, page=16, tokens=4),
    lambda: ops.page_step(_i(2), _i(2), _i(2, 4), _i(8), ENDS.int(), page=16, tokens=4),
    lambda: ops.page_step(_i(2), _i(2), _i(2, 4), _i(16)[::2], ENDS, page=16, tokens=4),
    lambda: ops.page_step(_i(2), _i(2), _i(2, 4), _i(8), ENDS, page=0, tokens=4),
    lambda: ops.page_step(_i(2), _i(2), _i(2, 4), _i(8), ENDS, page=16, tokens=-1),
    lambda: ops.page_step(_i(2), _i(2), _i(2, 4), _i(8), ENDS, page=16, tokens=4, slots=_i(4)),
    lambda: ops.page_step(_i(2), _i(2), _i(1, 4).expand(2, 4), _i(8), ENDS, page=16, tokens=4),
    lambda: ops.page_step(_i(2), _i(2), _i(2, 4), _i(8), ENDS, page=16, tokens=4),                 # not on a GPU
    lambda: ops.kv_append(_bf(3, 2, 64), KC, SLOTS, v=_bf(3, 2, 64)),
    lambda: ops.kv_append(_bf(3, 2, 64), KC, SLOTS[:2]),
    lambda: ops.kv_append(_bf(3, 2, 64), KC, SLOTS.int()),
    lambda: ops.kv_append(_bf(3, 3, 64), KC, SLOTS),
    lambda: ops.kv_append(_bf(3, 2, 64).float(), KC, SLOTS),
    lambda: ops.kv_append(_bf(3, 2, 64), KC.half(), SLOTS),
    lambda: ops.kv_append(_bf(3, 2, 64), KC, SLOTS, k_scale=torch.zeros(8, 2, 16)),
    lambda: ops.kv_append(_bf(3, 2, 64), _e4(8, 16, 2, 64), SLOTS),
    lambda: ops.kv_append(_bf(3, 2, 64), _e4(8, 16, 2, 64), SLOTS, k_scale=torch.zeros(8, 16, 2)),
    lambda: ops.kv_append(_bf(3, 2, 64), KC, SLOTS, v_scale=torch.zeros(8, 2, 16)),
    lambda: ops.kv_append(_bf(3, 128), KC, SLOTS),
    lambda: ops.kv_append(_bf(3, 2, 128)[..., ::2], KC, SLOTS),
    lambda: ops.kv_append(_bf(3, 2, 64), KC, SLOTS),
    lambda: paged(q=_bf(2, 4, 64).float()), lambda: paged(q=_bf(2, 3, 64)), lambda: paged(q=_bf(2, 4, 128)), lambda: paged(q=_bf(4, 64)), lambda: paged(table=_i(3, 4)),
    lambda: paged(table=_i(2, 4).long()), lambda: paged(lens=_i(3)), lambda: paged(v=_bf(8, 16, 2, 128)), lambda: paged(v=_e4(8, 16, 2, 64)), lambda: paged(window=-1),
    lambda: paged(scale=0.0), lambda: paged(scale=float("nan")), lambda: paged(k_scale=torch.zeros(8, 2, 16)), lambda: paged(out=_bf(2, 4, 32)), lambda: paged(lse=torch.zeros(2, 3)),
    lambda: paged(k=_e4(8, 16, 2, 64), v=_e4(8, 16, 2, 64)), lambda: paged(k=_bf(8, 8, 2, 64), v=_bf(8, 8, 2, 64)), lambda: paged(k=_bf(0, 16, 2, 64), v=_bf(0, 16, 2, 64)),
    lambda: paged(),
    lambda: latent(w=_bf(4, 200, 512)), lambda: latent(w=_bf(3, 256, 512)), lambda: latent(q=_bf(2, 4, 160)), lambda: latent(cache=_bf(8, 16, 512)), lambda: latent(nope=64),
    lambda: latent(cache=LAT.float()), lambda: latent(cache=_bf(8, 8, 576)), lambda: latent(out=_bf(2, 4, 192)), lambda: latent(w=_bf(4, 512, 256).transpose(1, 2)),
    lambda: latent(scale=-1.0), lambda: latent(),
    lambda: prompt(starts=_i(0)), lambda: prompt(starts=_i(3).long()), lambda: prompt(k_starts=_i(4)), lambda: prompt(lat=_bf(9, 500)), lambda: prompt(lat=_bf(9, 576).float()),
    lambda: prompt(out=_bf(9, 4, 192)), lambda: prompt(q=_bf(9, 3, 192)), lambda: prompt(),
])
def test_binding_refuses(call):
    with pytest.raises(fg.FgError) as e:
        call()
    assert e.value.code == fg.EINVAL


@pytest.mark.parametrize("call", [lambda: paged(q=None), lambda: paged(lse="yes"), lambda: latent(w=3), lambda: prompt(nope="128"), lambda: prompt(nope=None),
                                  lambda: ops.kv_append(None, KC, SLOTS), lambda: paged(scale="1"), lambda: paged(window=1.5)])
def test_binding_refuses_other_types(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call", [
    lambda g: paged(q=g(2, 4, 64)), lambda g: paged(k=g(8, 16, 2, 64)), lambda g: latent(w=g(4, 256, 512)), lambda g: prompt(lat=g(9, 576)), lambda g: paged(out=g(2, 4, 64)),
    lambda g: ops.kv_append(g(3, 2, 64), KC, SLOTS), lambda g: ops.kv_append(_bf(3, 2, 64), g(8, 16, 2, 64), SLOTS)])
def test_gradients_are_refused(call):
    """There is no backward pass; on the CPU the device is refused as well, so the message is looked at."""
    with pytest.raises(fg.FgError, match="backward"):
        call(lambda *s: torch.zeros(*s, dtype=torch.bfloat16, requires_grad=True))
