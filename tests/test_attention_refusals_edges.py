"""Refusals of the attention half's operators in rarer calls, without a GPU: nothing is launched."""
import pytest

from sync_protocols_amd import fg
from test_attention_refusals import C, GAP, P, _append, _cache, _latent, _pages, _paged, _prompt


@pytest.mark.parametrize("kw", [dict(starts=None), dict(ends=None), dict(ends_out=None)])
def test_page_step_of_nothing_has_outputs(kw):
    assert _pages(batch=0, tokens=0, **kw) == fg.EINVAL


@pytest.mark.parametrize("call", [
    lambda **kw: _paged(q_b=0, out_b=4096, lse_b=8, **kw), lambda **kw: _latent(q_b=0, out_b=4096, lse_b=8, **kw), lambda **kw: _prompt(q_t=0, out_t=4096, lse_t=8, **kw)])
@pytest.mark.parametrize("at", [2048, 0, 8192 - 256])
def test_broadcast_queries_between_or_on_the_rows_of_the_output(call, at):
    """The one row of queries lies behind the output's first row, or on it, or reaches into the second; refused at the latest since lse lies on the output."""
    out = P + 6 * GAP
    assert call(q=out + at, out=out, lse=out) == fg.EINVAL


def test_broadcast_rows_on_a_cache():
    assert _append(dict(x=P + GAP + 16384, x_row=0, x_head=0)) == fg.EINVAL


def test_broadcast_caches_and_outputs_on_them():
    out = P + 6 * GAP
    flat = _cache(out + 64, page_stride=0, row_stride=0, head_stride=0)
    assert _paged(out=out, k=C.byref(flat)) == fg.EINVAL and _latent(out=out, cache=out + 64, page_stride=0, row_stride=0) == fg.EINVAL


@pytest.mark.parametrize("by", [16, 128, -128, 512, 8192 - 256, -8192, 8 * 8192 - 512 - 16])
def test_append_refuses_caches_that_partly_lie_on_each_other(by):
    """A cache of 8 pages of 16 rows of 4 heads of 64: some columns, heads, rows or pages further on in itself, with the same strides or others."""
    assert _append(values=dict(cache=P + GAP + by)) == fg.EINVAL
    assert _append(values=dict(cache=P + GAP + by, row_stride=512, page_stride=8192)) == fg.EINVAL
    wide = dict(row_stride=512, page_stride=8192)                # rows and their gaps are as long
    assert _append(wide, dict(cache=P + GAP + 512 - 16, **wide)) == fg.EINVAL and _append(wide, dict(cache=P + GAP + 512 + 16, **wide)) == fg.EINVAL


@pytest.mark.parametrize("at", [16, 8192 - 8])
def test_append_refuses_8_bit_caches_that_partly_lie_on_each_other(at):
    keys, values = dict(scale=P + 5 * GAP), dict(cache=P + GAP + at, scale=P + 6 * GAP)
    assert _append(keys, values, t=2) == fg.EINVAL
