"""Refusals of the attention half's operators in rarer calls, without a GPU: nothing is launched."""
import pytest

from sync_protocols_amd import fg
from test_attention_refusals import _pages


@pytest.mark.parametrize("kw", [dict(starts=None), dict(ends=None), dict(ends_out=None)])
def test_page_step_of_nothing_has_outputs(kw):
    assert _pages(batch=0, tokens=0, **kw) == fg.EINVAL
