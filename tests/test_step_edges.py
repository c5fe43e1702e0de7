"""CPU tests of the decode step's operators: calls at the edge of what the header allows, answered before any HIP call."""
from __future__ import annotations

import pytest

from test_step import NULL, OK, SHAPE, attn, qk, read, sample, w4


# ------------------------------------------------------------ empty problems
# An array without elements may have no address: torch gives 0 for such a tensor.
@pytest.mark.parametrize("call,kwargs", [
    (attn, dict(T=0, q=None, out=None)), (attn, dict(B=0, lens=None, table=None)),
    (attn, dict(T=0, B=0, q=None, out=None, lens=None, table=None, q_start=None)),
    (qk, dict(T=0, q=None, k=None, v=None, qo=None, ko=None, pos=None, slots=None)),
    (qk, dict(T=0, cache=False, q=None, k=None, qo=None, ko=None, pos=None)), (qk, dict(T=0, hq=0, q=None, qo=None, k=None)),
    (read, dict(n=0, slots=None, ko=None, vo=None)), (read, dict(n=0, slots=None, vo=None)),
    (sample, dict(rows=0, logits=None, u=None, tokens=None, t=None, k=None, p=None, m=None, ws=None, wsb=0)),
])
def test_empty_problems_need_no_addresses(call, kwargs):
    assert call(**kwargs) == OK


@pytest.mark.parametrize("call,kwargs,status", [
    (attn, dict(T=0, lens=None), NULL), (attn, dict(T=0, table=None), NULL), (attn, dict(B=0, q=None, lens=None), NULL),
    (qk, dict(T=0, cs=None), NULL), (qk, dict(T=0, reach=0), SHAPE), (qk, dict(T=0, kc=None), NULL),
    (read, dict(n=0, kc=None), NULL), (sample, dict(rows=0, vocab=0), SHAPE), (sample, dict(rows=1, u=None), NULL),
])
def test_empty_problems_are_checked_for_the_rest(call, kwargs, status):
    assert call(**kwargs) == status


# ---------------------------------------------------------------- launch sizes
@pytest.mark.parametrize("call,kwargs", [
    (qk, dict(T=1 << 26)), (qk, dict(T=(1 << 26) - 3, cache=False)), (qk, dict(T=2 ** 31 - 1, hq=1, hkv=1, dim=64, rot=64)),
    (read, dict(n=1 << 27, hkv=2)), (read, dict(n=(1 << 28) - 15, hkv=1)), (read, dict(n=1 << 29, hkv=1, dim=64)),
    (read, dict(n=1 << 22, hkv=32, dim=256)),
])
def test_launches_past_2_32_work_items_are_refused(call, kwargs):
    """A launch counts its work-items in 32 bits: 64 for each token from 8192 tokens on, one for 8 values read back."""
    assert call(**kwargs) == SHAPE
    assert "too many rows" in w4.w4_last_error()


