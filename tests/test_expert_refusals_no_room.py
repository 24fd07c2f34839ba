"""Slabs without rows at the C entries: with a status the offsets are needed, since rows may be dropped
(EP_ERR_INVALID before anything is launched). CPU only; the pointers are never dereferenced."""
import pytest

from test_expert_refusals import CALLS, F, INVALID, L, ODD, OK, call  # noqa: F401


@pytest.mark.parametrize("name", list(CALLS))
def test_offsets_are_needed_where_rows_can_be_reported(L, name):  # noqa: F811
    fn, base = getattr(L, "ep_expert_" + name), CALLS[name]
    for offsets in (None, ODD):
        assert call(fn, base, max_rows=0, status=F, offsets=offsets) == INVALID
    if name != "wgrad":  # which clears dw
        nothing = {n: None for n, v in base.items() if v is F}
        assert call(fn, base, max_rows=0, **nothing) == OK
