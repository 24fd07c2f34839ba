"""How many rows the slabs of the experts' products may have: 32 bits hold a row, the stage of 64 rows or the
tile of up to 256 that begins there, and a box of its copies. CPU only; the pointers are never dereferenced."""
import pytest

from test_expert_refusals import CALLS, INVALID, L, call  # noqa: F401


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("R,max_rows", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 64), (1, 2 ** 31 - 511), (4, 2 ** 29 - 127),
                                        (2, 2 ** 30 - 255)])
def test_slabs_that_end_beside_2_31_are_refused(L, name, R, max_rows):  # noqa: F811
    assert call(getattr(L, "ep_expert_" + name), CALLS[name], R=R, max_rows=max_rows) == INVALID


def test_sums_of_rows_stay_below_2_32():
    """The plan's arithmetic in 32 bits, at the most rows and the smallest tiles of each height."""
    most = 2 ** 31 - 512
    for height in (256, 128, 64, 32):
        tiles = (most + height - 1) // height
        assert most + height - 1 < 2 ** 32 and most + tiles - 1 < 2 ** 32
        each = ((most + tiles - 1) // tiles + 31) & ~31
        assert each <= height and (tiles - 1) * each < most
        assert most - 1 + 64 + 256 < 2 ** 31 - 64  # a stage's end, a tile's last box
