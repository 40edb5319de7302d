"""The page bookkeeping where its inputs are at their limits: partial last pages that do
not exist."""
import pytest
import torch

from parametrized_local_linear_gb300 import plx_check_device_error, plx_kv_update

from helpers import device
from test_moves_gpu import I32, Cache, ints, reported

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -7, 30, 2**31 - 1, -2**31])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("fork", [True, False])
def test_a_partial_last_page_that_does_not_exist_stays_an_entry(bad, in_place, fork):
    """It is reported and kept, as a whole page is: no page is given in its place, and the
    other rows get theirs."""
    device()
    c = Cache(4, 6, 30, 16, 1, False)
    c.update([40, 40, 0, 16])  # pages 0 1 2, 3 4 5, none, 6
    c.dev["block_table"][0, 2] = bad
    pages = c.dev["kpages"].clone()
    outs = {} if in_place else dict(block_table_out=torch.full((4, 6), -9, dtype=I32, device="cuda"),
                                    seqlens_out=torch.empty(4, dtype=I32, device="cuda"),
                                    page_refs_out=torch.empty(30, dtype=I32, device="cuda"))
    got = plx_kv_update(lens=ints([41, 50, 40 if fork else 0, 0]), src=ints([0, 1, 0, 3]) if fork else None, **c.dev, **outs)
    reported()
    table, lens, refs = (x.tolist() for x in got)
    assert lens == [41, 50, 40 if fork else 0, 0]
    assert table[0][:3] == [0, 1, bad] and table[1][:4] == [3, 4, 5, 6]
    if fork:
        assert table[2][:3] == [0, 1, bad]
    # Page 2 has lost its entry, not its count; page 6 was row 3's.
    assert refs == [1 + fork, 1 + fork, 1, 1, 1, 1, 1] + [0] * 23
    assert torch.equal(c.dev["kpages"], pages)
    # The row grows past it, is cut in front of it, and ends.
    c.dev.update(zip(("block_table", "seqlens", "page_refs"), got))
    got = plx_kv_update(lens=ints([49, 50, 32 if fork else 0, 0]), **c.dev)
    reported()
    assert got[0].tolist()[0][:4] == [0, 1, bad, 7] and got[1].tolist() == [49, 50, 32 if fork else 0, 0]
    got = plx_kv_update(lens=ints([0, 0, 0, 0]), **c.dev)
    reported()
    assert got[2].tolist() == [0, 0, 1] + [0] * 27
    plx_check_device_error()
