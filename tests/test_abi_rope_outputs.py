"""C-ABI: rotary positions refuse an output whose own elements overlap (several threads would write, and in place read, the
same ones); layouts in any order of the axes pass that check (no GPU: those end at the next bad argument)."""
import os

import pytest

import selective_state_space_41_amd as V
from test_abi_blocks import ERR_SHAPE, rope, st


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(V.LIB_PATH):
        pytest.fail(f"{V.LIB_PATH} not built (run __graft_entry__.build())")
    return V.load()


# 2 batches of 9 tokens, 4 heads of 32
@pytest.mark.parametrize("strides", [(0, 128, 32), (4096, 0, 32), (4096, 128, 0), (4096, 128, 31), (1151, 128, 32), (4096, 127, 32),
                                     (4096, 32, 32), (32, 63, 4096), (-1151, 128, 32)])
def test_overlapping(lib, strides):
    assert rope(lib, qos=st(*strides)) == ERR_SHAPE
    assert rope(lib, kos=st(*strides)) == ERR_SHAPE
