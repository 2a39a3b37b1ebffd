"""C-ABI: states that overlap without being the same buffer are refused before anything is enqueued (no GPU)."""
import ctypes
import os

import pytest

import selective_state_space_41_amd as V
from test_abi_blocks import ERR_UNSUPPORTED, bwd, fwd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(V.LIB_PATH):
        pytest.fail(f"{V.LIB_PATH} not built (run __graft_entry__.build())")
    return V.load()


BYTES = 2 * 4 * 32 * 32 * 4  # of the states of those calls
BASE, ENOUGH = 0x10000000, 1 << 40


@pytest.mark.parametrize("step", [16, BYTES - 16, -16, 16 - BYTES])
def test_overlap(lib, step):
    assert fwd(lib, s0=BASE, sT=BASE + step, wsb=ENOUGH) == ERR_UNSUPPORTED
    assert bwd(lib, dsT=BASE, ds0=BASE + step, wsb=ENOUGH) == ERR_UNSUPPORTED
    assert bwd(lib, s0=BASE, dsT=2 * BASE, ds0=BASE + step, wsb=ENOUGH) == ERR_UNSUPPORTED
