"""C-ABI: the row stride of the norm's gradient (no GPU)."""
import os

import pytest

import selective_state_space_41_amd as V
from test_abi_blocks import ERR_ALIGN, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, P


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(V.LIB_PATH):
        pytest.fail(f"{V.LIB_PATH} not built (run __graft_entry__.build())")
    return V.load()


def call(lib, **kw):
    a = dict(dy=P[0], r=P[1], stride=96, w=P[2], rstd=P[3], dro=P[4], dx=P[5], dres=P[6], dw=P[7], rows=4, dim=64, dt=1, rdt=0,
             ws=P[8], wsb=0)
    a.update(kw)
    return lib.vmscan_rmsnorm_bwd_ex(*a.values(), None)


def test_refusals(lib):
    assert call(lib) == ERR_WORKSPACE  # everything before it is right
    assert call(lib, r=None) == ERR_NULL and call(lib, stride=63) == ERR_SHAPE and call(lib, stride=-64) == ERR_SHAPE
    assert call(lib, stride=1 << 41) == ERR_SHAPE and call(lib, rdt=1) == ERR_UNSUPPORTED and call(lib, r=P[1] + 8) == ERR_ALIGN
