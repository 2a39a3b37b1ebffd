"""How a linear-attention call is cut up: the occupancies it is planned with are the ones the build holds the kernels to,
and the query's refusals (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

import selective_state_space_41_amd as V
from selective_state_space_41_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(V.LIB_PATH):
        pytest.fail(f"{V.LIB_PATH} not built (run __graft_entry__.build())")
    return V.load()


def test_planned_occupancies_are_the_checked_ones():
    src = open(os.path.join(ROOT, "selective_state_space_41_amd", "csrc", "linattn.hip")).read()
    table = re.search(r"constexpr Walk kWalks\[2\]\[2\]\[3\]\[3\] = (.*?);", src, re.S).group(1)
    places = [int(n or 0) for n in re.findall(r"\{(?:(\d+), [\d.]+, [\d.]+)?\}", table)]
    want = [n for kernel in ("fwd", "grad") for t in "tf" for dk in (32, 64, 128) for n in build.WALKS_PER_CU[kernel][t][dk]]
    assert places == want and len(places) == 36


def _report(name, occ, lds, scratch=0):
    return {name: dict(VGPRs=100, AGPRs=0, ScratchSize=scratch, Occupancy=occ, LDS=lds)}


@pytest.mark.parametrize("name,occ,lds,scratch,bad", [
    ("linattn_fwd_kernelIfLi64ELi64E", 2, 52224, 0, 0), ("linattn_fwd_kernelIfLi64ELi64E", 1, 52224, 0, 1),
    ("linattn_fwd_kernelItLi128ELi64E", 2, 90000, 0, 1), ("linattn_grad_kernelItLi64ELi64E", 4, 81168, 48, 0),
    ("linattn_grad_kernelItLi64ELi64E", 2, 81168, 0, 1), ("linattn_grad_kernelIfLi64ELi64E", 2, 99600, 0, 0),
    ("linattn_fwd_kernelItLi32ELi32E", 4, 17408, 8, 1), ("linattn_prefix_kernelILb1E", 8, 0, 16, 1),
    ("rmsnorm_bwd_kernelItfLi64ELi16ELi4E", 4, 128, 440, 1), ("rmsnorm_bwd_kernelItfLi64ELi16ELi4E", 4, 128, 208, 0),
    ("rmsnorm_fwd_kernelIffLb0ELi64ELi1ELi4E", 4, 0, 4, 1), ("rope_kernelIfLi4ELb0E", 8, 0, 4, 1)])
def test_guard(name, occ, lds, scratch, bad):
    assert len(build.check_resources(_report(name, occ, lds, scratch))) == bad


def test_query(lib):
    plan = V.linattn_plan(128, 197, 6, 64, 64)
    assert plan == dict(block=64, width=64, segments=1, parts=1, join=None)
    long = V.linattn_plan(1, 6085, 6, 64, 64)
    assert long["segments"] > 1 and long["join"] == "walk"
    assert V.linattn_plan(1, 500, 1, 128, 128, torch.float32, gradient=True)["block"] == 32
    cut = (ctypes.c_int32 * 5)()
    call = lambda *a: lib.vmscan_linattn_plan(*a)
    assert call(1, 9, 1, 64, 64, 1, 0, None) == 1
    assert call(0, 9, 1, 64, 64, 1, 0, cut) == 2 and call(1, 1 << 30, 1, 64, 64, 1, 0, cut) == 2
    assert call(1, 9, 1, 60, 64, 1, 0, cut) == 3 and call(1, 9, 1, 64, 64, 2, 0, cut) == 3 and call(1, 9, 1, 64, 64, 1, 2, cut) == 3
    with pytest.raises(TypeError):
        V.linattn_plan(1, 9, 1, 64, 64, torch.float16)
