"""Rates e^A_log past float32's largest number: a channel that forgets at once, its decay 0 and the gradient of its rate 0."""
import numpy as np
import pytest
import torch

import test_gpu_gated_scan as S
from oracle import gated_oracle as GO

pytestmark = pytest.mark.gpu

RATES = np.array([80.0, 87.9, 88.1, 88.8, 90.0, 200.0, 700.0], np.float32)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


@pytest.mark.parametrize("codes", [False, True], ids=["whole", "8 bits"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 300])
def test_a_rate_past_the_largest_number(T, dtype, codes):
    import selective_state_space_41_amd as V
    dim = len(RATES)
    p = S.make(2, T, dim, dtype, T)
    p["A_log"] = RATES
    x, r, i, d = (S.td(p[k], dtype) for k in ("x", "r", "i", "dout"))
    A, first, dlast = S.td(p["A_log"]), S.td(p["first"]), S.td(p["dlast"])
    out, last, kept = V.gated_scan_fwd(x, r, i, A, initial_state=first, keep=codes)
    (h, hl), (room, rl) = GO.gated_scan(p["x"], p["r"], p["i"], p["A_log"], p["first"])
    S.near("h", out, h, room + S.unit(dtype) * np.abs(h))
    S.near("final state", last, hl, rl)
    vals = S.values_of(*kept) if codes else (p["x"], p["r"], p["i"], S.rnd(h, dtype))
    g = V.gated_scan_bwd(kept if codes else (x, r, i, S.td(vals[3], dtype)), A, d, initial_state=first, dfinal_state=dlast)
    want, rooms = GO.gated_scan_bwd(*vals, p["A_log"], p["dout"], p["first"], dlast=p["dlast"])
    for k in ("dx", "dr", "di"):
        S.near(k, g[k], want[k], rooms[k] + S.unit(dtype) * np.abs(want[k]))
    S.near("dA_log", g["dA_log"], want["dA"], rooms["dA"])
    S.near("dinitial_state", g["dinitial_state"], want["dfirst"], rooms["dfirst"])


def test_a_shut_gate_under_such_a_rate():
    """sigmoid(r) that is 0 in float32 leaves the state as it is, whatever the rate; a rate that is no number stays one."""
    import selective_state_space_41_amd as V
    A = torch.tensor([0.0, 88.8, 200.0, float("inf"), float("nan")], device="cuda")
    x, i = torch.ones(1, 3, 5, device="cuda"), torch.zeros(1, 3, 5, device="cuda")
    r = torch.full((1, 3, 5), -1e4, device="cuda")
    first = torch.full((1, 5), 2.0, device="cuda")
    out, last, _ = V.gated_scan_fwd(x, r, i, A, initial_state=first)
    assert (out[..., :4] == 2.0).all() and (last[:, :4] == 2.0).all() and torch.isnan(out[..., 4]).all()
    state = first.clone()
    assert (V.gated_scan_step(x[:, 0], r[:, 0], i[:, 0], A, state)[:, :4] == 2.0).all() and (state[:, :4] == 2.0).all()
    g = V.gated_scan_bwd((x, r, i, out), A, x, initial_state=first)
    assert all(torch.isfinite(g[k][..., :4]).all() for k in ("dx", "dr", "di", "dA_log", "dinitial_state"))
    assert (g["dinitial_state"][:, :4] == 3.0).all()
