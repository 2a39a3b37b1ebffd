"""The group norm's statistics where one workgroup walks over many tokens of a row and its first tokens lie far from the
others, as a register token's or a border pixel's do: neither they nor a large mean cost the deviation anything.

Rooms of test_gpu_groupnorm.py: (80 + 8 |mean| / std) U on the reciprocal deviation.  A thread adds up to 1000 squares to
one float32 sum here; roundings to nearest that add up at random, each within U of the sum: under 2 sqrt(1000) U = 64 U of
the variance, 32 U of its root.  The sums' recentring, once in eight tokens, adds a fourth as many at most."""
import numpy as np
import pytest
import torch

import test_gpu_groupnorm as N
from oracle import gated_oracle as GO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


@pytest.mark.parametrize("what", ["plain", "first x 100", "first x 1e3", "first x 1e4", "last x 1e4", "mean 3000", "drift"])
@pytest.mark.parametrize("B,T,dim,groups,dtype", [(257, 1000, 2048, 4, "f32"), (512, 3136, 512, 32, "bf16"), (300, 1000, 1030, 5, "f32")],
                         ids=["a token a step", "four tokens a step", "odd groups"])
def test_far_tokens_in_long_runs(B, T, dim, groups, dtype, what):
    """One image for all rows (a batch stride of 0): a run is a whole row."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(T + dim)
    x = rng.standard_normal((1, T, dim))
    if what.startswith("first"):
        x[0, :4] *= float(what.split()[-1])  # the first token of every row of a step
    elif what.startswith("last"):
        x[0, -4:] *= 1e4
    elif what == "mean 3000":
        x += 3000.0
    elif what == "drift":
        x += np.linspace(0.0, 300.0, T)[None, :, None]
    x = N.rnd(x, dtype)
    w, b = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32), (0.3 * rng.standard_normal(dim)).astype(np.float32)
    y, mean, rstd, _ = V.groupnorm_fwd(N.td(x, dtype).expand(B, T, dim), N.td(w), N.td(b), groups, act=False)
    ry, rmean, rrstd = GO.groupnorm(x, w, b, groups, act=False)
    tm, tr, ty = N.forward_rooms(x, w, b, groups, rmean, rrstd, False, None, 1e-5)
    assert torch.equal(mean, mean[:1].expand(B, groups)) and torch.equal(rstd, rstd[:1].expand(B, groups))
    N.near("mean", mean[:1], rmean, tm)
    N.near("rstd", rstd[:1], rrstd, tr)
    for row in (0, B - 1):
        N.near("y", y[row:row + 1], ry, ty + N.unit(dtype) * np.abs(ry))


@pytest.mark.parametrize("T", [1, 2, 3, 5, 257, 1003])
def test_few_and_odd_tokens(T):
    """Runs whose last steps are short: a channel a group of 4096, a row a step."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(T)
    x = rng.standard_normal((2, T, 4096)).astype(np.float32)
    x[:, 0] *= 1e3
    lengths = [T, max(1, T - 2)]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    w, b = np.ones(4096, np.float32), np.zeros(4096, np.float32)
    y, mean, rstd, _ = V.groupnorm_fwd(N.td(x), N.td(w), N.td(b), 1, act=False, lengths=n)
    ry, rmean, rrstd = GO.groupnorm(x, w, b, 1, act=False, lengths=lengths)
    tm, tr, ty = N.forward_rooms(x, w, b, 1, rmean, rrstd, False, lengths, 1e-5)
    N.near("mean", mean, rmean, tm)
    N.near("rstd", rstd, rrstd, tr)
    N.near("y", y, ry, ty + GO.U * np.abs(ry))
