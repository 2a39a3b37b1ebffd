"""Rotary positions of more work items than one launch holds (2^32): the tokens on both sides of the first launch's end, the
first and the last ones against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu


def test_more_than_one_launch():
    import selective_state_space_41_amd as V
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    # one pair or channel a thread: 31 pairs and 2 channels that pass through of each token's 64
    tokens, dim, pairs = 2 ** 32 // 33 + 1000, 64, 31
    end = ((2 ** 24 - 1) * 256) // 33
    print(f"[rope] {tokens} tokens of {dim}", flush=True)
    q = torch.empty(1, tokens, 1, dim, dtype=torch.bfloat16, device="cuda")
    row = torch.randn(dim, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    q.copy_(row.expand_as(q))
    pos = torch.arange(tokens, device="cuda").remainder_(1000).float()[:, None].contiguous()
    freq = torch.logspace(0, -3, pairs, device="cuda")
    axis = torch.zeros(pairs, dtype=torch.int32, device="cuda")
    V.rope_axes(q, None, pos, freq, axis, q_out=q)
    torch.cuda.synchronize()
    for at in (0, end - 50, tokens - 100):
        got = q[:, at:at + 100].float().cpu().numpy()
        x = np.broadcast_to(row.float().cpu().numpy(), (1, 100, 1, dim))
        want = BO.rope_axes(x, pos[at:at + 100].cpu().numpy(), freq.cpu().numpy(), axis.cpu().numpy())
        # half a unit of bfloat16 and 2^-20 of a pair's length (no larger than 8)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17), at
        assert np.array_equal(got[..., 62:], x[..., 62:])
    # the same values where positions repeat, everywhere
    assert torch.equal(q[0, :1000], q[0, tokens // 2000 * 1000:][:1000])
