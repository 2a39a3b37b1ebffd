"""The example block (examples/linear_attention_block.py): its gradients through the library's operators against
torch's autograd of the same block in float64, and its serving path against the whole sequence."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "linear_attention_block.py")


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    spec = importlib.util.spec_from_file_location("linear_attention_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_block(p, x, residual, pos, inv_freq, axis, heads, kheads, d, lengths):
    """The block in torch operations, the attention as a loop over the tokens."""
    r = x + residual
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-5) * p["norm"]
    qkv = (y @ p["qkv"].t()).unflatten(-1, (2 * kheads + heads, d))
    q, k, v = qkv[..., :kheads, :], qkv[..., kheads:2 * kheads, :], qkv[..., 2 * kheads:, :]
    decay = -torch.nn.functional.softplus(y @ p["step"].t() + p["step_bias"])
    angle = pos[:, axis.long()] * inv_freq
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def turn(a):
        u, w = a[..., :d // 2], a[..., d // 2:]
        return torch.cat([u * c - w * s, u * s + w * c], -1)

    q, k = (turn(a).repeat_interleave(heads // kheads, 2) for a in (q, k))
    S, out = torch.zeros(len(x), heads, d, d, dtype=x.dtype), []
    for t in range(x.shape[1]):
        live = (t < lengths).to(x.dtype)[:, None, None]
        S = torch.where(live[..., None] > 0, torch.exp(decay[:, t])[..., None, None] * S
                        + k[:, t, :, :, None] * v[:, t, :, None, :], S)
        out.append(live * d ** -0.5 * (q[:, t, :, :, None] * S).sum(-2))
    return torch.stack(out, 1).flatten(-2) @ p["out"].t(), r


def test_training_step(E):
    """Every parameter's and input's gradient, float32 against float64.  A gradient passes about ten
    float32 operators with sums of up to 4096 terms; relative to its norm that is below 1e-5."""
    torch.manual_seed(1)
    B, side, dim, heads, kheads, d = 3, 6, 40, 4, 2, 16
    block = E.Block(dim, heads, kheads, d, dtype=torch.float32)
    pos = E.grid_positions(side, "cuda")
    L = len(pos)
    x, residual = (torch.randn(B, L, dim, device="cuda", requires_grad=True) for _ in range(2))
    w1, w2 = torch.randn(B, L, dim, device="cuda"), torch.randn(B, L, dim, device="cuda")
    lengths = torch.tensor([L, 0, 11], dtype=torch.int32, device="cuda")
    out, r = block(x, residual, pos, lengths)
    ((out * w1).sum() + (r * w2).sum()).backward()

    f64 = lambda t: t.detach().double().cpu()
    p = {n: f64(t).requires_grad_() for n, t in block.named_parameters()}
    x64, r64 = f64(x).requires_grad_(), f64(residual).requires_grad_()
    o2, s2 = plain_block(p, x64, r64, f64(pos), f64(block.inv_freq), block.axis.cpu(), heads, kheads, d, lengths.cpu())
    ((o2 * f64(w1)).sum() + (s2 * f64(w2)).sum()).backward()
    pairs = dict(output=(out, o2), x=(x.grad, x64.grad), residual=(residual.grad, r64.grad),
                 **{n: (t.grad, p[n].grad) for n, t in block.named_parameters()})
    for n, (a, b) in pairs.items():
        err = float((f64(a) - b.detach()).norm() / b.detach().norm())
        print(f"[example] {n}: {err:.2e}", flush=True)
        assert err <= 1e-5, n


def test_prompt_then_tokens(E):
    """A prompt cut in two with a state between, then single tokens, equals the whole sequence."""
    torch.manual_seed(2)
    B, side, dim = 2, 5, 48
    block = E.Block(dim, 2, 1, 32, dtype=torch.float32)
    pos = E.grid_positions(side, "cuda")
    L = len(pos)
    x, residual = torch.randn(2, B, L, dim, device="cuda")
    whole, _, last = block.prompt(x, residual, pos)
    cut = lambda t, a, b: t[:, a:b].contiguous()
    a, _, state = block.prompt(cut(x, 0, 9), cut(residual, 0, 9), pos[:9].contiguous())
    b, _, state = block.prompt(cut(x, 9, 20), cut(residual, 9, 20), pos[9:20].contiguous(), state=state)
    torch.testing.assert_close(torch.cat([a, b], 1), whole[:, :20], rtol=1e-4, atol=1e-4)
    pool = torch.zeros(4, *state.shape[1:], device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(20, L):
        o, _ = block.token(x[:, t].contiguous(), residual[:, t].contiguous(), pos[t].expand(B, 2), pool, slots)
        torch.testing.assert_close(o, whole[:, t], rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(pool[slots.long()], last, rtol=1e-4, atol=1e-4)
    assert torch.all(pool[0] == 0) and torch.all(pool[2] == 0)


def test_runs(E):
    r = subprocess.run([sys.executable, PATH, "--batch", "2", "--side", "7"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "training step" in r.stdout and "norm in 8 bits" in r.stdout
