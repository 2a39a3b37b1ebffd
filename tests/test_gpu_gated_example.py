"""The example block (examples/gated_recurrence_block.py): its gradients through the library's operators against torch's
autograd of the same block in float64, with activations whole and in 8 bits, and its serving path against the whole
sequence."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "gated_recurrence_block.py")


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    spec = importlib.util.spec_from_file_location("gated_recurrence_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_block(p, tokens, groups, ways, lengths):
    """The block in torch operations, token by token, float64 on the CPU."""
    B, L, dim = tokens.shape
    live = (torch.arange(L)[None] < lengths[:, None]).to(tokens.dtype)
    count = (lengths * (dim // groups)).to(tokens.dtype)[:, None]
    x = tokens.view(B, L, groups, -1) * live[..., None, None]
    mean = x.sum((1, 3)) / count
    d = (x - mean[:, None, :, None]) * live[..., None, None]
    rstd = (d.square().sum((1, 3)) / count + 1e-5) ** -0.5
    u = ((d * rstd[:, None, :, None]).reshape(B, L, dim) * p["weight"] + p["bias"])
    y = u * torch.sigmoid(u) * live[..., None]
    inner = p["out"].shape[1]
    parts = (y @ p["xri"].t()).split(inner, -1)
    total = 0
    for w in range(ways):
        x, r, i = parts[3 * w:3 * w + 3]
        la = -torch.exp(p["A_log"][w]) * torch.sigmoid(r)
        a, b = torch.exp(la), torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * x
        h, out = torch.zeros(B, inner, dtype=tokens.dtype), [None] * L
        for t in range(L - 1, -1, -1) if w else range(L):
            m = live[:, t, None]
            h = m * (a[:, t] * h + b[:, t]) + (1 - m) * h
            out[t] = m * h
        total = total + torch.stack(out, 1)
    return tokens + total / ways @ p["out"].t()


def grads_of(E, keep, seed=1):
    torch.manual_seed(seed)
    B, L, dim, inner, groups = 3, 90, 24, 40, 3
    block = E.Block(dim, inner, groups, keep=keep, dtype=torch.float32)
    tokens = torch.randn(B, L, dim, device="cuda", requires_grad=True)
    lengths = torch.tensor([90, 1, 57], dtype=torch.int32, device="cuda")
    w = torch.randn(B, L, dim, device="cuda") * (torch.arange(L, device="cuda")[None] < lengths[:, None])[..., None]
    (block(tokens, lengths) * w).sum().backward()
    got = {n: q.grad for n, q in block.named_parameters()}
    got["tokens"] = tokens.grad
    p = {n: q.detach().double().cpu().requires_grad_() for n, q in block.named_parameters()}
    t64 = tokens.detach().double().cpu().requires_grad_()
    (plain_block(p, t64, groups, 2, lengths.cpu().long()) * w.double().cpu()).sum().backward()
    want = {n: q.grad for n, q in p.items()}
    want["tokens"] = t64.grad
    return got, want


def off(got, want):
    return {n: ((got[n].double().cpu() - want[n]).norm() / want[n].norm()).item() for n in want}


def test_training_step(E):
    """Every gradient, float32 against float64: some ten operators of sums of up to 270 terms, each within about 2^-21 of
    its magnitudes: below 1e-5 of the gradient's norm."""
    err = off(*grads_of(E, keep=False))
    print(err)
    assert all(e < 1e-5 for e in err.values()), err


def test_training_step_from_8_bits(E):
    """The same with activations in 8 bits.  A kept value is off by at most 2^-4 of itself, in the mean by under 0.03; a
    term of a gradient has at most four of them as factors (x or the state, the gates, the norm's x), and errors of
    different tokens add up at random: under 0.12 of the gradient's norm, 0.25 with the gates' slopes."""
    err = off(*grads_of(E, keep=True))
    print(err)
    assert all(e < 0.25 for e in err.values()), err
    assert any(e > 1e-4 for e in err.values())  # 8 bits were used


def test_serving(E):
    """bfloat16: a prompt and single tokens against the whole sequence: the recurrence is the same in float32, so outputs
    differ by the rounding of h to bfloat16 (2^-8 of it) and its sum in the projection over 64 channels."""
    torch.manual_seed(2)
    block = E.Block(32, inner=64, groups=4, both=False)
    y = torch.randn(2, 40, 32, device="cuda").bfloat16()
    whole, last = block.scan(y)
    _, state = block.scan(y[:, :30])
    pool, slots = torch.zeros(4, 64, device="cuda"), torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(30, 40):
        o = block.token(y[:, t], pool, slots)
        assert (o - whole[:, t]).float().abs().max() <= 2.0 ** -6 * whole.float().abs().max()
    assert (pool[slots.long()] - last).abs().max() <= 1e-4 * last.abs().max()
    assert not pool[[0, 2]].any()


def test_it_runs():
    r = subprocess.run([sys.executable, PATH, "--batch", "2", "--side", "9"], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "in 8 bits" in r.stdout and "single ones" in r.stdout
