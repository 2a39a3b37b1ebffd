"""The example blocks' operators have first gradients only: a gradient of a gradient is refused, not given without their share."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def twice(block, out, *inputs):
    """The penalty of a gradient's square, as far as torch lets it be differentiated."""
    of = [p for p in block.parameters()] + list(inputs)
    first = torch.autograd.grad(out.float().square().sum(), of, create_graph=True)
    sum(g.float().square().sum() for g in first).backward()


@pytest.mark.parametrize("keep", [False, True])
def test_gated_recurrence_block(keep):
    torch.manual_seed(0)
    block = load("gated_recurrence_block").Block(24, 40, 3, keep=keep, dtype=torch.float32)
    tokens = torch.randn(2, 30, 24, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        twice(block, block(tokens), tokens)


def test_linear_attention_block():
    torch.manual_seed(0)
    m = load("linear_attention_block")
    block, tokens = m.Block(64, heads=2, kheads=1, head_dim=32, dtype=torch.float32), torch.randn(1, 30, 64, device="cuda", requires_grad=True)
    residual = torch.randn(1, 30, 64, device="cuda", requires_grad=True)
    positions = torch.rand(30, 2, device="cuda")
    with pytest.raises(RuntimeError, match="differentiate twice"):
        twice(block, block(tokens, residual, positions)[0], tokens, residual)
