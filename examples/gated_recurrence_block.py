"""A gated recurrence block over image tokens, put together from the library's operators: group norm with SiLU on
channels-last tokens, projections, the gated linear recurrence walked in both directions, and training that keeps what
the gradients need in 8 bits.

    python examples/gated_recurrence_block.py            # a training step with activations whole and in 8 bits, then tokens

Training goes through torch's autograd: each operator's (first) gradient is the library's.  A block of one direction also
serves: a prompt leaves one float32 state per channel in a pool, and tokens are added one by one.  The projections are
torch's matrix products.
"""
import argparse
import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_41_amd as V  # noqa: E402


class GroupNormSiLU(torch.autograd.Function):
    """silu(group norm of x); with ``keep`` the gradient reads an 8-bit copy of x instead of x."""

    @staticmethod
    def forward(ctx, x, weight, bias, groups, lengths, keep):
        y, mean, rstd, kept = V.groupnorm_fwd(x, weight, bias, groups, lengths=lengths, keep=keep)
        ctx.save_for_backward(weight, bias, mean, rstd, *(kept if keep else (x,)))
        ctx.lengths = lengths
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, bias, mean, rstd, *kept = ctx.saved_tensors
        g = V.groupnorm_bwd(dy.contiguous(), tuple(kept) if len(kept) == 2 else kept[0], weight, bias, mean, rstd,
                            lengths=ctx.lengths)
        return g["dx"], g["dweight"], g["dbias"], None, None, None


class GatedScan(torch.autograd.Function):
    """The recurrence's states; with ``keep`` the gradient reads 8-bit copies of x, r, i and the states."""

    @staticmethod
    def forward(ctx, x, r, i, A_log, lengths, reverse, keep):
        h, _, kept = V.gated_scan_fwd(x, r, i, A_log, lengths=lengths, reverse=reverse, keep=keep)
        ctx.save_for_backward(A_log, *(kept if keep else (x, r, i, h)))
        ctx.lengths, ctx.reverse = lengths, reverse
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        A_log, *kept = ctx.saved_tensors
        g = V.gated_scan_bwd(tuple(kept), A_log, dh.contiguous(), lengths=ctx.lengths, reverse=ctx.reverse)
        return g["dx"], g["dr"], g["di"], g["dA_log"], None, None, None


class Block(torch.nn.Module):
    """inner channels of state for each of one or two directions; ``keep``: what the gradients need is kept in 8 bits."""

    def __init__(self, dim, inner, groups, both=True, keep=False, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.inner, self.groups, self.ways, self.keep = inner, groups, 2 if both else 1, keep
        init = lambda *s: torch.nn.Parameter((torch.randn(*s, device=device) / math.sqrt(s[-1])).to(dtype))
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device))
        self.xri, self.out = init(3 * self.ways * inner, dim), init(dim, inner)
        # decays at a full gate from exp(-0.001) to exp(-1)
        self.A_log = torch.nn.Parameter(torch.linspace(math.log(1e-3), 0.0, inner, device=device).repeat(self.ways, 1))

    def _project(self, y):
        """[..., dim] -> per direction (x, r, i), slices of one product."""
        return (y @ self.xri.t()).unflatten(-1, (self.ways, 3, self.inner)).flatten(-3).split(self.inner, -1)

    def forward(self, tokens, lengths=None):
        """tokens: [batch, L, dim], rows of ``lengths`` tokens; returns tokens plus the block's output."""
        y = GroupNormSiLU.apply(tokens, self.weight, self.bias, self.groups, lengths, self.keep)
        parts = self._project(y)
        h = sum(GatedScan.apply(*parts[3 * w:3 * w + 3], self.A_log[w].contiguous(), lengths, bool(w), self.keep)
                for w in range(self.ways)) / self.ways
        return tokens + h @ self.out.t()

    @torch.no_grad()
    def scan(self, y, state=None):
        """Normalised tokens [batch, L, dim] of a block of one direction, from and to a state: (output, state)."""
        h, state, _ = V.gated_scan_fwd(*self._project(y), self.A_log[0], initial_state=state)
        return h @ self.out.t(), state

    @torch.no_grad()
    def token(self, y, pool, slots):
        """One normalised token of each sequence: y [batch, dim]; updates the sequences' states in the pool."""
        return V.gated_scan_step(*self._project(y), self.A_log[0], pool, slots=slots) @ self.out.t()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--side", type=int, default=28, help="tokens along an image's side")
    a = ap.parse_args()
    torch.manual_seed(0)
    dim, L = 192, a.side * a.side
    block = Block(dim, inner=384, groups=6)
    image = torch.randn(a.batch, L, dim, device="cuda").bfloat16()
    grads = {}
    for keep in (False, True):
        block.keep = keep
        block.zero_grad()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        loss = block(image).float().square().mean()
        held = torch.cuda.memory_allocated() - before
        loss.backward()
        grads[keep] = {n: p.grad.float().clone() for n, p in block.named_parameters()}
        print(f"training step, activations {'in 8 bits' if keep else 'whole'}: {a.batch} x {L} tokens, loss {loss.item():.4f}, "
              f"{held / 2 ** 20:.1f} MiB held for the gradients")
    print("gradients from 8 bits off by " + ", ".join(
        f"{n} {((grads[True][n] - g).norm() / g.norm()).item():.3f}" for n, g in grads[False].items()))

    # one direction: a prompt of all but the last 5 tokens, then those one by one, against the whole sequence
    block = Block(dim, inner=384, groups=6, both=False)
    y = V.groupnorm_fwd(image, block.weight.detach(), block.bias.detach(), 6)[0]
    whole, last = block.scan(y)
    _, state = block.scan(y[:, :L - 5])
    pool = torch.zeros(a.batch + 3, 384, device="cuda")
    slots = torch.randperm(a.batch + 3, device="cuda")[:a.batch].to(torch.int32)
    pool[slots.long()] = state
    worst = max((block.token(y[:, t], pool, slots) - whole[:, t]).float().abs().max().item() for t in range(L - 5, L))
    off = (pool[slots.long()] - last).abs().max().item()
    print(f"prompt of {L - 5} tokens, then 5 single ones: outputs within {worst:.3g}, states within {off:.3g} of the whole "
          "sequence's")


if __name__ == "__main__":
    main()
