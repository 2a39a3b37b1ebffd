"""Edges of the gated block's operators on the GPU: the wait status word, rows without tokens under eps = 0, a channel per
group at the widest, and inputs that are broadcast views."""
import numpy as np
import pytest
import torch

import test_gpu_gated_scan as S
import test_gpu_groupnorm as N
from oracle import gated_oracle as GO

pytestmark = pytest.mark.gpu
U = GO.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


@pytest.mark.parametrize("B,T,dim", [(1, 129, 3), (2, 1100, 130), (3, 9000, 64)])
def test_status_word(B, T, dim):
    """A workspace of any contents: the word reads 0 after the call, and the results are those of any other workspace."""
    import selective_state_space_41_amd as V
    p = S.make(B, T, dim, "f32", T)
    x, r, i, a, dout = (S.td(p[k]) for k in ("x", "r", "i", "A_log", "dout"))
    word = lambda ws: int(ws[:4].cpu().numpy().view(np.int32)[0])
    ws = torch.full((V.lib.vmscan_gated_scan_fwd_workspace_bytes(B, T, dim),), 255, dtype=torch.uint8, device="cuda")
    out, last, _ = V.gated_scan_fwd(x, r, i, a, workspace=ws)
    assert word(ws) == 0
    out2, last2, _ = V.gated_scan_fwd(x, r, i, a)
    assert torch.equal(out, out2) and torch.equal(last, last2)
    wb = torch.full((V.lib.vmscan_gated_scan_bwd_workspace_bytes(B, T, dim),), 255, dtype=torch.uint8, device="cuda")
    g = V.gated_scan_bwd((x, r, i, out), a, dout, workspace=wb)
    assert word(wb) == 0
    g2 = V.gated_scan_bwd((x, r, i, out), a, dout)
    assert all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)


@pytest.mark.parametrize("B,T,dim,groups", [(2, 5, 16, 2), (2, 7, 12, 4), (2, 3000, 48, 6)], ids=["slab", "narrow", "runs"])
@pytest.mark.parametrize("codes", [False, True])
def test_a_row_without_tokens_under_no_eps(B, T, dim, groups, codes):
    """Its reciprocal deviation is infinite and has no share in any gradient."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(T)
    x, dy = (rng.standard_normal((B, T, dim)).astype(np.float32) for _ in range(2))
    w, b = (rng.standard_normal(dim).astype(np.float32) for _ in range(2))
    lengths = [0] + [T - 1] * (B - 1)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, mean, rstd, kept = V.groupnorm_fwd(N.td(x), N.td(w), N.td(b), groups, eps=0.0, lengths=n, keep=codes)
    assert not y[0].any() and torch.isfinite(y).all() and torch.isinf(rstd[0]).all()
    g = V.groupnorm_bwd(N.td(dy), kept if codes else N.td(x), N.td(w), N.td(b), mean, rstd, lengths=n)
    one = V.groupnorm_bwd(N.td(dy[1:]), tuple(t[1:].contiguous() for t in kept) if codes else N.td(x[1:]), N.td(w), N.td(b),
                          mean[1:].contiguous(), rstd[1:].contiguous(), lengths=n[1:].contiguous())
    assert not g["dx"][0].any() and torch.equal(g["dx"][1:], one["dx"])
    xs = x[1:] if not codes else kept[0][1:].float().cpu().numpy() * GO.act8_spread(kept[1][1:].cpu().numpy(), dim)
    (_, dw, db), (_, mw, mb) = GO.groupnorm_bwd(dy[1:], xs, w, b, mean[1:].cpu().numpy(), rstd[1:].cpu().numpy(), True, lengths[1:])
    N.near("dweight", g["dweight"], dw, (120 + B * T / 64) * U * mw)
    N.near("dbias", g["dbias"], db, (120 + B * T / 64) * U * mb)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 1100], ids=["slab", "runs"])
def test_a_channel_per_group_at_the_widest(T, dtype):
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(T)
    B, dim = 1, 4096
    x, dy = (N.rnd(rng.standard_normal((B, T, dim)), dtype) for _ in range(2))
    w, b = (rng.standard_normal(dim).astype(np.float32) for _ in range(2))
    y, mean, rstd, _ = V.groupnorm_fwd(N.td(x, dtype), N.td(w), N.td(b), dim)
    ry, rmean, rrstd = GO.groupnorm(x, w, b, dim)
    tm, tr, ty = N.forward_rooms(x, w, b, dim, rmean, rrstd, True, None, 1e-5)
    N.near("mean", mean, rmean, tm)
    N.near("rstd", rstd, rrstd, tr)
    N.near("y", y, ry, ty + N.unit(dtype) * np.abs(ry))
    g = V.groupnorm_bwd(N.td(dy, dtype), N.td(x, dtype), N.td(w), N.td(b), mean, rstd)
    (dx, dw, db), (mx, mw, mb) = GO.groupnorm_bwd(dy, x, w, b, mean.cpu().numpy(), rstd.cpu().numpy(), True, None)
    N.near("dx", g["dx"], dx, 120 * U * mx + N.unit(dtype) * np.abs(dx))
    N.near("dweight", g["dweight"], dw, (120 + T / 64) * U * mw)
    N.near("dbias", g["dbias"], db, (120 + T / 64) * U * mb)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dim", [7, 136])
def test_broadcast_inputs(dim, keep):
    """A gate that is one row for all tokens, one of all sequences and a gradient that is one row: strides of 0."""
    import selective_state_space_41_amd as V
    B, T = 3, 150
    p = S.make(B, T, dim, "bf16", dim)
    x = S.td(p["x"], "bf16")
    r = S.td(p["r"][:, :1], "bf16").expand(B, T, dim)
    i = S.td(p["i"][:1], "bf16").expand(B, T, dim)
    d = S.td(p["dout"][:1, :1], "bf16").expand(B, T, dim)
    a = S.td(p["A_log"])
    out, last, kept = V.gated_scan_fwd(x, r, i, a, keep=keep)
    out2, last2, kept2 = V.gated_scan_fwd(x, r.contiguous(), i.contiguous(), a, keep=keep)
    assert torch.equal(out, out2) and torch.equal(last, last2)
    if keep:
        assert torch.equal(kept[0].view(torch.uint8), kept2[0].view(torch.uint8)) and torch.equal(kept[1], kept2[1])
    g = V.gated_scan_bwd(kept or (x, r, i, out), a, d)
    g2 = V.gated_scan_bwd(kept or (x, r.contiguous(), i.contiguous(), out), a, d.contiguous())
    assert all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)
    y = V.groupnorm_fwd(i, a, a, 1, keep=keep)
    y2 = V.groupnorm_fwd(i.contiguous(), a, a, 1, keep=keep)
    assert torch.equal(y[0], y2[0]) and torch.equal(y[1], y2[1]) and torch.equal(y[2], y2[2])
    h = V.groupnorm_bwd(d, i, a, a, y[1], y[2])
    h2 = V.groupnorm_bwd(d.contiguous(), i.contiguous(), a, a, y[1], y[2])
    assert all(torch.equal(h[k], h2[k]) for k in h)


def test_many_rows():
    """More batch rows than a grid's second dimension holds: the rows of a large call are those of small ones."""
    import selective_state_space_41_amd as V
    B, T, dim = 70000, 3, 6
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, r, i, d = (torch.randn(B, T, dim, device="cuda", generator=gen) for _ in range(4))
    a, w = torch.randn(dim, device="cuda", generator=gen), torch.randn(dim, device="cuda", generator=gen)
    n = torch.randint(0, T + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
    first = torch.randn(B, dim, device="cuda", generator=gen)
    out, last, kept = V.gated_scan_fwd(x, r, i, a, initial_state=first, lengths=n, keep=True)
    g = V.gated_scan_bwd((x, r, i, out), a, d, initial_state=first, lengths=n, dfinal_state=first)
    few = slice(B - 5, B)
    sub = lambda t: t[few].contiguous()
    out2, last2, kept2 = V.gated_scan_fwd(sub(x), sub(r), sub(i), a, initial_state=sub(first), lengths=sub(n), keep=True)
    g2 = V.gated_scan_bwd((sub(x), sub(r), sub(i), out2), a, sub(d), initial_state=sub(first), lengths=sub(n), dfinal_state=sub(first))
    assert torch.equal(out[few], out2) and torch.equal(last[few], last2)
    assert torch.equal(kept[0][:, few].view(torch.uint8), kept2[0].view(torch.uint8)) and torch.equal(kept[1][:, few], kept2[1])
    assert all(torch.equal(g[k][few], g2[k]) for k in ("dx", "dr", "di", "dinitial_state"))
    x, d, n = x[:65535], d[:65535], n[:65535]
    y, mean, rstd, _ = V.groupnorm_fwd(x, w, a, 2, lengths=n)
    h = V.groupnorm_bwd(d, x, w, a, mean, rstd, lengths=n)
    few = slice(65530, 65535)
    y2, mean2, rstd2, _ = V.groupnorm_fwd(sub(x), w, a, 2, lengths=sub(n))
    h2 = V.groupnorm_bwd(sub(d), sub(x), w, a, mean2, rstd2, lengths=sub(n))
    assert torch.equal(y[few], y2) and torch.equal(mean[few], mean2) and torch.equal(h["dx"][few], h2["dx"])
    with pytest.raises(RuntimeError):
        V.groupnorm_fwd(out, w, a, 2)  # 70000 rows
    assert torch.equal(V.act8_unpack(*V.act8_pack(out), dtype=torch.float32)[few],
                       V.act8_unpack(*V.act8_pack(out[few]), dtype=torch.float32))
