"""The gated recurrence block's dense outputs past 2^31 elements, and batch rows more than 2^31 elements apart.

All batch rows are one (a batch stride of 0): the last row, whose elements lie past 2^31, has the first one's bits, and the
first one those of a call of its own."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, T, DIM = 3, 180001, 4096  # the last row: elements 1.5e9 to 2.2e9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def rows(*seeds):
    out = []
    for s in seeds:
        gen = torch.Generator(device="cuda").manual_seed(s)
        base = torch.randn(1, 1000, DIM, device="cuda", generator=gen).bfloat16()
        out.append(base.repeat(1, -(-T // 1000), 1)[:, :T])
    return out


def same(big, one):
    assert big.numel() > 1 << 31
    axis = big.dim() - 3  # kept planes stand before the batch
    for row in (0, B - 1):
        got = big.select(axis, row)
        want = one.select(axis, 0)
        kind = {1: torch.uint8, 2: torch.int16}[got.element_size()]
        for t in range(0, T, 20000):  # (a part at a time)
            assert torch.equal(got.narrow(-2, t, min(20000, T - t)).view(kind), want.narrow(-2, t, min(20000, T - t)).view(kind)), (row, t)


def test_group_norm():
    import selective_state_space_41_amd as V
    x, dy = rows(1, 2)
    w, b = torch.rand(DIM, device="cuda"), torch.rand(DIM, device="cuda")
    one = V.groupnorm_fwd(x, w, b, 32, keep=True)
    # a run's place and length follow the batch: another call's sums are joined in other places, so its bits may differ
    y, mean, rstd, kept = V.groupnorm_fwd(x.expand(B, T, DIM), w, b, 32, keep=True)
    assert y.numel() > 1 << 31 and torch.equal(mean[0], mean[-1]) and torch.equal(rstd[0], rstd[-1])
    same(y, y[:1])
    same(kept[0], one[3][0])
    assert torch.equal(kept[1][-1], one[3][1][0])
    assert (mean[0] - one[1][0]).abs().max() <= 40 * 2.0 ** -24 * x.abs().max() and (rstd[0] / one[2][0] - 1).abs().max() <= 100 * 2.0 ** -24
    for t in (0, T - 5):
        d = (y[-1, t:t + 5].float() - one[0][0, t:t + 5].float()).abs()
        assert (d <= 2.0 ** -7 * one[0][0, t:t + 5].float().abs() + 1e-5).all()
    dys = dy.expand(B, T, DIM)
    del y, one
    for form in (x.expand(B, T, DIM), kept):
        g = V.groupnorm_bwd(dys, form, w, b, mean, rstd)
        same(g["dx"], g["dx"][:1])
        first = V.groupnorm_bwd(dy, x if form is not kept else tuple(t[:1].contiguous() for t in kept), w, b, mean[:1].contiguous(),
                                rstd[:1].contiguous())
        d = (g["dx"][-1, -50:].float() - first["dx"][0, -50:].float()).abs()
        assert (d <= 2.0 ** -7 * first["dx"][0, -50:].float().abs() + 1e-5).all()
        del g, first


def test_gated_scan():
    import selective_state_space_41_amd as V
    x, r, i, d = rows(3, 4, 5, 6)
    A = torch.linspace(-7.0, 1.0, DIM, device="cuda")
    far = lambda t: t.expand(B, T, DIM)
    one = V.gated_scan_fwd(x, r, i, A, keep=True)
    out, last, kept = V.gated_scan_fwd(far(x), far(r), far(i), A, keep=True)
    same(out, one[0])
    same(kept[0], one[2][0])
    assert torch.equal(last[0], one[1][0]) and torch.equal(last[-1], one[1][0]) and torch.equal(kept[1][:, -1], one[2][1][:, 0])
    for reverse in (False, True):
        g1 = V.gated_scan_bwd((x, r, i, one[0]), A, d, reverse=reverse)
        g = V.gated_scan_bwd((far(x), far(r), far(i), out), A, far(d), reverse=reverse)
        for k in ("dx", "dr", "di"):
            same(g[k], g1[k])
        del g, g1
    g1, g = V.gated_scan_bwd(one[2], A, d), V.gated_scan_bwd(kept, A, far(d))
    for k in ("dx", "dr", "di"):
        same(g[k], g1[k])


def test_rows_apart():
    """Batch strides of 2^31 + 24 elements, and the 8-bit form of more than 2^31 elements."""
    import selective_state_space_41_amd as V
    torch.manual_seed(7)
    nb, L, dim, apart = 2, 300, 40, (1 << 31) + 24
    big = torch.empty(apart + 4 * L * dim, dtype=torch.bfloat16, device="cuda")
    views = [big.as_strided((nb, L, dim), (apart, dim, 1), k * L * dim) for k in range(4)]
    near = [torch.randn(nb, L, dim, device="cuda").bfloat16() for _ in range(4)]
    for v, c in zip(views, near):
        v.copy_(c)
    A = torch.linspace(-5.0, 0.0, dim, device="cuda")
    a, c = V.gated_scan_fwd(*views[:3], A), V.gated_scan_fwd(*near[:3], A)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    g, h = V.gated_scan_bwd((*views[:3], c[0]), A, views[3]), V.gated_scan_bwd((*near[:3], c[0]), A, near[3])
    assert all(torch.equal(g[k], h[k]) for k in g if g[k] is not None)
    a, c = V.groupnorm_fwd(views[0], A.exp(), A, 5), V.groupnorm_fwd(near[0], A.exp(), A, 5)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], c[:3]))
    g, h = (V.groupnorm_bwd(d, x, A.exp(), A, c[1], c[2]) for d, x in ((views[3], views[0]), (near[3], near[0])))
    assert all(torch.equal(g[k], h[k]) for k in g)
    del big, views
    rows, dim = 1 << 21, 1032
    x = torch.randn(1 << 11, dim, device="cuda").bfloat16()
    codes, scale = V.act8_pack(x.repeat(rows >> 11, 1))
    want, ws = V.act8_pack(x)
    assert codes.numel() > 1 << 31 and torch.equal(codes[-2048:].view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale[-2048:], ws)
    back = V.act8_unpack(codes, scale)
    assert torch.equal(back[-2048:], V.act8_unpack(want, ws))
