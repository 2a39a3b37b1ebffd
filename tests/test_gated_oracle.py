"""The gated recurrence block's oracle against closed forms and finite differences (no GPU, no library)."""
import numpy as np
import pytest

from oracle import gated_oracle as GO


def test_sigmoid_and_decay_limits():
    assert GO.sigmoid(0.0) == 0.5 and GO.sigmoid(-1000.0) == 0.0 and GO.sigmoid(1000.0) == 1.0


def test_scan_is_a_weighted_sum():
    """h_t = sum over s <= t of (prod of a between) b_s: against the explicit lower-triangular matrix."""
    rng = np.random.default_rng(0)
    T, dim = 9, 3
    x, r, i = (rng.standard_normal((1, T, dim)) for _ in range(3))
    A_log, first = rng.standard_normal(dim), rng.standard_normal((1, dim))
    (h, last), _ = GO.gated_scan(x, r, i, A_log, first)
    a = np.exp(-np.exp(A_log) * GO.sigmoid(r[0]))
    b = np.sqrt(1 - a * a) * GO.sigmoid(i[0]) * x[0]
    for t in range(T):
        want = sum(np.prod(a[s + 1:t + 1], axis=0) * b[s] for s in range(t + 1)) + np.prod(a[:t + 1], axis=0) * first[0]
        assert np.allclose(h[0, t], want, rtol=1e-12, atol=1e-14)
    assert np.array_equal(last[0], h[0, -1])
    (hr, _), _ = GO.gated_scan(x[:, ::-1], r[:, ::-1], i[:, ::-1], A_log, first, reverse=True)
    assert np.allclose(hr[:, ::-1], h)
    (hn, ln), _ = GO.gated_scan(x, r, i, A_log, first, lengths=[4], reverse=True)
    (hs, ls), _ = GO.gated_scan(x[:, :4], r[:, :4], i[:, :4], A_log, first, reverse=True)
    assert np.array_equal(hn[:, :4], hs) and np.array_equal(ln, ls) and not hn[:, 4:].any()
    (he, le), _ = GO.gated_scan(x, r, i, A_log, first, lengths=[0])
    assert not he.any() and np.array_equal(le, first)


@pytest.mark.parametrize("reverse", [False, True])
def test_scan_gradient_against_differences(reverse):
    rng = np.random.default_rng(1)
    B, T, dim = 2, 6, 3
    p = dict(x=rng.standard_normal((B, T, dim)), r=rng.standard_normal((B, T, dim)), i=rng.standard_normal((B, T, dim)),
             A=rng.standard_normal(dim), first=rng.standard_normal((B, dim)))
    lengths, dout, dlast = [6, 4], rng.standard_normal((B, T, dim)), rng.standard_normal((B, dim))
    dout[1, 4:] = 0

    def loss(q):
        (h, last), _ = GO.gated_scan(q["x"], q["r"], q["i"], q["A"], q["first"], lengths, reverse)
        return (h * dout).sum() + (last * dlast).sum()

    (h, _), _ = GO.gated_scan(p["x"], p["r"], p["i"], p["A"], p["first"], lengths, reverse)
    g, _ = GO.gated_scan_bwd(p["x"], p["r"], p["i"], h, p["A"], dout, p["first"], lengths, reverse, dlast)
    for name, grad in (("x", g["dx"]), ("r", g["dr"]), ("i", g["di"]), ("A", g["dA"]), ("first", g["dfirst"])):
        for at in np.ndindex(p[name].shape):
            q = {k: v.copy() for k, v in p.items()}
            q[name][at] += 1e-6
            hi = loss(q)
            q[name][at] -= 2e-6
            assert abs((hi - loss(q)) / 2e-6 - grad[at]) < 1e-7, (name, at)


@pytest.mark.parametrize("act", [False, True])
def test_groupnorm_gradient_against_differences(act):
    rng = np.random.default_rng(2)
    B, T, dim, groups = 2, 5, 6, 2
    p = dict(x=rng.standard_normal((B, T, dim)) + 0.5, w=rng.standard_normal(dim), b=rng.standard_normal(dim))
    lengths, dy = [5, 3], rng.standard_normal((B, T, dim))
    loss = lambda q: (GO.groupnorm(q["x"], q["w"], q["b"], groups, act=act, lengths=lengths)[0] * dy).sum()
    y, mean, rstd = GO.groupnorm(p["x"], p["w"], p["b"], groups, act=act, lengths=lengths)
    assert not y[1, 3:].any()
    n = (p["x"][0].reshape(T, groups, 3) - mean[0][:, None]) * rstd[0][:, None]
    assert np.allclose(n.mean((0, 2)), 0, atol=1e-12) and np.allclose((n ** 2).mean((0, 2)), 1, rtol=1e-3)
    (dx, dw, db), _ = GO.groupnorm_bwd(dy, p["x"], p["w"], p["b"], mean, rstd, act, lengths)
    for name, grad in (("x", dx), ("w", dw), ("b", db)):
        for at in np.ndindex(p[name].shape):
            q = {k: v.copy() for k, v in p.items()}
            q[name][at] += 1e-6
            hi = loss(q)
            q[name][at] -= 2e-6
            assert abs((hi - loss(q)) / 2e-6 - grad[at]) < 1e-7, (name, at)


def test_step_is_the_scan_token_by_token():
    rng = np.random.default_rng(3)
    x, r, i = (rng.standard_normal((2, 4, 5)) for _ in range(3))
    A_log, first = rng.standard_normal(5), rng.standard_normal((3, 5))
    (h, last), _ = GO.gated_scan(x, r, i, A_log, first[[2, 0]])
    pool = first
    for t in range(4):
        out, pool = GO.gated_scan_step(x[:, t], r[:, t], i[:, t], A_log, pool, [2, 0])
        assert np.allclose(out, h[:, t], rtol=1e-13)
    assert np.allclose(pool[[2, 0]], last) and np.array_equal(pool[1], first[1])


def test_act8_scale():
    x = np.zeros((2, 130))
    x[0, 5], x[0, 129], x[1, 129] = -896.0, 2.0, 0.0
    assert np.allclose(GO.act8_scale(x), [[2.0, 2.0 / 448], [1.0, 1.0]])
    assert GO.act8_spread(GO.act8_scale(x), 130).shape == (2, 130)
