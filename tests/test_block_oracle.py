"""The linear-attention block's oracle against closed forms and finite differences (CPU, float64)."""
import numpy as np
import pytest

from oracle import block_oracle as BO


def _inputs(rng, B=2, T=7, H=4, Hk=2, dk=3, dv=5, per_head=False):
    q, k = rng.standard_normal((2, B, T, Hk, dk))
    v, dout = rng.standard_normal((2, B, T, H, dv))
    g = -rng.random((H,) if per_head else (B, T, H))
    s0, dsT = rng.standard_normal((2, B, H, dk, dv))
    return q, k, v, g, dout, s0, dsT


def test_linattn_quadratic_form():
    """The recurrence equals the masked quadratic form with the decays between two tokens."""
    rng = np.random.default_rng(0)
    q, k, v, g, _, s0, _ = _inputs(rng)
    out, sT = BO.linattn(q, k, v, g, 0.5, s0)
    G = np.cumsum(g, axis=1)
    for b in range(2):
        for h in range(4):
            for i in range(7):
                want = np.exp(G[b, i, h]) * q[b, i, h // 2] @ s0[b, h]
                for j in range(i + 1):
                    want = want + np.exp(G[b, i, h] - G[b, j, h]) * (q[b, i, h // 2] @ k[b, j, h // 2]) * v[b, j, h]
                np.testing.assert_allclose(out[b, i, h], 0.5 * want, rtol=1e-11, atol=1e-12)
    # the state: one sequence after the other
    first = BO.linattn(q[:, :3], k[:, :3], v[:, :3], g[:, :3], 0.5, s0)[1]
    np.testing.assert_allclose(BO.linattn(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:], 0.5, first)[1], sT, rtol=1e-12)


def test_linattn_lengths_and_clearing():
    rng = np.random.default_rng(1)
    q, k, v, g, _, s0, _ = _inputs(rng)
    out, sT = BO.linattn(q, k, v, g, 1.0, s0, lengths=[0, 4])
    assert np.all(out[0] == 0) and np.array_equal(sT[0], s0[0]) and np.all(out[1, 4:] == 0)
    np.testing.assert_allclose(sT[1], BO.linattn(q[1:, :4], k[1:, :4], v[1:, :4], g[1:, :4], 1.0, s0[1:])[1][0])
    g[:, 3] = -np.inf  # the state forgets what came before token 3
    np.testing.assert_allclose(BO.linattn(q, k, v, g, 1.0, s0)[0][:, 3:],
                               BO.linattn(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:], 1.0)[0])


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("lengths", [None, [3, 7]])
def test_linattn_bwd_differences(per_head, lengths):
    rng = np.random.default_rng(2)
    q, k, v, g, dout, s0, dsT = _inputs(rng, per_head=per_head)
    grads = BO.linattn_bwd(q, k, v, g, dout, 0.7, s0, lengths, dsT)

    def loss(q, k, v, g, s0):
        out, sT = BO.linattn(q, k, v, g, 0.7, s0, lengths)
        return np.sum(out * dout) + np.sum(sT * dsT)

    args = [q, k, v, g, s0]
    for n, name in enumerate(("dq", "dk", "dv", "dg", "ds0")):
        step = rng.standard_normal(args[n].shape)
        eps = 1e-5
        hi, lo = ([a + s * eps * step if i == n else a for i, a in enumerate(args)] for s in (1, -1))
        want = (loss(*hi) - loss(*lo)) / (2 * eps)
        np.testing.assert_allclose(np.sum(grads[name] * step), want, rtol=1e-7, atol=1e-8, err_msg=name)


def test_linattn_step_is_the_recurrence():
    rng = np.random.default_rng(3)
    q, k, v, g, _, s0, _ = _inputs(rng, T=3)
    state = s0
    for t in range(3):
        o, state = BO.linattn_step(q[:, t], k[:, t], v[:, t], g[:, t], state, 0.5)
        np.testing.assert_allclose(o, BO.linattn(q, k, v, g, 0.5, s0)[0][:, t])
    # a pool: the second sequence's state lies first, the first row has none
    o, pool = BO.linattn_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], s0, 0.5, slots=[-1, 0])
    assert np.all(o[0] == 0) and np.array_equal(pool[1], s0[1]) and not np.array_equal(pool[0], s0[0])


def test_rmsnorm_bwd_differences():
    rng = np.random.default_rng(4)
    x, res, dy, dres = rng.standard_normal((4, 3, 9))
    w = rng.standard_normal(9)
    _, r, rstd = BO.rmsnorm(x, w, res, 1e-3)
    dr, dw = BO.rmsnorm_bwd(dy, r, w, rstd, dres)

    def loss(x, w):
        y, r, _ = BO.rmsnorm(x, w, res, 1e-3)
        return np.sum(y * dy) + np.sum(r * dres)

    for grad, at in ((dr, 0), (dw, 1)):
        step, eps = rng.standard_normal((x, w)[at].shape), 1e-5
        hi, lo = ([a + s * eps * step if i == at else a for i, a in enumerate((x, w))] for s in (1, -1))
        np.testing.assert_allclose(np.sum(grad * step), (loss(*hi) - loss(*lo)) / (2 * eps), rtol=1e-8)
    np.testing.assert_allclose(np.mean(BO.rmsnorm(x, np.ones(9), None, 0.0)[0] ** 2, axis=1), 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_axes(interleaved):
    """Length kept, the inverse undoes it, and scores depend on differences of positions only."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((1, 6, 1, 10))
    f, axis = np.array([1.0, 0.3, 0.5, 0.1]), [0, 0, 1, 7]
    pos = rng.integers(0, 50, (6, 2)).astype(float)
    y = BO.rope_axes(x, pos, f, axis, interleaved)
    np.testing.assert_allclose(np.sum(y * y, -1), np.sum(x * x, -1))
    np.testing.assert_allclose(BO.rope_axes(y, pos, f, axis, interleaved, inverse=True), x, atol=1e-12)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.array_equal(y[..., [6, 7] if interleaved else [3, 7]], x[..., [6, 7] if interleaved else [3, 7]])
    z = BO.rope_axes(x, pos + np.array([5.0, -3.0]), f, axis, interleaved)
    np.testing.assert_allclose(np.einsum("btha,bsha->ts", z, z), np.einsum("btha,bsha->ts", y, y), atol=1e-10)
