"""Linear attention of bfloat16 activations computes in float32: what its products lose beside the outputs' own rounding.

The operands that are not activations (the state, its gradient, the masked scores and their gradients) enter
the bfloat16 matrix products in pieces that hold all 24 bits of a float32 number, so that the arithmetic is float32's. That does not
show where an output is as large as its terms: there its rounding to bfloat16 hides everything below 2^-9. So the terms
here cancel, in pairs that differ by 2^-12 of themselves.

Tolerance of a whole output, in the 2-norm: |y - r| <= 2^-9 |r| + SUM 2^-24 |m|, with m the sums of the terms'
magnitudes. 2^-9: half a unit in the last place of 8 bits. SUM: a float32 sum of n terms of random signs passes partial sums
of the size sqrt(n) of a term, each rounded to 2^-25 of itself in the mean, which adds up to 2^-25 |m| in the root mean square; twice that,
because a matrix instruction may cut instead of round, is 1. That is it for states. A score is a sum of products itself, whose last
few partial sums have its size: 1 for each of up to 3 instructions and the factor 2^(decays), rounded too; SUM = 4.
|m| / |r| is between 2^13 and 2^15, which makes the room up to 0.004, where operands of 16 bits (two pieces) are off by about
2^-18 / sqrt(12) sqrt(2 / n) of m: 0.008 to 0.02 of r.

The results that stay float32 (states, their gradient, the decays' gradient) are held to 2^-21 and, for the decays, whose terms
partly cancel, 2^-20 of their norm: about 20 additions of 2^-25 in the mean, and the decays' exponentials, 2^-24."""
import numpy as np
import pytest
import torch

import synth
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu

SIZES = [(32, 64), (64, 64), (64, 128), (128, 64), (128, 128), (24, 40), (96, 104)]
NEAR = 2.0 ** -12


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def act(a):
    return synth.round_bf16(np.asarray(a, np.float32))


def td(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)


def near(name, y, r, m, terms):
    y = y.double().cpu().numpy()
    assert y.shape == r.shape and np.all(np.isfinite(y)), name
    norm = np.linalg.norm
    room = 2.0 ** -9 * norm(r) + terms * 2.0 ** -24 * norm(m)
    off = norm(y - r)
    print(f"[linattn precision] {name}: {off / norm(r):.5f} of the norm, {off / room:.3f} of the tolerance; terms 2^"
          f"{np.log2(norm(m) / norm(r)):.1f}", flush=True)
    assert off <= room, f"{name}: {off / room:.2f} times the tolerance"


def cancelling_states(rng, shape):
    """Neighbouring rows, and neighbouring columns, opposite but for 2^-12 of themselves."""
    s = np.repeat(np.repeat(rng.standard_normal(shape[:-2] + (shape[-2] // 2, shape[-1] // 2)), 2, -1), 2, -2)
    s *= 1 + NEAR * rng.standard_normal(shape)
    s[..., 1::2, :] *= -1
    s[..., 1::2] *= -1
    return s.astype(np.float32)


def paired(rng, *shape):
    return act(np.repeat(rng.standard_normal(shape[:-1] + (shape[-1] // 2,)), 2, -1))


@pytest.mark.parametrize("dk,dv", SIZES)
def test_states(dk, dv):
    """S in out and dq, the gradient R of the final state in dk and dv; no decay, nothing from the tokens themselves."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(dk + dv)
    B, T, H = 2, 21, 2
    s0, dsT = cancelling_states(rng, (B, H, dk, dv)), cancelling_states(rng, (B, H, dk, dv))
    q, k, v, do = (paired(rng, B, T, H, d) for d in (dk, dk, dv, dv))
    zk, zv, g = np.zeros_like(k), np.zeros_like(v), np.zeros((B, T, H), np.float32)
    t32 = lambda a: td(a, torch.float32)
    print(f"[linattn precision] states {dk} x {dv}", flush=True)
    out, _ = V.linattn_fwd(td(q), td(zk), td(zv), t32(g), scale=1.0, initial_state=t32(s0))
    a = np.abs
    near("out", out, np.einsum("bthi,bhij->bthj", q.astype(float), s0), np.einsum("bthi,bhij->bthj", a(q), a(s0)), 1)
    grads = V.linattn_bwd(td(q), td(zk), td(zv), t32(g), td(do), scale=1.0, initial_state=t32(s0))
    near("dq", grads["dq"], np.einsum("bthj,bhij->bthi", do.astype(float), s0), np.einsum("bthj,bhij->bthi", a(do), a(s0)), 1)
    grads = V.linattn_bwd(td(zk), td(k), td(v), t32(g), td(zv), scale=1.0, dfinal_state=t32(dsT))
    near("dk", grads["dk"], np.einsum("bthj,bhij->bthi", v.astype(float), dsT), np.einsum("bthj,bhij->bthi", a(v), a(dsT)), 1)
    near("dv", grads["dv"], np.einsum("bthi,bhij->bthj", k.astype(float), dsT), np.einsum("bthi,bhij->bthj", a(k), a(dsT)), 1)


def twins(rng, B, T, H, d):
    """Tokens in pairs that agree but in the last quarter of their channels, which is small."""
    x = np.repeat(rng.standard_normal((B, T // 2, H, d)), 2, 1)
    x[..., -(d // 4):] = 2 * NEAR * rng.standard_normal((B, T, H, d // 4))
    return act(x)


def opposite(rng, B, T, H, d):
    x = np.repeat(rng.standard_normal((B, T // 2, H, d)), 2, 1)
    x[:, 1::2] *= -1
    return act(x)


@pytest.mark.parametrize("dk,dv", SIZES)
def test_scores(dk, dv):
    """P in out (odd tokens see whole pairs of keys) and dv (even keys whole pairs of queries), X in dq and dk."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(dk * dv)
    B, T, H = 2, 18, 2
    g = np.zeros((B, T, H), np.float32)
    seen = np.tril(np.ones((T, T)))
    odd, even = slice(1, None, 2), slice(0, None, 2)

    def scores(x, y):  # [b, h, i, j], and their magnitudes
        p = np.einsum("bihd,bjhd->bhij", x.astype(float), y) * seen
        return p, np.abs(p)

    print(f"[linattn precision] scores {dk} x {dv}", flush=True)
    any_ = lambda d: act(rng.standard_normal((B, T, H, d)))
    sums = lambda w, x: np.einsum("bhij,bjhd->bihd", w, x)
    back = lambda w, x: np.einsum("bhij,bihd->bjhd", w, x)
    t32 = td(g, torch.float32)
    q, k, v = any_(dk), twins(rng, B, T, H, dk), opposite(rng, B, T, H, dv)
    p = scores(q, k)
    out, _ = V.linattn_fwd(td(q), td(k), td(v), t32, scale=1.0)
    near("out", out[:, odd], sums(p[0], v)[:, odd], sums(p[1], np.abs(v))[:, odd], 4)
    q, k, do = twins(rng, B, T, H, dk), any_(dk), opposite(rng, B, T, H, dv)
    p = scores(q, k)
    grads = V.linattn_bwd(td(q), td(k), td(any_(dv)), t32, td(do), scale=1.0)
    near("dv", grads["dv"][:, even], back(p[0], do)[:, even], back(p[1], np.abs(do))[:, even], 4)
    do, v, k = any_(dv), twins(rng, B, T, H, dv), opposite(rng, B, T, H, dk)
    x = scores(do, v)
    grads = V.linattn_bwd(td(any_(dk)), td(k), td(v), t32, td(do), scale=1.0)
    near("dq", grads["dq"][:, odd], sums(x[0], k)[:, odd], sums(x[1], np.abs(k))[:, odd], 4)
    do, v, q = twins(rng, B, T, H, dv), any_(dv), opposite(rng, B, T, H, dk)
    x = scores(do, v)
    grads = V.linattn_bwd(td(q), td(any_(dk)), td(v), t32, td(do), scale=1.0)
    near("dk", grads["dk"][:, even], back(x[0], q)[:, even], back(x[1], np.abs(q))[:, even], 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", SIZES)
def test_float32_results(dk, dv, dtype):
    """The norm of what states, their gradient and the decays' gradient are off by."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(dk + 2 * dv)
    B, T, H, Hk = 2, 150, 2, 1
    rnd = act if dtype == "bf16" else (lambda a: a.astype(np.float32))
    to = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k = rnd(rng.standard_normal((B, T, Hk, dk))), rnd(rng.standard_normal((B, T, Hk, dk)))
    v, do = rnd(rng.standard_normal((B, T, H, dv))), rnd(rng.standard_normal((B, T, H, dv)))
    g = -np.exp(rng.uniform(np.log(1e-3), np.log(0.3), (B, T, H))).astype(np.float32)
    s0, dsT = rng.standard_normal((2, B, H, dk, dv)).astype(np.float32)
    scale = dk ** -0.5
    t32 = lambda a: td(a, torch.float32)
    print(f"[linattn precision] float32 results {dk} x {dv} {dtype}", flush=True)
    _, sT = V.linattn_fwd(td(q, to), td(k, to), td(v, to), t32(g), scale=scale, initial_state=t32(s0))
    grads = V.linattn_bwd(td(q, to), td(k, to), td(v, to), t32(g), td(do, to), scale=scale, initial_state=t32(s0),
                          dfinal_state=t32(dsT))
    r_sT = BO.linattn(q, k, v, g, scale, s0)[1]
    r = BO.linattn_bwd(q, k, v, g, do, scale, s0, None, dsT)
    for name, y, want, most in (("final_state", sT, r_sT, 2.0 ** -21), ("dinitial_state", grads["dinitial_state"], r["ds0"], 2.0 ** -21),
                                ("dlog_decay", grads["dlog_decay"], r["dg"], 2.0 ** -20)):
        off = np.linalg.norm(y.double().cpu().numpy() - want) / np.linalg.norm(want)
        print(f"[linattn precision] {name}: {off:.2e} of the norm", flush=True)
        assert off <= most, f"{name}: {off:.2e} of the norm"
