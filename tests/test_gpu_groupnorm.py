"""Group norm with its activation, and activations in 8 bits, on the GPU against the fp64 oracle.

Tolerances, from the operations (U = 2^-24):
  * a group's mean is a tree of a thread's differences to its first token: 40 U of the largest magnitude;
  * its deviation relative: a thread's sum of up to 64 squares, their tree, and twice the means' own rounding against the
    deviation: (80 + 8 |mean| / std) U;
  * y: that on each term, the difference x - mean (4 U of |x| and |mean|), the sigmoid (14 U), and the output's rounding;
  * gradient: each of the terms in float32: 120 U of their magnitudes and a share of the tokens' sums for dweight, dbias."""
import numpy as np
import pytest
import torch

import synth
from oracle import gated_oracle as GO

pytestmark = pytest.mark.gpu
U = GO.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def rnd(a, dtype):
    return synth.round_bf16(np.asarray(a, np.float32)) if dtype == "bf16" else np.asarray(a, np.float32)


def td(a, dtype="f32"):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def unit(dtype):
    return 2.0 ** -8 if dtype == "bf16" else U


def near(name, y, r, room):
    y = y.double().cpu().numpy()
    assert y.shape == r.shape and np.all(np.isfinite(y)), name
    used = float(np.max(np.abs(y - r) / (room + 1e-37)))
    print(f"[groupnorm] {name}: {used:.3f} of the tolerance", flush=True)
    assert used <= 1.0, f"{name}: {used:.2f} times the tolerance"


def forward_rooms(x, w, b, groups, mean, rstd, act, lengths, eps):
    B, T, dim = x.shape
    up = lambda a: np.repeat(a, dim // groups, axis=1)[:, None]
    top = np.zeros(mean.shape)
    for k in range(B):
        n = T if lengths is None else lengths[k]
        if n:
            top[k] = np.abs(x[k, :n].astype(np.float64)).reshape(n, groups, -1).max((0, 2))
    rm = 40 * U * top
    rel = (80 + 8 * np.abs(mean) * rstd) * U + 0.5 * (rm * rstd) ** 2
    rr = rel * rstd
    d = np.abs(x - up(mean))
    u = np.abs(d * up(rstd) * w + b)
    ru = np.abs(w) * up(rstd) * (d * (up(rel) + 4 * U) + up(rm) + 4 * U * (np.abs(x) + np.abs(up(mean)))) + 2 * U * (u + np.abs(b))
    return rm, rr, 1.1 * ru + (14 * U * u if act else 0.0)


# one channel a group, groups across 8-channel runs, one group, rows that fill 1 to 512 threads
CASES = [  # B, T, dim, groups, lengths
    (1, 1, 1, 1, None), (2, 3, 6, 2, None), (2, 50, 7, 7, [50, 1]), (2, 197, 64, 8, None), (3, 64, 100, 4, [64, 0, 33]),
    (1, 300, 96, 32, None), (2, 77, 384, 6, [77, 5]), (2, 197, 512, 32, None), (1, 33, 520, 1, None), (2, 20, 1030, 5, [20, 19]),
    (1, 9, 4096, 64, None), (1, 2500, 40, 5, [2411]), (1, 21, 2056, 257, None),
]


@pytest.mark.parametrize("act", [False, True], ids=["plain", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,dim,groups,lengths", CASES)
def test_groupnorm_and_gradient(B, T, dim, groups, lengths, dtype, act):
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(B * T + dim)
    x = rnd(1.5 * rng.standard_normal((B, T, dim)) + 0.5 * rng.standard_normal(dim), dtype)
    w, b = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32), (0.3 * rng.standard_normal(dim)).astype(np.float32)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    wide = torch.full((B, T, dim + 5), float("nan"), device="cuda", dtype=td(x, dtype).dtype)  # rows apart, odd places
    xt = wide[..., 3:3 + dim]
    xt.copy_(td(x, dtype))
    dy = rnd(rng.standard_normal((B, T, dim)), dtype)
    dyt = td(dy, dtype)
    for k, m in enumerate(lengths or []):  # never read
        xt[k, m:], dyt[k, m:] = float("nan"), float("nan")
    y, mean, rstd, kept = V.groupnorm_fwd(xt, td(w), td(b), groups, act=act, lengths=n)
    assert kept is None
    ry, rmean, rrstd = GO.groupnorm(x, w, b, groups, act=act, lengths=lengths)
    tm, tr, ty = forward_rooms(x, w, b, groups, rmean, rrstd, act, lengths, 1e-5)
    near("mean", mean, rmean, tm)
    near("rstd", rstd, rrstd, tr)
    near("y", y, ry, ty + unit(dtype) * np.abs(ry))

    m32, r32 = rmean.astype(np.float32), rrstd.astype(np.float32)
    g = V.groupnorm_bwd(dyt, xt, td(w), td(b), td(m32), td(r32), act=act, lengths=n)
    (dx, dw, db), (mx, mw, mb) = GO.groupnorm_bwd(dy, x, w, b, m32, r32, act, lengths)
    share = (120 + B * T / 64) * U
    near("dx", g["dx"], dx, 120 * U * mx + unit(dtype) * np.abs(dx))
    near("dweight", g["dweight"], dw, share * mw)
    near("dbias", g["dbias"], db, share * mb)
    again = V.groupnorm_bwd(dyt, xt, td(w), td(b), td(m32), td(r32), act=act, lengths=n)
    assert all(torch.equal(g[k], again[k]) for k in g)


def check_codes(codes, scale, v):
    s = GO.act8_scale(v)
    near("scale", scale, s, 4 * U * s)
    s = GO.act8_spread(scale.double().cpu().numpy(), v.shape[-1])
    # half a step: 2^-4 of a code, 2^-10 below the normal codes
    near("codes", codes.float(), v / s, (2.0 ** -4 + 8 * U) * np.abs(v / s) + 2.0 ** -10)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,dim,groups,lengths", [(1, 1, 1, 1, None), (2, 40, 100, 4, [40, 17]), (2, 197, 384, 6, None),
                                                    (1, 60, 1160, 8, None), (3, 130, 512, 32, [0, 130, 64])])
def test_groupnorm_kept_in_8_bits(B, T, dim, groups, lengths, dtype):
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(T + dim)
    x = rnd(rng.standard_normal((B, T, dim)) + 0.3, dtype)
    w, b = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32), (0.3 * rng.standard_normal(dim)).astype(np.float32)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, mean, rstd, kept = V.groupnorm_fwd(td(x, dtype), td(w), td(b), groups, lengths=n, keep=True)
    y2, mean2, rstd2, _ = V.groupnorm_fwd(td(x, dtype), td(w), td(b), groups, lengths=n)
    ry, rmean, rrstd = GO.groupnorm(x, w, b, groups, lengths=lengths)
    tm, tr, ty = forward_rooms(x, w, b, groups, rmean, rrstd, True, lengths, 1e-5)
    near("y", y, ry, ty + unit(dtype) * np.abs(ry))
    near("y without", y2, ry, ty + unit(dtype) * np.abs(ry))
    v = x.astype(np.float64)
    for k, m in enumerate(lengths or []):
        v[k, m:] = 0
    check_codes(*kept, v)
    dy = rnd(rng.standard_normal((B, T, dim)), dtype)
    g = V.groupnorm_bwd(td(dy, dtype), kept, td(w), td(b), mean, rstd, lengths=n)
    x8 = kept[0].float().double().cpu().numpy() * GO.act8_spread(kept[1].double().cpu().numpy(), dim)
    (dx, dw, db), (mx, mw, mb) = GO.groupnorm_bwd(dy, x8, w, b, mean.cpu().numpy(), rstd.cpu().numpy(), True, lengths)
    near("dx", g["dx"], dx, 120 * U * mx + unit(dtype) * np.abs(dx))
    near("dweight", g["dweight"], dw, (120 + B * T / 64) * U * mw)
    near("dbias", g["dbias"], db, (120 + B * T / 64) * U * mb)


def test_large_means_and_first_tokens():
    """A mean of 3000 deviations, and a first token 10^4 times the others: the deviation loses nothing to either."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 500, 64)).astype(np.float32)
    x[0] += 3000.0
    x[1, 0] *= 1e4
    w, b = np.ones(64, np.float32), np.zeros(64, np.float32)
    y, mean, rstd, _ = V.groupnorm_fwd(td(x), td(w), td(b), 4, act=False)
    ry, rmean, rrstd = GO.groupnorm(x, w, b, 4, act=False)
    tm, tr, ty = forward_rooms(x, w, b, 4, rmean, rrstd, False, None, 1e-5)
    near("mean", mean, rmean, tm)
    near("rstd", rstd, rrstd, tr)
    near("y", y, ry, ty + U * np.abs(ry))


def test_images_and_batches_on_another_stream():
    """[batch, H, W, dim] is [batch, H * W, dim]; a call on another stream."""
    import selective_state_space_41_amd as V
    x = torch.randn(3, 7, 9, 48, device="cuda").bfloat16()
    w, b = torch.rand(48, device="cuda"), torch.rand(48, device="cuda")
    y, mean, rstd, (codes, scale) = V.groupnorm_fwd(x, w, b, 6, keep=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, _, _, kept2 = V.groupnorm_fwd(x.view(3, 63, 48), w, b, 6, keep=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert y.shape == x.shape and codes.shape == x.shape and scale.shape == (3, 7, 9, 1)
    assert torch.equal(y.view(3, 63, 48), y2) and torch.equal(codes.view(3, 63, 48).float(), kept2[0].float())
    g = V.groupnorm_bwd(y, (codes, scale), w, b, mean, rstd)
    g2 = V.groupnorm_bwd(y2, kept2, w, b, mean, rstd)
    assert g["dx"].shape == x.shape and torch.equal(g["dx"].view(3, 63, 48), g2["dx"])


def test_nan_and_infinity_stay_in_their_group():
    import selective_state_space_41_amd as V
    x = torch.randn(2, 50, 32, device="cuda")
    w, b = torch.ones(32, device="cuda"), torch.zeros(32, device="cuda")
    clean = V.groupnorm_fwd(x, w, b, 4, act=False)[0]
    x[0, 3, 9], x[1, 7, 30] = float("nan"), float("inf")
    y, mean, rstd, _ = V.groupnorm_fwd(x, w, b, 4, act=False)
    bad = torch.zeros(2, 50, 32, dtype=torch.bool, device="cuda")
    bad[0, :, 8:16], bad[1, :, 24:] = True, True
    assert torch.isnan(y[0, :, 8:16]).all() and torch.isnan(y[1, :, 24:]).all() and torch.equal(y[~bad], clean[~bad])


def test_in_a_graph():
    import selective_state_space_41_amd as V
    x, dy = torch.randn(2, 900, 96, device="cuda"), torch.randn(2, 900, 96, device="cuda")
    w, b = torch.rand(96, device="cuda"), torch.rand(96, device="cuda")

    def both():
        y, mean, rstd, kept = V.groupnorm_fwd(x, w, b, 8, keep=True)
        return y, V.groupnorm_bwd(dy, kept, w, b, mean, rstd), V.groupnorm_bwd(dy, x, w, b, mean, rstd)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        x.normal_()
        dy.normal_()
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0])
        for p, q in zip(got[1:], want[1:]):
            assert all(torch.equal(p[k], q[k]) for k in p)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 128), (17, 130), (9, 384), (4, 2050), (1000, 72)])
def test_act8(rows, dim, dtype):
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(rows + dim)
    x = rnd(rng.standard_normal((rows, dim)) * np.exp(3 * rng.standard_normal((rows, 1))), dtype)
    x[0] = 0.0
    wide = torch.full((rows, dim + 3), float("nan"), device="cuda", dtype=td(x, dtype).dtype)
    wide[:, 2:2 + dim] = td(x, dtype)
    for t in (td(x, dtype), wide[:, 2:2 + dim]):
        codes, scale = V.act8_pack(t)
        check_codes(codes, scale, x.astype(np.float64))
        assert (codes[0].float() == 0).all() and (scale[0] == 1).all()
        back = V.act8_unpack(codes, scale, dtype=t.dtype)
        want = codes.float().double().cpu().numpy() * GO.act8_spread(scale.double().cpu().numpy(), dim)
        near("back", back, want, (U + unit(dtype)) * np.abs(want))


def test_act8_edges():
    """Equal to the norm's 8-bit form; tiny groups; a NaN or infinity makes its group NaN and no other."""
    import selective_state_space_41_amd as V
    x = torch.randn(40, 200, device="cuda")
    ones = torch.ones(200, device="cuda")
    codes, scale, _, _ = V.rmsnorm_fwd(x, ones, out_dtype=torch.float8_e4m3fn, group=128)
    y = V.rmsnorm_fwd(x, ones)[0]
    c2, s2 = V.act8_pack(y)
    assert torch.equal(codes.float(), c2.float()) and torch.equal(scale, s2)
    t = torch.full((2, 130), 1e-42, device="cuda")
    t[0, 3], t[1, 129] = float("nan"), float("inf")
    c, s = V.act8_pack(t)
    back = V.act8_unpack(c, s, dtype=torch.float32)
    assert torch.isnan(back[0, :128]).all() and not torch.isfinite(back[1, 128:]).any()
    assert torch.isfinite(back[0, 128:]).all() and torch.isfinite(back[1, :128]).all()


def test_refusals():
    import selective_state_space_41_amd as V
    x, w = torch.zeros(2, 9, 8, device="cuda"), torch.zeros(8, device="cuda")
    stat = torch.zeros(2, 2, device="cuda")
    for bad in (lambda: V.groupnorm_fwd(x, w, w, 3), lambda: V.groupnorm_fwd(x, w[:4], w, 2), lambda: V.groupnorm_fwd(x, w, w, 0),
                lambda: V.groupnorm_fwd(x.transpose(1, 2), w, w, 2), lambda: V.groupnorm_fwd(x[0], w, w, 2),
                lambda: V.groupnorm_fwd(x[..., ::2], w[:4], w[:4], 2),
                lambda: V.groupnorm_bwd(x, x, w, w, stat[:1], stat), lambda: V.groupnorm_bwd(x, x[:, :4], w, w, stat, stat),
                lambda: V.act8_pack(x.transpose(1, 2))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: V.groupnorm_fwd(x.half(), w, w, 2), lambda: V.groupnorm_fwd(x, w.bfloat16(), w, 2), lambda: V.act8_pack([1.0]),
                lambda: V.groupnorm_bwd(x.bfloat16(), x, w, w, stat, stat), lambda: V.act8_unpack(x, w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: V.groupnorm_fwd(x[:, :0], w, w, 2), lambda: V.groupnorm_fwd(x, w, w, 2, eps=-1.0), lambda: V.act8_pack(x[:0])):
        with pytest.raises(RuntimeError):
            bad()
