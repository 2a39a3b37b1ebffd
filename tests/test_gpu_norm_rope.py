"""The residual norm and the rotary positions on the GPU against the fp64 oracle.

Tolerances, derived from the operation counts:
  * norm: a row's sum of squares is good to (log2(dim) + 8) 2^-24 of itself (butterfly over lanes of
    runs of 8) and its square root halves that; y takes three more roundings: 16 * 2^-24 |y| in
    float32 for dim up to 32768, plus half a unit of the output's type: with 8 significant bits that
    is up to 2^-8 |y| for bfloat16.
  * its gradient: a difference of two terms, so the same relative to the sum of their magnitudes; the
    weight's gradient sums rows in a tree: (rows' share per lane + 32 + 10) 2^-24 of the magnitudes.
  * rope: the angle's revolutions are good to 2^-24 of a revolution (2 pi 2^-24 radians < 2^-21), so a
    turned channel is off by at most that times the pair's length plus two roundings: 2^-20 |pair|."""
import numpy as np
import pytest
import torch

import synth
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def rnd(a, dtype):
    return synth.round_bf16(a.astype(np.float32)) if dtype == "bf16" else a.astype(np.float32)


def td(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def near(name, y, r, room):
    y = y.double().cpu().numpy()
    assert y.shape == r.shape and np.all(np.isfinite(y)), name
    used = float(np.max(np.abs(y - r) / (room + 1e-37)))
    print(f"[norm/rope] {name}: {used:.3f} of the tolerance", flush=True)
    assert used <= 1.0, f"{name}: {used:.2f} times the tolerance"


def unit(dtype):
    return UBF if dtype == "bf16" else U32


# one lane's run, a partial run, every row layout's edges, rows that need several waves
DIMS = [1, 7, 8, 37, 64, 65, 128, 192, 256, 260, 384, 512, 520, 768, 1024, 1032, 2048, 2056, 8192, 8200, 32768]
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("x,res", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_norm(dim, x, res):
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(dim)
    rows = 5 if dim > 64 else 133  # more rows than one workgroup holds where they are short
    a, b = rnd(rng.standard_normal((rows, dim)), x), rnd(2 * rng.standard_normal((rows, dim)), res)
    w = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32)
    eps = 1e-5
    y, scale, r, rstd = V.rmsnorm_fwd(td(a, x), td(w, "f32"), residual=td(b, res), eps=eps)
    assert scale is None and r.dtype == (torch.bfloat16 if res == "bf16" else torch.float32)
    ry, rr, rrstd = BO.rmsnorm(a, w, b, eps)
    near("y", y, ry, (16 * U32 + unit(x)) * np.abs(ry))
    near("residual_out", r, rr, (U32 + unit(res)) * np.abs(rr))
    near("rstd", rstd, rrstd, 16 * U32 * rrstd)
    y2, _, r2, _ = V.rmsnorm_fwd(td(a, x), td(w, "f32"), eps=eps)  # without a residual
    ry2 = BO.rmsnorm(a, w, None, eps)[0]
    near("y alone", y2, ry2, (16 * U32 + unit(x)) * np.abs(ry2))

    dy, dres = rnd(rng.standard_normal((rows, dim)), x), rnd(rng.standard_normal((rows, dim)), res)
    r_in, rstd_in = rnd(rr, res), rrstd.astype(np.float32)
    g = V.rmsnorm_bwd(td(dy, x), td(r_in, res), td(w, "f32"), td(rstd_in, "f32"), dresidual_out=td(dres, res))
    dr, dw = BO.rmsnorm_bwd(dy, r_in, w, rstd_in, dres)
    n = np.abs(r_in) * rstd_in[:, None]
    mag = rstd_in[:, None] * (np.abs(w * dy) + n * np.mean(n * np.abs(w * dy), axis=1, keepdims=True)) + np.abs(dres)
    near("dx", g["dx"], dr, 24 * U32 * mag + unit(x) * np.abs(dr))
    near("dresidual", g["dresidual"], dr, 24 * U32 * mag + unit(res) * np.abs(dr))
    assert (g["dresidual"] is g["dx"]) == (x == res)
    near("dweight", g["dweight"], dw, 64 * U32 * np.sum(np.abs(dy) * n, axis=0))
    g2 = V.rmsnorm_bwd(td(dy, x), td(r_in, res), td(w, "f32"), td(rstd_in, "f32"))
    dr2 = BO.rmsnorm_bwd(dy, r_in, w, rstd_in)[0]
    near("dx alone", g2["dx"], dr2, 24 * U32 * mag + unit(x) * np.abs(dr2))
    assert torch.equal(g["dweight"], g2["dweight"])


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("x,res", TYPES)
@pytest.mark.parametrize("dim", [8, 37, 64, 128, 130, 192, 384, 768, 1000, 2048, 2200, 9000])
def test_norm_fp8(dim, x, res, group):
    """The codes stand for y to half a code step (2^-4 of the value, or 2^-10 of a code unit for the
    subnormal codes), the scales for max|y| / 448."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(dim + group)
    rows = 9
    a, b = rnd(rng.standard_normal((rows, dim)), x), rnd(rng.standard_normal((rows, dim)), res)
    a[2], b[2] = 0.0, 0.0  # a row of zeros: scale 1, codes 0
    w = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32)
    y, scale, r, _ = V.rmsnorm_fwd(td(a, x), td(w, "f32"), residual=td(b, res), out_dtype=torch.float8_e4m3fn,
                                   group=group)
    assert y.dtype == torch.float8_e4m3fn
    ry = BO.rmsnorm(a, w, b)[0]
    width = group or dim
    ng = -(-dim // width)
    assert scale.shape == (rows, ng)
    pad = np.pad(ry, ((0, 0), (0, ng * width - dim))).reshape(rows, ng, width)
    amax = np.max(np.abs(pad), axis=-1)
    want = np.where(amax > 0, amax / 448, 1.0)
    near("scale", scale, want, 20 * U32 * want)
    s = np.repeat(scale.double().cpu().numpy(), width, axis=1)[:, :dim]
    codes = y.float().double().cpu().numpy()
    assert np.all(np.abs(codes) <= 448)
    near("codes", y.float(), ry / s, (2.0 ** -4 + 24 * U32) * np.abs(ry / s) + 2.0 ** -10)
    assert np.all(codes[2] == 0) and np.all(scale[2].cpu().numpy() == 1)
    top = np.take_along_axis(np.pad(codes, ((0, 0), (0, ng * width - dim))).reshape(rows, ng, width),
                             np.argmax(np.abs(pad), -1)[..., None], -1)[..., 0]
    assert np.all(np.abs(top[amax > 0]) == 448)  # the largest value takes the largest code


def test_norm_rows_and_values():
    """Rows apart, in place, many rows, a NaN and an infinity confined to their rows."""
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(1)
    rows, dim = 20000, 72
    a, b = (rng.standard_normal((rows, dim)).astype(np.float32) for _ in range(2))
    w = np.ones(dim, np.float32)
    wide = torch.zeros(rows, dim + 24, device="cuda")
    wide[:, :dim] = td(a, "f32")
    res = td(b, "f32")
    y, _, r, _ = V.rmsnorm_fwd(wide[:, :dim], td(w, "f32"), residual=res, residual_out=res)
    assert r is res
    ry, rr, _ = BO.rmsnorm(a, w, b)
    near("strided y", y, ry, 17 * U32 * np.abs(ry))
    near("in place", r, rr, U32 * np.abs(rr))
    bad = td(a, "f32")
    bad[3, 5], bad[7, 0] = float("nan"), float("inf")
    for dt in (None, torch.float8_e4m3fn):
        y, scale, _, rstd = V.rmsnorm_fwd(bad, td(w, "f32"), out_dtype=dt)
        yf = y.float()
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[[3, 7]] = False
        assert torch.isnan(yf[3]).all() and torch.isnan(yf[7, 0]) and torch.isfinite(yf[keep]).all()
        if scale is not None:
            assert torch.isnan(scale[3]) and torch.isfinite(scale[keep]).all()


def test_norm_bwd_many_rows():
    import selective_state_space_41_amd as V
    rng = np.random.default_rng(2)
    rows, dim = 40001, 40
    dy, r = rng.standard_normal((2, rows, dim)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal(dim)).astype(np.float32)
    rstd = (1 / np.sqrt(np.mean(r * r, 1) + 1e-5)).astype(np.float32)
    g = V.rmsnorm_bwd(td(dy, "f32"), td(r, "f32"), td(w, "f32"), td(rstd, "f32"))
    dr, dw = BO.rmsnorm_bwd(dy, r, w, rstd)
    mag = np.sum(np.abs(dy * r) * rstd[:, None], axis=0)
    near("dweight", g["dweight"], dw, 128 * U32 * mag)
    again = V.rmsnorm_bwd(td(dy, "f32"), td(r, "f32"), td(w, "f32"), td(rstd, "f32"))
    assert torch.equal(g["dweight"], again["dweight"])


def test_norm_gradient_by_differences():
    """Central differences of the kernel's own loss, step 2^-7, in float32: truncation (h^2) and rounding
    (2^-24 sqrt(terms) / h) both below 1e-3 of the gradient's norm."""
    import selective_state_space_41_amd as V
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, res, dy, dres = (torch.randn(6, 200, generator=gen, device="cuda") for _ in range(4))
    w = 1 + 0.2 * torch.randn(200, generator=gen, device="cuda")

    def loss(x, w):
        y, _, r, _ = V.rmsnorm_fwd(x, w, residual=res)
        return (y.double() * dy).sum() + (r.double() * dres).sum()

    _, _, r, rstd = V.rmsnorm_fwd(x, w, residual=res)
    g = V.rmsnorm_bwd(dy, r, w, rstd, dresidual_out=dres)
    for name, at in (("dx", 0), ("dweight", 1)):
        step, h = torch.randn((x, w)[at].shape, generator=gen, device="cuda"), 2.0 ** -7
        hi, lo = ([a + s * h * step if i == at else a for i, a in enumerate((x, w))] for s in (1, -1))
        want, got = float((loss(*hi) - loss(*lo)) / (2 * h)), float((g[name].double() * step).sum())
        assert abs(got - want) <= 1e-3 * float(g[name].double().norm()), (name, got, want)


# ---- rotary positions


def rope_case(seed, B, T, H, Hk, dim, pairs, axes, dtype, top=100.0):
    rng = np.random.default_rng(seed)
    return dict(q=rnd(rng.standard_normal((B, T, H, dim)), dtype), k=rnd(rng.standard_normal((B, T, Hk, dim)), dtype),
                pos=(rng.uniform(0, top, (T, axes))).astype(np.float32),
                f=np.exp(rng.uniform(np.log(1e-4), 0, pairs)).astype(np.float32),
                axis=rng.integers(0, axes, pairs).astype(np.int32))


def rope_check(name, y, x, p, dtype, pos=None, **kw):
    r = BO.rope_axes(x, p["pos"] if pos is None else pos, p["f"], p["axis"], **kw)
    pairs = len(p["f"])
    m = np.abs(np.array(x, np.float64))
    i, j = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if kw.get("interleaved") else \
        (slice(0, pairs), slice(pairs, 2 * pairs))
    m[..., i] = m[..., j] = np.hypot(m[..., i], m[..., j])
    near(name, y, r, 2.0 ** -20 * m + unit(dtype) * np.abs(r))
    assert np.array_equal(y.float().cpu().numpy()[..., 2 * pairs:], x[..., 2 * pairs:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,pairs,axes", [(64, 32, 2), (64, 24, 3), (128, 64, 3), (16, 4, 1), (10, 5, 2), (10, 2, 1),
                                            (72, 20, 2), (2, 1, 1), (40, 9, 4)])
def test_rope(dim, pairs, axes, interleaved, dtype):
    import selective_state_space_41_amd as V
    p = rope_case(dim + pairs, 2, 37, 6, 2, dim, pairs, axes, dtype)
    q, k = td(p["q"], dtype), td(p["k"], dtype)
    pos, f, axis = td(p["pos"], "f32"), td(p["f"], "f32"), torch.from_numpy(p["axis"]).cuda()
    for inverse in (False, True):
        yq, yk = V.rope_axes(q, k, pos, f, axis, interleaved=interleaved, inverse=inverse)
        rope_check(f"q {dim} {pairs}", yq, p["q"], p, dtype, interleaved=interleaved, inverse=inverse)
        rope_check(f"k {dim} {pairs}", yk, p["k"], p, dtype, interleaved=interleaved, inverse=inverse)
    alone, none = V.rope_axes(q, None, pos, f, axis, interleaved=interleaved, inverse=True)
    assert none is None and torch.equal(alone, yq)
    q2, k2 = q.clone(), k.clone()  # in place
    a, b = V.rope_axes(q2, k2, pos, f, axis, interleaved=interleaved, inverse=True, q_out=q2, k_out=k2)
    assert a is q2 and b is k2 and torch.equal(q2, yq) and torch.equal(k2, yk)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_strides_and_batches(interleaved):
    """Slices of one projection (on and off the 16-byte grid), positions per batch, one token, many."""
    import selective_state_space_41_amd as V
    for B, T, H, Hk, dim, pairs, cut in ((3, 1, 4, 2, 32, 16, 0), (2, 300, 6, 3, 16, 8, 0), (1, 50, 2, 1, 10, 5, 3)):
        p = rope_case(T, B, T, H, Hk, dim, pairs, 2, "bf16")
        both = torch.zeros(B, T, (H + Hk) * dim + cut, dtype=torch.bfloat16, device="cuda")
        heads = both[..., cut:].unflatten(-1, (H + Hk, dim))
        q, k = heads[:, :, :H], heads[:, :, H:]
        q.copy_(td(p["q"], "bf16"))
        k.copy_(td(p["k"], "bf16"))
        pos = np.random.default_rng(0).uniform(0, 30, (B, T, 2)).astype(np.float32)
        y = V.rope_axes(q, k, td(pos, "f32"), td(p["f"], "f32"), torch.from_numpy(p["axis"]).cuda(),
                        interleaved=interleaved)
        rope_check("slice q", y[0], p["q"], p, "bf16", pos=pos, interleaved=interleaved)
        rope_check("slice k", y[1], p["k"], p, "bf16", pos=pos, interleaved=interleaved)


def test_rope_large_positions_and_axes():
    """Positions in the millions lose nothing (the angle is reduced from the exact product); a pair whose
    axis does not exist is not turned."""
    import selective_state_space_41_amd as V
    p = rope_case(3, 1, 64, 2, 2, 32, 16, 2, "f32", top=2.0 ** 23)
    p["axis"][3], p["axis"][4] = -1, 2
    y = V.rope_axes(td(p["q"], "f32"), None, td(p["pos"], "f32"), td(p["f"], "f32"), torch.from_numpy(p["axis"]).cuda())
    rope_check("large", y[0], p["q"], p, "f32")
    assert np.array_equal(y[0][..., [3, 4, 19, 20]].cpu().numpy(), p["q"][..., [3, 4, 19, 20]])


def test_rope_offsets_past_32_bits():
    import selective_state_space_41_amd as V
    p = rope_case(4, 2, 9, 1, 1, 16, 8, 1, "bf16")
    gap = 2 ** 31 + 64
    pool = torch.empty(gap + 9 * 16, dtype=torch.bfloat16, device="cuda")
    q = pool.as_strided((2, 9, 1, 16), (gap, 16, 16, 1))
    q.copy_(td(p["q"], "bf16"))
    y = V.rope_axes(q, None, td(p["pos"], "f32"), td(p["f"], "f32"), torch.from_numpy(p["axis"]).cuda(), q_out=q)
    rope_check("far", y[0], p["q"], p, "bf16")


def test_streams():
    """On another stream than the tensors' own, ordered by the caller, with outputs made by the call."""
    import selective_state_space_41_amd as V
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, w = torch.randn(300, 96, generator=gen, device="cuda"), torch.ones(96, device="cuda")
    q = torch.randn(2, 50, 4, 24, generator=gen, device="cuda")
    pos, f, axis = torch.rand(50, 1, generator=gen, device="cuda"), torch.ones(12, device="cuda"), \
        torch.zeros(12, dtype=torch.int32, device="cuda")
    want = V.rmsnorm_fwd(x, w)[0], V.rope_axes(q, None, pos, f, axis)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = V.rmsnorm_fwd(x, w, stream=side)[0], V.rope_axes(q, None, pos, f, axis, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    import selective_state_space_41_amd as V
    x, w = torch.zeros(4, 16, device="cuda"), torch.ones(16, device="cuda")
    q, f, axis = torch.zeros(2, 9, 4, 16, device="cuda"), torch.ones(8, device="cuda"), \
        torch.zeros(8, dtype=torch.int32, device="cuda")
    pos = torch.zeros(9, 1, device="cuda")
    for bad, kind in (
        (lambda: V.rmsnorm_fwd(x, w.double()), TypeError),
        (lambda: V.rmsnorm_fwd(x, w[:8]), ValueError),
        (lambda: V.rmsnorm_fwd(x.half(), w), TypeError),
        (lambda: V.rmsnorm_fwd(x.cpu(), w), ValueError),
        (lambda: V.rmsnorm_fwd(x[:, ::2], w[:8]), ValueError),
        (lambda: V.rmsnorm_fwd(x, w, residual=x.bfloat16()), RuntimeError),   # float32 with a narrower residual
        (lambda: V.rmsnorm_fwd(x, w, out_dtype=torch.bfloat16), TypeError),
        (lambda: V.rmsnorm_fwd(x, w, out_dtype=torch.float8_e4m3fn, group=64), RuntimeError),
        (lambda: V.rmsnorm_fwd(x, w, group=128), RuntimeError),
        (lambda: V.rmsnorm_fwd(x[:0], w), RuntimeError),
        (lambda: V.rmsnorm_fwd(x, w, eps=-1.0), RuntimeError),
        (lambda: V.rmsnorm_fwd(torch.zeros(1, 32776, device="cuda"), torch.zeros(32776, device="cuda")), RuntimeError),
        (lambda: V.rmsnorm_bwd(x, x, w, torch.ones(3, device="cuda")), ValueError),
        (lambda: V.rope_axes(q, None, pos, f, axis.long()), TypeError),
        (lambda: V.rope_axes(q, None, pos[:8], f, axis), ValueError),
        (lambda: V.rope_axes(q, q[:, :8], pos, f, axis), ValueError),
        (lambda: V.rope_axes(q, q.bfloat16(), pos, f, axis), TypeError),
        (lambda: V.rope_axes(q[..., :14], None, pos, f, axis), RuntimeError),  # 8 pairs need 16 channels
        (lambda: V.rope_axes(q[..., ::2], None, pos, f[:4], axis[:4]), ValueError),
        (lambda: V.rope_axes(q[:, :0], None, pos[:0], f, axis), RuntimeError),
    ):
        with pytest.raises(kind):
            bad()
