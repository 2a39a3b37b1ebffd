"""Linear attention against the fp64 oracle on every kernel that a call can reach: activations' type, padded key channels,
a workgroup's value channels, and how the states of segments (in the gradient also parts of segments) are joined, each with
an initial state, rows of unequal length among them an empty one, and shared heads.

The shapes come from the library's own choice (``linattn_plan``): a table of shapes is searched for the cheapest one that
takes the wanted path, and a path that none of them takes fails the test, so that a changed choice cannot drop one
unseen.  Joining by a launch of its own is also forced at the small shapes, by states updated in place; long shapes
that take it by themselves would keep the oracle busy for minutes."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from test_gpu_linattn import ACT, WIDE, check, dev, make, oracle_bwd, oracle_fwd

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# (padded key channels, value channels of a workgroup) that have a forward, a gradient
FORWARD = {"bf16": [(32, 32), (32, 64), (32, 128), (64, 32), (64, 64), (64, 128), (128, 32), (128, 64)],
           "f32": [(32, 32), (32, 64), (32, 128), (64, 32), (64, 64), (128, 32), (128, 64)]}
GRADIENT = [(k, v) for k in (32, 64, 128) for v in (64, 128)]
DK = {32: (32, 24), 64: (64, 48), 128: (128, 80)}
DV = {32: (32, 64, 72), 64: (64, 40, 104, 128), 128: (128, 104)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def shape_for(dtype, key, width, join, parts, gradient):
    """(B, T, H, dk, dv) with the least work for the oracle, which goes token by token."""
    import selective_state_space_41_amd as V
    best = None
    for dk, dv in itertools.product(DK[key], DV[width]):
        for B, H, T in itertools.product((1, 2, 3, 6, 12, 16), (2, 4, 6, 8, 12, 16, 32), (65, 100, 130, 200, 300, 530, 870, 1950)):
            cost = B * T * (1 + H * dk * dv / 30000)
            if best and cost >= best[0]:
                continue
            p = V.linattn_plan(B, T, H, dk, dv, TYPES[dtype], gradient)
            if (p["width"], p["join"], p["parts"] > 1) == (width, join, parts):
                best = (cost, (B, T, H, dk, dv))
    assert best, f"no shape takes the path {dtype} {key} {width} {join} parts {parts}"
    return best[1]


def case(dtype, key, width, join, parts, gradient):
    B, T, H, dk, dv = shape_for(dtype, key, width, join, parts, gradient)
    Hk = H // 2
    p = make(key + width + T, B, T, H, Hk, dk, dv, dtype)
    n = [T - 3] if B == 1 else [0 if b == 1 else T - 7 * b for b in range(B)]
    name = f"{B} x {T}, {H} heads of {dk} x {dv}, {dtype}, width {width}, join {join}, parts {parts}"
    print(f"[linattn paths] {'gradient' if gradient else 'forward'} {name}", flush=True)
    return name, p, n, torch.tensor(n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("join", [None, "walk"])
@pytest.mark.parametrize("dtype,key,width", [(t, k, w) for t in FORWARD for k, w in FORWARD[t]])
def test_forward(dtype, key, width, join):
    import selective_state_space_41_amd as V
    name, p, n, lengths = case(dtype, key, width, join, False, False)
    t = {k: dev(p, k) for k in ("q", "k", "v", "g", "s0")}
    (r_out, r_sT), (m_out, m_sT) = oracle_fwd(p, p["s0"], n)
    for where in ("apart", "in place"):  # in place: joined by a launch
        s0 = t["s0"].clone()
        out, sT = V.linattn_fwd(t["q"], t["k"], t["v"], t["g"], scale=p["scale"], initial_state=s0, lengths=lengths,
                                final_state=s0 if where == "in place" else None)
        torch.cuda.synchronize()
        check(f"{name}, {where}: out", out, r_out, m_out, ACT[dtype])
        check(f"{name}, {where}: final_state", sT, r_sT, m_sT, WIDE[dtype])


def gradient_in_place(p, t, lengths):
    """The C entry with dinitial_state in dfinal_state's buffer."""
    import selective_state_space_41_amd as V
    lib, dt = V.load(), int(p["dtype"] == "bf16")
    B, T, H, dv = p["v"].shape
    Hk, dk = p["q"].shape[2:]
    st = lambda x: (ctypes.c_int64 * 3)(*x.stride()[:3])
    g = dict(dq=torch.empty_like(t["q"]), dk=torch.empty_like(t["k"]), dv=torch.empty_like(t["v"]),
             dlog_decay=torch.empty_like(t["g"]), dinitial_state=t["dsT"].clone())
    ws = torch.empty(lib.vmscan_linattn_bwd_workspace_bytes(B, T, H, Hk, dk, dv, 0, dt), dtype=torch.uint8, device="cuda")
    code = lib.vmscan_linattn_bwd(
        t["q"].data_ptr(), st(t["q"]), t["k"].data_ptr(), st(t["k"]), t["v"].data_ptr(), st(t["v"]), t["g"].data_ptr(),
        st(t["g"]), t["s0"].data_ptr(), lengths.data_ptr(), t["dout"].data_ptr(), st(t["dout"]),
        g["dinitial_state"].data_ptr(), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(),
        g["dlog_decay"].data_ptr(), g["dinitial_state"].data_ptr(), B, T, H, Hk, dk, dv, p["scale"], dt, ws.data_ptr(),
        ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0
    return g


# heads of 128 x 128 are always joined by a launch, the others by the walks at these sizes
@pytest.mark.parametrize("cut", ["whole", "segments", "parts"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("key,width", GRADIENT)
def test_gradient(key, width, dtype, cut):
    import selective_state_space_41_amd as V
    join = None if cut == "whole" else "launch" if (key, width) == (128, 128) else "walk"
    name, p, n, lengths = case(dtype, key, width, join, cut == "parts", True)
    t = {k: dev(p, k) for k in ("q", "k", "v", "g", "s0", "dsT", "dout")}
    r, m = oracle_bwd(p, p["s0"], n, p["dsT"])
    for where in ("apart", "in place"):
        if where == "apart":
            g = V.linattn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], scale=p["scale"], initial_state=t["s0"],
                              lengths=lengths, dfinal_state=t["dsT"])
            torch.cuda.synchronize()
        else:
            g = gradient_in_place(p, t, lengths)
        for key_ in ("dq", "dk", "dv"):
            check(f"{name}, {where}: {key_}", g[key_], r[key_], m[key_], ACT[dtype])
        check(f"{name}, {where}: dlog_decay", g["dlog_decay"], r["dg"], m["dg"], WIDE[dtype])
        check(f"{name}, {where}: dinitial_state", g["dinitial_state"], r["ds0"], m["ds0"], WIDE[dtype])


LONG = [(False, 4, 2673, 3, 48, 104, "bf16"), (False, 1, 3632, 1, 88, 80, "f32"), (True, 5, 1918, 1, 96, 48, "bf16"),
        (True, 1, 4842, 6, 56, 16, "f32")]


@pytest.mark.parametrize("gradient,B,T,H,dk,dv,dtype", LONG)
def test_launch_by_itself(gradient, B, T, H, dk, dv, dtype):
    """Long shapes whose states are joined by a launch without being asked to: the same values as the tokens from the
    middle on, started from the state of the first half (gradient: the sum of both halves' calls)."""
    import selective_state_space_41_amd as V
    plan = V.linattn_plan(B, T, H, dk, dv, TYPES[dtype], gradient)
    assert plan["join"] == "launch", plan
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    a = TYPES[dtype]
    q, k, v, do = rnd(B, T, H, dk).to(a), rnd(B, T, H, dk).to(a), rnd(B, T, H, dv).to(a), rnd(B, T, H, dv).to(a)
    g, s0, dsT = -0.02 * torch.rand(B, T, H, generator=gen, device="cuda"), rnd(B, H, dk, dv), rnd(B, H, dk, dv)
    print(f"[linattn paths] by itself {B} x {T}, {H} heads of {dk} x {dv}, {dtype}, gradient {gradient}", flush=True)
    h = T // 2 + 3
    one, two = [x[:, :h] for x in (q, k, v, g)], [x[:, h:] for x in (q, k, v, g)]
    out1, mid = V.linattn_fwd(*one, initial_state=s0)
    rel = lambda x, y: float((x.double() - y.double()).norm() / y.double().norm())
    act = 2.0 ** -18 if dtype == "f32" else 2.0 ** -9  # two roundings to bfloat16 of nearly the same numbers
    if not gradient:
        out2, last = V.linattn_fwd(*two, initial_state=mid)
        out, sT = V.linattn_fwd(q, k, v, g, initial_state=s0)
        for x, y, most in ((out[:, :h], out1, act), (out[:, h:], out2, act), (sT, last, 2.0 ** -18)):
            assert rel(x, y) <= most
        return
    g2 = V.linattn_bwd(*two, do[:, h:], initial_state=mid, dfinal_state=dsT)
    g1 = V.linattn_bwd(*one, do[:, :h], initial_state=s0, dfinal_state=g2["dinitial_state"])
    whole = V.linattn_bwd(q, k, v, g, do, initial_state=s0, dfinal_state=dsT)
    for key in ("dq", "dk", "dv", "dlog_decay"):
        most = act if key != "dlog_decay" else 2.0 ** -18
        assert rel(whole[key][:, :h], g1[key]) <= most and rel(whole[key][:, h:], g2[key]) <= most, key
    assert rel(whole["dinitial_state"], g1["dinitial_state"]) <= 2.0 ** -18
