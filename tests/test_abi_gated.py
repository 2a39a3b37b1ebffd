"""C-ABI checks of the gated recurrence block's entry points that need no GPU: every bad argument is refused with the
documented status before HIP is touched.  No kernel is launched."""
import ctypes

import pytest
import torch

import selective_state_space_41_amd as V

ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE = 1, 2, 3, 4, 5
P = [0x1000000 + 0x100000 * i for i in range(24)]


@pytest.fixture(scope="module")
def lib():
    return V.load()


def st(*s):
    return (ctypes.c_int64 * len(s))(*s)


def pack(lib, **kw):
    a = dict(x=P[0], xs=64, codes=P[1], scale=P[2], rows=4, dim=64, dt=1)
    a.update(kw)
    return lib.vmscan_act8_pack(*a.values(), None)


def unpack(lib, **kw):
    a = dict(codes=P[1], scale=P[2], x=P[0], rows=4, dim=64, dt=1)
    a.update(kw)
    return lib.vmscan_act8_unpack(*a.values(), None)


def test_act8(lib):
    for call in (pack, unpack):
        for k in ("x", "codes", "scale"):
            assert call(lib, **{k: None}) == ERR_NULL
        for kw in (dict(rows=0), dict(dim=0), dict(rows=-1), dict(dim=(1 << 30) + 1), dict(rows=1 << 41), dict(rows=1 << 29)):
            assert call(lib, **kw) == ERR_SHAPE, kw
        assert call(lib, dt=2) == ERR_UNSUPPORTED
        assert call(lib, x=P[0] + 1) == ERR_ALIGN and call(lib, scale=P[2] + 2) == ERR_ALIGN
    assert pack(lib, xs=63) == ERR_SHAPE


def gn(lib, **kw):
    a = dict(x=P[0], xs=st(6400, 64), w=P[1], b=P[2], n=P[3], y=P[4], mean=P[5], rstd=P[6], kc=P[7], ks=P[8], nb=2, L=100,
             dim=64, groups=4, eps=1e-5, act=1, dt=1, ws=P[9], wsb=1 << 20)
    a.update(kw)
    return lib.vmscan_groupnorm_fwd(*a.values(), None)


def test_groupnorm(lib):
    for k in ("x", "xs", "w", "b", "y", "mean", "rstd", "kc", "ks"):
        assert gn(lib, **{k: None}) == ERR_NULL, k
    for kw in (dict(nb=0), dict(nb=65536), dict(L=0), dict(L=1 << 30), dict(dim=0), dict(dim=4104), dict(groups=0),
               dict(groups=5), dict(groups=128), dict(xs=st(-1, 64)), dict(xs=st(64, -1)), dict(eps=-1.0),
               dict(eps=float("nan"))):
        assert gn(lib, **kw) == ERR_SHAPE, kw
    for kw in (dict(act=2), dict(dt=2)):
        assert gn(lib, **kw) == ERR_UNSUPPORTED, kw
    for kw in (dict(x=P[0] + 1), dict(y=P[4] + 8), dict(w=P[1] + 2), dict(mean=P[5] + 1), dict(ks=P[8] + 2), dict(ws=P[9] + 8)):
        assert gn(lib, **kw) == ERR_ALIGN, kw
    need = lib.vmscan_groupnorm_fwd_workspace_bytes(2, 100, 64, 4, 1)
    assert lib.vmscan_groupnorm_fwd_workspace_bytes(2, 100, 64, 5, 1) == 0
    if need:
        assert gn(lib, wsb=need - 1) == ERR_WORKSPACE and gn(lib, ws=None) == ERR_WORKSPACE
    big = lib.vmscan_groupnorm_fwd_workspace_bytes(32, 3136, 512, 32, 0)
    assert big > 0 and gn(lib, nb=32, L=3136, dim=512, groups=32, xs=st(3136 * 512, 512), wsb=big - 1) == ERR_WORKSPACE


def gn_bwd(lib, **kw):
    a = dict(dy=P[0], dys=st(6400, 64), x=P[1], xs=st(6400, 64), c=None, cs=None, w=P[2], b=P[3], mean=P[4], rstd=P[5],
             n=P[6], dx=P[7], dw=P[8], db=P[9], nb=2, L=100, dim=64, groups=4, act=1, dt=1, ws=P[10], wsb=1 << 20)
    a.update(kw)
    return lib.vmscan_groupnorm_bwd(*a.values(), None)


def test_groupnorm_bwd(lib):
    for k in ("dy", "dys", "x", "xs", "w", "b", "mean", "rstd", "dx", "dw", "db"):
        assert gn_bwd(lib, **{k: None}) == ERR_NULL, k
    assert gn_bwd(lib, c=P[11], cs=P[12]) == ERR_NULL          # both forms of x
    assert gn_bwd(lib, x=None, c=P[11]) == ERR_NULL
    for kw in (dict(nb=0), dict(groups=3), dict(dys=st(-1, 64)), dict(xs=st(0, -2)), dict(dim=8192)):
        assert gn_bwd(lib, **kw) == ERR_SHAPE, kw
    for kw in (dict(act=-1), dict(dt=7)):
        assert gn_bwd(lib, **kw) == ERR_UNSUPPORTED, kw
    for kw in (dict(dy=P[0] + 1), dict(dx=P[7] + 4), dict(db=P[9] + 2)):
        assert gn_bwd(lib, **kw) == ERR_ALIGN, kw
    need = lib.vmscan_groupnorm_bwd_workspace_bytes(2, 100, 64, 4)
    assert need > 0 and gn_bwd(lib, wsb=need - 1) == ERR_WORKSPACE and gn_bwd(lib, ws=None) == ERR_WORKSPACE


def fwd(lib, **kw):
    s = st(64 * 6000, 64)
    a = dict(x=P[0], xs=s, r=P[1], rs=s, i=P[2], is_=s, A=P[3], s0=P[4], n=P[5], rev=0, out=P[6], sT=P[7], kc=P[8], ks=P[9],
             nb=2, L=6000, dim=64, dt=1, ws=P[10], wsb=0)
    a.update(kw)
    return lib.vmscan_gated_scan_fwd(*a.values(), None)


def bwd(lib, **kw):
    s = st(64 * 6000, 64)
    a = dict(x=P[0], xs=s, r=P[1], rs=s, i=P[2], is_=s, h=P[3], c=None, cs=None, A=P[4], s0=P[5], n=P[6], rev=0, do=P[7],
             dos=s, dsT=P[8], dx=P[9], dr=P[10], di=P[11], dA=P[12], ds0=P[13], nb=2, L=6000, dim=64, dt=1, ws=P[14], wsb=0)
    a.update(kw)
    return lib.vmscan_gated_scan_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [fwd, bwd], ids=["fwd", "bwd"])
def test_gated_scan(lib, call):
    need = ["x", "xs", "r", "rs", "i", "is_", "A"] + (["out", "kc", "ks"] if call is fwd else ["h", "do", "dos", "dx", "dr", "di", "dA"])
    for k in need:
        assert call(lib, **{k: None}) == ERR_NULL, k
    for kw in (dict(nb=0), dict(L=0), dict(L=1 << 30), dict(dim=0), dict(dim=1 << 20), dict(xs=st(-1, 64)), dict(rs=st(1, -1)),
               dict(is_=st(0, 1 << 24)), dict(nb=1 << 24)):
        assert call(lib, **kw) == ERR_SHAPE, kw
    for kw in (dict(dt=2), dict(rev=2)):
        assert call(lib, **kw) == ERR_UNSUPPORTED, kw
    for kw in (dict(x=P[0] + 1), dict(A=P[3] + 2), dict(s0=P[4] + 1), dict(n=P[5] + 2), dict(ws=P[10] + 8, wsb=1 << 30)):
        assert call(lib, **kw) == ERR_ALIGN, kw
    assert call(lib) == ERR_WORKSPACE and call(lib, ws=None, wsb=1 << 30) == ERR_WORKSPACE
    if call is fwd:
        assert call(lib, sT=P[4] + 4) == ERR_UNSUPPORTED      # states that overlap without being one buffer
    else:
        assert call(lib, ds0=P[8] + 4) == ERR_UNSUPPORTED and call(lib, ds0=P[5]) == ERR_UNSUPPORTED
        assert call(lib, c=P[15]) == ERR_NULL and call(lib, c=P[15], cs=P[16]) == ERR_UNSUPPORTED


def step(lib, **kw):
    a = dict(x=P[0], xs=64, r=P[1], rs=64, i=P[2], is_=64, A=P[3], state=P[4], slots=P[5], out=P[6], nb=2, pool=3, dim=64, dt=1)
    a.update(kw)
    return lib.vmscan_gated_scan_step(*a.values(), None)


def test_step(lib):
    for k in ("x", "r", "i", "A", "state", "out"):
        assert step(lib, **{k: None}) == ERR_NULL, k
    for kw in (dict(nb=0), dict(pool=0), dict(dim=0), dict(slots=None), dict(xs=-1), dict(is_=1 << 41)):
        assert step(lib, **kw) == ERR_SHAPE, kw
    assert step(lib, dt=3) == ERR_UNSUPPORTED
    for kw in (dict(x=P[0] + 1), dict(state=P[4] + 2), dict(slots=P[5] + 1)):
        assert step(lib, **kw) == ERR_ALIGN, kw


def test_binding_refuses_before_the_library():
    """Wrong kinds of tensors raise in Python; nothing reaches the GPU (there is none here to reach)."""
    x = torch.zeros(2, 5, 8)
    for call in (lambda: V.act8_pack(x), lambda: V.groupnorm_fwd(x, x[0, 0], x[0, 0], 2),
                 lambda: V.gated_scan_fwd(x, x, x, x[0, 0]), lambda: V.gated_scan_step(x[:, 0], x[:, 0], x[:, 0], x[0, 0], x[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        V.act8_pack(x.half())
    with pytest.raises(TypeError):
        V.act8_unpack(x, None)
    with pytest.raises(ValueError):
        V.groupnorm_fwd(x[0], x[0, 0], x[0, 0], 2)


def test_limits_of_a_launch(lib):
    """Tiles of channels times batch times chunks below 2^23: beyond, no workspace is named and the call refuses."""
    assert lib.vmscan_gated_scan_fwd_workspace_bytes(1, (1 << 30) - 1, 64) == 0
    assert lib.vmscan_gated_scan_bwd_workspace_bytes(1 << 12, 1 << 18, 64) == 0
    assert fwd(lib, L=(1 << 30) - 1, wsb=1 << 62) == ERR_SHAPE and bwd(lib, nb=1 << 12, L=1 << 18, wsb=1 << 62) == ERR_SHAPE
    assert lib.vmscan_gated_scan_fwd_workspace_bytes(1, (1 << 30) - 256, 64) > 1 << 30
    assert lib.vmscan_gated_scan_fwd_workspace_bytes(64, 128, 384) == 0  # one chunk: nothing waits
    assert lib.vmscan_gated_scan_bwd_workspace_bytes(64, 64, 384) == 64 * 384 * 4
    assert step(lib, nb=65536) == ERR_SHAPE
