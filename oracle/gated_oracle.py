"""fp64 oracle of a gated recurrence block's operators: activations in 8 bits, the group norm with its activation
and the gated linear recurrence, from the definitions in include/vmscan.h.  Shares no code with the library.

``*_room`` values bound a float32 evaluation's error, from the operations' own (``U`` = half a unit of 1 in float32):
a hardware exp2, reciprocal or square root is within 2 U of its value, a rounded operation within U."""
import numpy as np

U = 2.0 ** -24


def sigmoid(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def act8_scale(x):
    """The scale of each 128 channels of x [..., dim]: [..., ceil(dim / 128)]."""
    x = np.abs(np.asarray(x, np.float64))
    pad = -x.shape[-1] % 128
    top = np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, pad)]).reshape(*x.shape[:-1], -1, 128).max(-1)
    return np.where(top > 0, np.maximum(top / 448.0, 2.0 ** -126), 1.0)


def act8_spread(scale, dim):
    """[..., groups] -> [..., dim]"""
    return np.repeat(np.asarray(scale, np.float64), 128, axis=-1)[..., :dim]


def groupnorm(x, w, b, groups, eps=1e-5, act=True, lengths=None):
    """x [B, T, dim]; returns (y, mean, rstd)."""
    x, w, b = (np.asarray(a, np.float64) for a in (x, w, b))
    B, T, dim = x.shape
    y, mean, rstd = np.zeros(x.shape), np.zeros((B, groups)), np.full((B, groups), 1.0 / np.sqrt(eps) if eps else np.inf)
    for k in range(B):
        n = T if lengths is None else int(np.clip(lengths[k], 0, T))
        if n == 0:
            continue
        g = x[k, :n].reshape(n, groups, -1)
        mean[k] = g.mean((0, 2))
        rstd[k] = 1.0 / np.sqrt(((g - mean[k][:, None]) ** 2).mean((0, 2)) + eps)
        u = ((g - mean[k][:, None]) * rstd[k][:, None]).reshape(n, dim) * w + b
        y[k, :n] = u * sigmoid(u) if act else u
    return y, mean, rstd


def groupnorm_bwd(dy, x, w, b, mean, rstd, act=True, lengths=None):
    """Returns (dx, dw, db) and their magnitudes: the same with absolute terms."""
    dy, x, w, b, mean, rstd = (np.asarray(a, np.float64) for a in (dy, x, w, b, mean, rstd))
    B, T, dim = x.shape
    G = mean.shape[1]
    dx, dw, db = np.zeros(x.shape), np.zeros(dim), np.zeros(dim)
    mx, mw, mb = np.zeros(x.shape), np.zeros(dim), np.zeros(dim)
    for k in range(B):
        n = T if lengths is None else int(np.clip(lengths[k], 0, T))
        if n == 0:
            continue
        up = lambda a: np.repeat(a, dim // G)[None]
        hat = (x[k, :n] - up(mean[k])) * up(rstd[k])
        u = hat * w + b
        s = sigmoid(u)
        g = dy[k, :n] * (s * (1 + u * (1 - s)) if act else 1.0)
        ga = np.abs(dy[k, :n]) * (1 + np.abs(u) if act else 1.0)
        over = lambda a: up(a.reshape(n, G, -1).mean((0, 2)))
        dx[k, :n] = up(rstd[k]) * (w * g - over(w * g) - hat * over(w * g * hat))
        wa, ha = np.abs(w) * ga, np.abs(hat)
        mx[k, :n] = up(rstd[k]) * (wa + over(wa) + ha * over(wa * ha))
        dw += (g * hat).sum(0)
        db += g.sum(0)
        mw += (ga * ha).sum(0)
        mb += ga.sum(0)
    return (dx, dw, db), (mx, mw, mb)


def _order(n, reverse):
    return range(n - 1, -1, -1) if reverse else range(n)


def _gates(x, r, i, A_log):
    x, r, i = (np.asarray(a, np.float64) for a in (x, r, i))
    with np.errstate(under="ignore"):
        y = np.exp(np.asarray(A_log, np.float64)) * sigmoid(r)
        return x, y, np.exp(-y), np.sqrt(-np.expm1(-2 * y)), sigmoid(r), sigmoid(i)


def _room_a(y, r):
    """Relative room of a = e^-y: the exponent's error (the gate's sigmoid, rate and products) and the exponential's."""
    return y * (12 + np.abs(r)) * U + 4 * U


def gated_scan(x, r, i, A_log, first=None, lengths=None, reverse=False):
    """x, r, i [B, T, dim]; returns (h, last) and the room of each."""
    B, T, dim = np.shape(x)
    r0, i0 = np.asarray(r, np.float64), np.asarray(i, np.float64)
    x, y, a, beta, _, q = _gates(x, r, i, A_log)
    h, room = np.zeros(x.shape), np.zeros(x.shape)
    last, rlast = np.zeros((B, dim)), np.zeros((B, dim))
    for k in range(B):
        n = T if lengths is None else int(np.clip(lengths[k], 0, T))
        s = np.zeros(dim) if first is None else np.array(first[k], np.float64)
        mag, e = np.abs(s), np.zeros(dim)
        for t in _order(n, reverse):
            b = beta[k, t] * q[k, t] * x[k, t]
            e = a[k, t] * (e + _room_a(y[k, t], r0[k, t]) * mag) + (30 + np.abs(r0[k, t]) + np.abs(i0[k, t])) * U * np.abs(b)
            mag = a[k, t] * mag + np.abs(b)
            e = e + 4 * U * mag  # the walk's and the joins' own roundings
            s = a[k, t] * s + b
            h[k, t], room[k, t] = s, e
        last[k], rlast[k] = s, e
    return (h, last), (room, rlast)


def gated_scan_bwd(x, r, i, h, A_log, dout, first=None, lengths=None, reverse=False, dlast=None):
    """Gradients for given h: returns dicts of values and of rooms, dx, dr, di, dA, dfirst."""
    B, T, dim = np.shape(x)
    r0 = np.asarray(r, np.float64)
    x, y, a, beta, p, q = _gates(x, r, i, A_log)
    h, dout = np.asarray(h, np.float64), np.asarray(dout, np.float64)
    ratio = np.divide(y, beta, out=np.zeros_like(y), where=beta > 0)
    val = {k: np.zeros(x.shape) for k in ("dx", "dr", "di")}
    room = {k: np.zeros(x.shape) for k in ("dx", "dr", "di")}
    val["dA"], room["dA"] = np.zeros(dim), np.zeros(dim)
    val["dfirst"], room["dfirst"] = np.zeros((B, dim)), np.zeros((B, dim))
    for k in range(B):
        n = T if lengths is None else int(np.clip(lengths[k], 0, T))
        G = np.zeros(dim) if dlast is None else np.array(dlast[k], np.float64)
        start = np.zeros(dim) if first is None else np.asarray(first[k], np.float64)
        mag, e = np.abs(G), np.zeros(dim)
        walk = list(_order(n, reverse))
        for at in range(n - 1, -1, -1):
            t = walk[at]
            before = h[k, walk[at - 1]] if at else start
            G, mag = G + dout[k, t], mag + np.abs(dout[k, t])
            e = e + 4 * U * mag
            tr, ti = (40 + 2 * np.abs(r0[k, t])) * U, (40 + 2 * np.abs(np.asarray(i)[k, t])) * U
            val["dx"][k, t] = G * beta[k, t] * q[k, t]
            room["dx"][k, t] = (e + (tr + ti) * mag) * beta[k, t] * q[k, t]
            val["di"][k, t] = val["dx"][k, t] * x[k, t] * (1 - q[k, t])
            room["di"][k, t] = room["dx"][k, t] * np.abs(x[k, t])
            d = a[k, t] * (q[k, t] * x[k, t] * a[k, t] * ratio[k, t] - y[k, t] * before)
            dm = a[k, t] * (np.abs(q[k, t] * x[k, t]) * a[k, t] * ratio[k, t] + y[k, t] * np.abs(before))
            val["dr"][k, t] = G * d * (1 - p[k, t])
            here = (e + (tr + ti + _room_a(y[k, t], r0[k, t])) * mag) * dm
            room["dr"][k, t] = here
            val["dA"] += G * d
            room["dA"] += here + (T // 8 + 64) * U * mag * dm
            e = a[k, t] * (e + _room_a(y[k, t], r0[k, t]) * mag) + 2 * U * a[k, t] * mag
            G, mag = a[k, t] * G, a[k, t] * mag
        val["dfirst"][k], room["dfirst"][k] = G, e + 2 * U * mag
    return val, room


def gated_scan_step(x, r, i, A_log, state, slots=None):
    """x, r, i [B, dim], state [pool, dim]; returns (out, state)."""
    state = np.array(state, np.float64)
    x, _, a, beta, _, q = _gates(x, r, i, A_log)
    out = np.zeros(x.shape)
    for k in range(len(x)):
        s = k if slots is None else int(slots[k])
        if 0 <= s < len(state):
            state[s] = a[k] * state[s] + beta[k] * q[k] * x[k]
            out[k] = state[s]
    return out, state
