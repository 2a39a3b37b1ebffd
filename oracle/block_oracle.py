"""fp64 oracle of the linear-attention block's operators: the norm with its residual, the rotary
positions and the decayed linear attention with their gradients, token by token from the
definitions in include/vmscan.h.  Shares no code with the library.

The ``*_abs`` values are the same sums over absolute values: the scale against which a float
evaluation of a sum that cancels can be held."""
import numpy as np


def rmsnorm(x, w, residual=None, eps=1e-5):
    """Returns (y, r, rstd) for x [rows, dim]."""
    r = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r * rstd[:, None] * np.asarray(w, np.float64), r, rstd


def rmsnorm_bwd(dy, r, w, rstd, dres=None):
    """Returns (dr, dw)."""
    dy, r, w, rstd = (np.asarray(a, np.float64) for a in (dy, r, w, rstd))
    n = r * rstd[:, None]
    wdy = w * dy
    dr = rstd[:, None] * (wdy - n * np.mean(wdy * n, axis=1, keepdims=True))
    return dr + (0.0 if dres is None else np.asarray(dres, np.float64)), np.sum(dy * n, axis=0)


def rope_axes(x, positions, inv_freq, axis, interleaved=False, inverse=False):
    """x [batch, L, heads, dim]; positions [L, axes] or [batch, L, axes]."""
    y = np.array(x, np.float64)
    pos = np.asarray(positions, np.float64)
    pos = pos[None] if pos.ndim == 2 else pos
    pairs = len(inv_freq)
    for p in range(pairs):
        if not 0 <= axis[p] < pos.shape[-1]:
            continue
        a = pos[..., axis[p]] * np.float64(inv_freq[p]) * (-1.0 if inverse else 1.0)
        c, s = np.cos(a)[:, :, None], np.sin(a)[:, :, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
        u, v = y[..., i].copy(), y[..., j].copy()
        y[..., i], y[..., j] = u * c - v * s, u * s + v * c
    return y


def _per_head(q, k, v, g, H):
    share = H // q.shape[2]
    q, k = (np.repeat(np.asarray(a, np.float64), share, axis=2) for a in (q, k))
    with np.errstate(under="ignore"):
        a = np.exp(np.broadcast_to(np.asarray(g, np.float64), v.shape[:3]))
    return q, k, np.asarray(v, np.float64), a


def linattn(q, k, v, g, scale, s0=None, lengths=None, keep=False):
    """q, k [B, T, Hk, dk], v [B, T, H, dv], g [B, T, H] or [H]; returns (out, final state) and, with
    keep, the list of states before each token and after the last."""
    B, T, H, dv = v.shape
    q, k, v, a = _per_head(q, k, v, g, H)
    S = np.zeros((B, H, q.shape[3], dv)) if s0 is None else np.array(s0, np.float64)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    out, states = np.zeros(v.shape), [S]
    for t in range(T):
        S = S.copy()
        for b in np.nonzero(n > t)[0]:
            S[b] = a[b, t][:, None, None] * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            out[b, t] = scale * np.einsum("hi,hij->hj", q[b, t], S[b])
        if keep:
            states.append(S)
    return (out, S, states) if keep else (out, S)


def linattn_bwd(q, k, v, g, dout, scale, s0=None, lengths=None, dsT=None):
    """Returns dict dq, dk, dv, dg (of g's shape), ds0."""
    B, T, H, dv_ = v.shape
    Hk = q.shape[2]
    per_head = np.ndim(g) == 1
    _, _, states = linattn(q, k, v, g, scale, s0, lengths, keep=True)
    q, k, v, a = _per_head(q, k, v, g, H)
    do = np.asarray(dout, np.float64) * scale
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    R = np.zeros(states[0].shape) if dsT is None else np.array(dsT, np.float64)
    dq, dk, dv, dg = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros((B, T, H))
    for t in range(T - 1, -1, -1):
        for b in np.nonzero(n > t)[0]:
            R[b] += q[b, t][:, :, None] * do[b, t][:, None, :]
            dq[b, t] = np.einsum("hij,hj->hi", states[t + 1][b], do[b, t])
            dk[b, t] = np.einsum("hij,hj->hi", R[b], v[b, t])
            dv[b, t] = np.einsum("hij,hi->hj", R[b], k[b, t])
            dg[b, t] = a[b, t] * np.einsum("hij,hij->h", states[t][b], R[b])
            R[b] = a[b, t][:, None, None] * R[b]
    dq, dk = (x.reshape(B, T, Hk, H // Hk, -1).sum(3) for x in (dq, dk))
    return dict(dq=dq, dk=dk, dv=dv, dg=dg.sum((0, 1)) if per_head else dg, ds0=R)


def linattn_step(q, k, v, g, state, scale, slots=None):
    """q, k [B, Hk, dk], v [B, H, dv], g [B, H] or [H], state [pool, H, dk, dv]; returns (out, state)."""
    state = np.array(state, np.float64)
    B, H, dv = v.shape
    share = H // q.shape[1]
    out = np.zeros((B, H, dv))
    g = np.broadcast_to(np.asarray(g, np.float64), (B, H))
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < len(state):
            continue
        for h in range(H):
            qh, kh = np.asarray(q[b, h // share], np.float64), np.asarray(k[b, h // share], np.float64)
            state[s, h] = np.exp(g[b, h]) * state[s, h] + np.outer(kh, np.asarray(v[b, h], np.float64))
            out[b, h] = scale * qh @ state[s, h]
    return out, state
