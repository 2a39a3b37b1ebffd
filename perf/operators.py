"""Cases, plain forms and exact values for the operators of a linear-attention block over image and
video tokens: the residual addition with its root-mean-square norm, the rotary positions of
several axes, and the linear attention with a decay for each head.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes
one pass (the plain form in float32 torch operations, or with ``own`` the library's operator) and
``exact`` evaluates the definition in float64.

Where the sizes come from: 128 images of 197 tokens with 192, 384 or 768 channels are the Vim-Ti and
Vim-S layers of this repository's benchmark, 8 x 6085 tokens its 1248-pixel workload, and 32 x 56 x 56
pixels of 512 channels its SS2D workload; heads are 64 channels wide unless a case says otherwise.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
EPS = 1e-5
CHUNK = 64  # tokens per block of the plain form of the linear attention


def _device():
    return torch.device("cuda")


# ------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token of each of 4 sequences between two layers of a decoding loop: latency counts
        dict(name="norm_step", op="norm", rows=4, dim=384, x="bf16", res="f32", out="bf16", group=0),
        # the 1248-pixel workload's tokens on their way into a projection in 8 bits, a scale per 128 channels
        dict(name="norm_hires_fp8", op="norm", rows=8 * 6085, dim=768, x="bf16", res="bf16", out="fp8", group=128),
        # the gradient of the norm of a Vim-Ti layer with its float32 residual stream
        dict(name="norm_train", op="norm_bwd", rows=128 * 197, dim=384, x="bf16", res="f32"),
        # queries and keys of 128 images: row and column positions, channels rotated in neighbouring pairs
        dict(name="rope_image", op="rope", batch=128, seqlen=197, heads=6, kheads=6, dim=64, rot=64, axes=2, x="bf16",
             interleaved=True, inverse=False),
        # the gradient through the rotation of 8 frames of 28 x 28 patches: time, height and width,
        # 4 key heads for 12 query heads, three quarters of each head rotated in half-split pairs, float32
        dict(name="rope_video_grad", op="rope", batch=2, seqlen=8 * 28 * 28, heads=12, kheads=4, dim=128, rot=96,
             axes=3, x="f32", interleaved=False, inverse=True),
        # one image in float32: few heads and a ragged last block, latency counts
        dict(name="linattn_one_image", op="linattn", batch=1, seqlen=197, heads=6, kheads=6, dk=64, dv=64, x="f32",
             decay="token", state=False, ragged=False),
        # the Vim-Ti batch with a fixed decay per head: many short sequences
        dict(name="linattn_vim_ti", op="linattn", batch=128, seqlen=197, heads=6, kheads=6, dk=64, dv=64, x="bf16",
             decay="head", state=False, ragged=False),
        # 1248-pixel prompts of unequal length, keys shared by 3 heads each, going on from a state
        dict(name="linattn_hires", op="linattn", batch=8, seqlen=6085, heads=6, kheads=2, dk=128, dv=64, x="bf16",
             decay="token", state=True, ragged=True),
        # training on the 56 x 56 pixels of the SS2D workload
        dict(name="linattn_train", op="linattn_bwd", batch=32, seqlen=3136, heads=8, kheads=8, dk=64, dv=64, x="bf16",
             decay="token", state=False, ragged=False),
        # float32 training on few long sequences with small shared keys (d_state 32) and wide values
        dict(name="linattn_train_f32", op="linattn_bwd", batch=2, seqlen=1001, heads=8, kheads=2, dk=32, dv=128,
             x="f32", decay="head", state=True, ragged=True),
        # single tokens: one sequence (latency), and 256 running sequences in a pool of 320 states
        dict(name="linattn_step_one", op="step", batch=1, pool=1, heads=6, kheads=6, dk=64, dv=64, x="bf16",
             decay="token"),
        dict(name="linattn_step_256", op="step", batch=256, pool=320, heads=12, kheads=4, dk=64, dv=64, x="bf16",
             decay="token"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "linattn", "linattn", "linattn_bwd", "step"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        dim = 8 * _log_int(rng, 4, 256)
        case = dict(op=op, rows=_log_int(rng, 1, min(50000, 30000000 // dim)), dim=dim, x=x,
                    res=rng.choice(["f32", x]))
        if op == "norm":
            case["out"] = rng.choice([x, "fp8"])
            case["group"] = rng.choice([0, 128]) if case["out"] == "fp8" else 0
        return case
    if op == "rope":
        axes, dim = rng.choice([1, 2, 3]), 8 * rng.randint(4, 16)
        heads = rng.choice([2, 4, 6, 12])
        case = dict(op=op, batch=_log_int(rng, 1, 64), seqlen=0, heads=heads,
                    kheads=rng.choice([h for h in (1, 2, 4, 6, 12) if heads % h == 0]), dim=dim,
                    rot=dim if rng.random() < 0.6 else 2 * rng.randint(axes, dim // 2), axes=axes, x=x,
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4)
        case["seqlen"] = _log_int(rng, 1, min(6085, 30000000 // (case["batch"] * heads * dim)))
        return case
    heads = rng.choice([1, 2, 4, 6, 8, 12])
    case = dict(op=op, batch=0, heads=heads, kheads=rng.choice([h for h in (1, 2, 4, 6, 8, 12) if heads % h == 0]),
                dk=rng.choice([16, 24, 32, 64, 64, 96, 128]), dv=rng.choice([32, 40, 64, 64, 128]), x=x,
                decay=rng.choice(["token", "head"]))
    wide = heads * max(case["dk"], case["dv"])
    if op == "step":
        case["batch"] = _log_int(rng, 1, min(512, 10000000 // (heads * case["dk"] * case["dv"])))
        case["pool"] = case["batch"] + rng.randint(0, 8)
        return case
    case["batch"] = _log_int(rng, 1, 64)
    case["seqlen"] = _log_int(rng, 1, min(6085, (30000000 if op == "linattn" else 12000000) // (case["batch"] * wide)))
    case["state"], case["ragged"] = rng.random() < 0.5, rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------------------------
# inputs


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": FP8}[name]


def _log_decay(gen, heads, *lead):
    """-dt * A with dt log-uniform on [1e-3, 1e-1] and A = 1, 2, ... over the heads: the step and
    decay initialisation of this repository's scans."""
    dev = _device()
    dt = torch.exp(torch.rand(*lead, heads, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
    return -dt * torch.arange(1, heads + 1, device=dev, dtype=torch.float32)


def _positions(case):
    """Token positions along the axes of the smallest grid that holds the tokens, the first token
    (the class token) at the origin."""
    T, axes, dev = case["seqlen"], case["axes"], _device()
    side = max(1, math.ceil(T ** (1.0 / axes)))
    t = torch.clamp(torch.arange(T, device=dev) - 1, min=0)
    return torch.stack([(t // side ** (axes - 1 - a)) % side for a in range(axes)], -1).float().contiguous()


def _frequencies(case):
    """The pairs of a head shared out over the axes, each axis with frequencies from 1 down to 1e-4."""
    pairs, axes = case["rot"] // 2, case["axes"]
    axis = [p * axes // pairs for p in range(pairs)]
    first = [axis.index(a) for a in axis]
    count = [axis.count(a) for a in axis]
    freq = [10000.0 ** (-(p - f) / c) for p, (f, c) in enumerate(zip(first, count))]
    return (torch.tensor(freq, dtype=torch.float32, device=_device()),
            torch.tensor(axis, dtype=torch.int32, device=_device()))


def prepare(case, seed):
    dev, op, dt = _device(), case["op"], _dtype(case["x"])
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)
    s = dict(case=case)
    if op in ("norm", "norm_bwd"):
        rows, dim = case["rows"], case["dim"]
        s["w"] = 1.0 + 0.1 * normal(dim)
        if op == "norm":
            s["x"], s["res"] = normal(rows, dim).to(dt), (2.0 * normal(rows, dim)).to(_dtype(case["res"]))
            return s
        s["r"] = (2.0 * normal(rows, dim)).to(_dtype(case["res"]))
        s["rstd"] = torch.rsqrt(s["r"].float().square().mean(-1) + EPS)
        s["dy"], s["dres"] = normal(rows, dim).to(dt), normal(rows, dim).to(_dtype(case["res"]))
        return s
    H, Hk = case["heads"], case["kheads"]
    if op == "rope":
        # q and k as one projection wrote them, side by side
        qk = normal(case["batch"], case["seqlen"], H + Hk, case["dim"]).to(dt)
        s["q"], s["k"] = qk[:, :, :H], qk[:, :, H:]
        s["pos"] = _positions(case)
        s["inv_freq"], s["axis"] = _frequencies(case)
        return s
    B, dk, dv = case["batch"], case["dk"], case["dv"]
    lead = (B,) if op == "step" else (B, case["seqlen"])
    # q and k as the rotation wrote them; v as a slice of a projection that also holds a gate
    s["q"], s["k"] = normal(*lead, Hk, dk).to(dt), normal(*lead, Hk, dk).to(dt)
    s["v"] = normal(*lead, 2 * H, dv).to(dt)[..., :H, :]
    s["g"] = _log_decay(gen, H, *(lead if case["decay"] == "token" else ()))
    s["scale"] = dk ** -0.5
    if op == "step":
        s["state"] = normal(case["pool"], H, dk, dv)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=dev)[:B].to(torch.int32)
        return s
    s["state"] = normal(B, H, dk, dv) if case["state"] else None
    s["lengths"] = None
    if case["ragged"]:
        lo = max(1, case["seqlen"] // 2)
        s["lengths"] = torch.randint(lo, case["seqlen"] + 1, (B,), generator=gen, device=dev).to(torch.int32)
    if op == "linattn_bwd":
        s["dout"] = normal(*lead, H, dv).to(dt)
        s["dstate"] = normal(B, H, dk, dv) if case["state"] else None
    return s


# ------------------------------------------------------------------------------------------------
# plain forms


def _plain_norm(s):
    case = s["case"]
    r = s["x"].float() + s["res"].float()
    rstd = torch.rsqrt((r * r).mean(-1) + EPS)
    y = r * rstd[:, None] * s["w"]
    res = r.to(s["res"].dtype)
    if case["out"] != "fp8":
        return y.to(_dtype(case["out"])), res, rstd
    rows, dim = y.shape
    group = case["group"] or dim
    y = torch.nn.functional.pad(y, (0, -dim % group)).view(rows, -1, group)
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    return (y / scale[..., None]).view(rows, -1)[:, :dim].to(FP8), scale, res, rstd


def _plain_norm_bwd(s):
    r, dy = s["r"].float(), s["dy"].float()
    rh = r * s["rstd"][:, None]
    wdy = dy * s["w"]
    dr = s["rstd"][:, None] * (wdy - rh * (rh * wdy).mean(-1, keepdim=True)) + s["dres"].float()
    return dr.to(s["dy"].dtype), dr.to(s["r"].dtype), (dy * rh).sum(0)


def _plain_rotate(x, cos, sin, rot, interleaved):
    f = x.float()
    head = f[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., : rot // 2], head[..., rot // 2:])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1)
    return torch.cat([y, f[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    angle = s["pos"][:, s["axis"].long()] * s["inv_freq"]
    cos, sin = torch.cos(angle)[None, :, None], torch.sin(angle)[None, :, None]
    sin = -sin if case["inverse"] else sin
    return tuple(_plain_rotate(s[n], cos, sin, case["rot"], case["interleaved"]) for n in ("q", "k"))


def _segment_sums(g):
    """[..., n] -> [..., n, n]: the sum of g over (j, i] at [i, j], -inf above the diagonal.  Each
    sum starts at its own j, so that long rows lose no precision."""
    n = g.shape[-1]
    at = torch.arange(n, device=g.device)
    below = at[:, None] > at[None, :]
    sums = torch.where(below, g[..., :, None].expand(*g.shape, n), g.new_zeros(())).cumsum(-2)
    return sums.masked_fill(at[:, None] < at[None, :], -math.inf)


def _plain_linattn(s, q, k, v, g, state):
    """Blocks of CHUNK tokens: inside a block the masked product of the scores, between blocks the
    states, which a matrix of the decays between blocks sums up."""
    case = s["case"]
    B, T, H, Hk, dk, dv = (case[n] for n in ("batch", "seqlen", "heads", "kheads", "dk", "dv"))
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    g = g.expand(B, T, H)
    if s["lengths"] is not None:
        live = torch.arange(T, device=q.device)[None, :] < s["lengths"][:, None]
        g, k, v = g * live[..., None], k * live[..., None, None], v * live[..., None, None]
    blocks = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(B, n, CHUNK, x.shape[2], -1).permute(0, 3, 1, 2, 4)
    heads = lambda x: blocks(x).repeat_interleave(H // Hk, 1)
    q, k, v, g = heads(q), heads(k), blocks(v), blocks(g[..., None])[..., 0]
    G = g.cumsum(-1)
    total = G[..., -1]
    scores = (q @ k.transpose(-1, -2)) * torch.exp(_segment_sums(g))
    per_block = (k * torch.exp(total[..., None] - G)[..., None]).transpose(-1, -2) @ v
    # the decays from the end of block j (the state given: the start) to the start of block i
    between = torch.exp(_segment_sums(torch.nn.functional.pad(total, (1, 0))))
    first = state if state is not None else per_block.new_zeros(B, H, dk, dv)
    states = between @ torch.cat([first[:, :, None], per_block], 2).flatten(-2)
    states = states.view(B, H, n + 1, dk, dv)
    out = scores @ v + torch.exp(G)[..., None] * (q @ states[:, :, :n])
    out = (s["scale"] * out).permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, dv)[:, :T]
    if s["lengths"] is not None:
        out = out * live[..., None, None]
    return out, states[:, :, n]


def _plain_linattn_fwd(s):
    out, last = _plain_linattn(s, s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["state"])
    return out.to(s["q"].dtype), last


def _plain_linattn_bwd(s):
    ins = [s["q"].float(), s["k"].float(), s["v"].float(), s["g"]]
    ins += [s["state"]] if s["state"] is not None else []
    ins = [x.detach().requires_grad_() for x in ins]
    out, last = _plain_linattn(s, *ins[:4], ins[4] if len(ins) > 4 else None)
    outs, grads = [out], [s["dout"].float()]
    if s["dstate"] is not None:
        outs, grads = outs + [last], grads + [s["dstate"]]
    got = torch.autograd.grad(outs, ins, grads)
    return tuple(x.to(s["q"].dtype) for x in got[:3]) + tuple(got[3:])


def _plain_step(s):
    case = s["case"]
    share = case["heads"] // case["kheads"]
    q, k = (s[n].float().repeat_interleave(share, 1) for n in ("q", "k"))
    at = s["slots"].long()
    new = s["state"][at] * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    s["state"][at] = new
    return (s["scale"] * (q[..., None] * new).sum(-2)).to(s["q"].dtype), s["state"]


def _run_plain(s):
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "rope": _plain_rope, "linattn": _plain_linattn_fwd,
            "linattn_bwd": _plain_linattn_bwd, "step": _plain_step}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------
# the library's operators


def _run_own(s):
    import selective_state_space_41_amd as V

    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, scale, res, rstd = V.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS, out_dtype=_dtype(case["out"]),
                                            group=case["group"])
        return (y, res, rstd) if scale is None else (y, scale, res, rstd)
    if op == "norm_bwd":
        g = V.rmsnorm_bwd(s["dy"], s["r"], s["w"], s["rstd"], dresidual_out=s["dres"])
        return g["dx"], g["dresidual"], g["dweight"]
    if op == "rope":
        return V.rope_axes(s["q"], s["k"], s["pos"], s["inv_freq"], s["axis"], interleaved=case["interleaved"],
                           inverse=case["inverse"])
    if op == "linattn":
        return V.linattn_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], initial_state=s["state"],
                             lengths=s["lengths"])
    if op == "linattn_bwd":
        g = V.linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], scale=s["scale"], initial_state=s["state"],
                          lengths=s["lengths"], dfinal_state=s["dstate"])
        names = ["dq", "dk", "dv", "dlog_decay"] + (["dinitial_state"] if s["state"] is not None else [])
        return tuple(g[n] for n in names)
    return V.linattn_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"], slots=s["slots"]), s["state"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    size = {"bf16": 2, "f32": 4, "fp8": 1}
    e, op = size[case["x"]], case["op"]
    if op in ("norm", "norm_bwd"):
        n, dim, er = case["rows"] * case["dim"], case["dim"], size[case["res"]]
        if op == "norm":
            scales = 0 if case["out"] != "fp8" else 4 * case["rows"] * (-(-dim // (case["group"] or dim)))
            return {"bytes": n * (e + 2 * er + size[case["out"]]) + 4 * dim + 4 * case["rows"] + scales, "flops": 6 * n}
        return {"bytes": n * (2 * e + 3 * er) + 8 * dim + 4 * case["rows"], "flops": 12 * n}
    H, Hk, B = case["heads"], case["kheads"], case["batch"]
    if op == "rope":
        T = case["seqlen"]
        n = B * T * (H + Hk) * case["dim"]
        return {"bytes": 2 * e * n + 4 * T * case["axes"] + 8 * (case["rot"] // 2), "flops": 3 * n}
    dk, dv = case["dk"], case["dv"]
    if op == "step":
        n = B * H * dk * dv
        return {"bytes": 8 * n + e * B * (2 * Hk * dk + 2 * H * dv) + 4 * (B * H if case["decay"] == "token" else H),
                "flops": 5 * n}
    T = case["seqlen"]
    decays = 4 * (B * T * H if case["decay"] == "token" else H)
    states = 4 * B * H * dk * dv
    qk, vo = e * B * T * Hk * dk, e * B * T * H * dv
    if op == "linattn":
        return {"bytes": 2 * qk + 2 * vo + decays + states * (2 if case["state"] else 1), "flops": 4 * B * T * H * dk * dv}
    return {"bytes": 4 * qk + 3 * vo + 2 * decays + (3 * states if case["state"] else 0), "flops": 12 * B * T * H * dk * dv}


# ------------------------------------------------------------------------------------------------
# the definitions in float64


def _exact_norm(s):
    case = s["case"]
    r = s["x"].double() + s["res"].double()
    rstd = 1.0 / torch.sqrt((r ** 2).sum(-1) / case["dim"] + EPS)
    y = s["w"].double() * (r * rstd[:, None])
    if case["out"] != "fp8":
        return y, r, rstd
    codes, scales = [], []
    for first in range(0, case["dim"], case["group"] or case["dim"]):
        part = y[:, first: first + (case["group"] or case["dim"])]
        scales.append(part.abs().max(-1).values / FP8_MAX)
        codes.append(part / scales[-1][:, None])  # the value that the code is the nearest one to
    return torch.cat(codes, 1), torch.stack(scales, 1), r, rstd


def _exact_norm_bwd(s):
    r, dy, w, rstd = (s[n].double() for n in ("r", "dy", "w", "rstd"))
    # d(rstd)/dr_i = -rstd^3 r_i / dim, from the chain rule
    along = (dy * w * r).sum(-1, keepdim=True) * rstd[:, None] ** 3 / s["case"]["dim"]
    dr = dy * w * rstd[:, None] - r * along + s["dres"].double()
    return dr, dr, torch.einsum("rd,rd,r->d", dy, r, rstd)


def _exact_rope(s):
    case = s["case"]
    angle = s["inv_freq"].double() * s["pos"].double()[:, s["axis"].long()]
    turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[None, :, None]
    outs = []
    for x in (s["q"], s["k"]):
        y, rot = x.double().clone(), case["rot"]
        first = torch.arange(rot // 2, device=x.device) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else rot // 2)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_inputs(s):
    """Per head and in float64, [T or one][B, H, ...] with what lies past a row's length taken out."""
    case = s["case"]
    share = case["heads"] // case["kheads"]
    q, k = (s[n].double().repeat_interleave(share, -2) for n in ("q", "k"))
    return q, k, s["v"].double()


def _exact_linattn(s, keep=False):
    """The recurrence token by token; with keep also the state before every token and after the last."""
    case = s["case"]
    B, T, H = case["batch"], case["seqlen"], case["heads"]
    q, k, v = _exact_inputs(s)
    decay = torch.exp(s["g"].double()).expand(B, T, H)
    S = s["state"].double() if s["state"] is not None else q.new_zeros(B, H, case["dk"], case["dv"])
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=q.device)
    out, kept = torch.zeros_like(v), []
    for t in range(T):
        live = (lengths > t)[:, None, None, None]
        if keep:
            kept.append(S)
        S = torch.where(live, decay[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :], S)
        out[:, t] = torch.where(live[..., 0], s["scale"] * torch.matmul(q[:, t, :, None, :], S)[:, :, 0], out[:, t])
    return (out, S, kept + [S]) if keep else (out, S)


def _exact_linattn_bwd(s):
    """The adjoint recurrence: R_t = dL/dS_t, token by token from the last."""
    case = s["case"]
    B, T, H, Hk = case["batch"], case["seqlen"], case["heads"], case["kheads"]
    _, _, S = _exact_linattn(s, keep=True)
    q, k, v = _exact_inputs(s)
    decay = torch.exp(s["g"].double()).expand(B, T, H)
    dout = s["scale"] * s["dout"].double()
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=q.device)
    R = s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(S[0])
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(decay)
    for t in range(T - 1, -1, -1):
        live = (lengths > t)[:, None, None]
        at = torch.where(live[..., None], R + q[:, t, :, :, None] * dout[:, t, :, None, :], R)
        dq[:, t] = torch.where(live, torch.matmul(S[t + 1], dout[:, t, :, :, None])[..., 0], dq[:, t])
        dk[:, t] = torch.where(live, torch.matmul(at, v[:, t, :, :, None])[..., 0], dk[:, t])
        dv[:, t] = torch.where(live, torch.matmul(k[:, t, :, None, :], at)[:, :, 0], dv[:, t])
        dg[:, t] = torch.where(live[..., 0], decay[:, t] * (S[t] * at).sum((-1, -2)), dg[:, t])
        R = torch.where(live[..., None], decay[:, t, :, None, None] * at, at)
    dq, dk = (x.view(B, T, Hk, H // Hk, -1).sum(3) for x in (dq, dk))
    dg = dg if case["decay"] == "token" else dg.sum((0, 1))
    return (dq, dk, dv, dg) + ((R,) if s["state"] is not None else ())


def _exact_step(s):
    q, k, v = _exact_inputs(s)
    pool, rows = s["state"].double().clone(), s["slots"].long()
    S = pool[rows] * torch.exp(s["g"].double())[..., None, None] + torch.einsum("bhi,bhj->bhij", k, v)
    pool[rows] = S
    return s["scale"] * torch.einsum("bhi,bhij->bhj", q, S), pool


def exact(case, seed):
    s = prepare(case, seed)
    # the states before every token are held for the gradient: past 100 GB there is no value
    if case["op"] == "linattn_bwd" and 8 * case["batch"] * case["seqlen"] * case["heads"] * case["dk"] * case["dv"] > 100e9:
        return None
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "rope": _exact_rope, "linattn": _exact_linattn,
            "linattn_bwd": _exact_linattn_bwd, "step": _exact_step}[case["op"]](s)
