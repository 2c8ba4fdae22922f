"""Measured cases of the operators on the way of the indexer's keys and queries: layer norm (forward, backward with the
weight's and bias' gradients), its 8-bit activation checkpoints, and rotary positions of several axes.

Shapes follow the repository's workloads (64 indexer heads of 128, 8,192 queries of a shard, a 131,072-token prompt) or
are generic hidden sizes.  With ``own`` false ``run`` computes an operator in elementary torch operations; with ``own``
true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32  # elements that share one E8M0 scale
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token's key of each of 64 sequences, normalised on its way to the rotation: latency
        dict(name="norm_tokens", op="norm", n=64, heads=1, d=128, x="bf16", y="bf16"),
        # the hidden states of a long chunk before the indexer's projections; odd token count
        dict(name="norm_hidden", op="norm", n=5003, heads=1, d=7168, x="bf16", y="bf16"),
        # the gradient of a 131,072-token prompt's keys (fp32, from the indexer's backward) through their norm
        dict(name="grad_prompt", op="grad", n=131072, heads=1, d=128, x="bf16", dy="fp32", dx="bf16"),
        # a shard's hidden states in training: wide rows, everything in bf16
        dict(name="grad_hidden", op="grad", n=8192, heads=1, d=5120, x="bf16", dy="bf16", dx="bf16"),
        # the first tokens of a short sequence, every head's query normalised by itself; an odd width, fp32
        dict(name="grad_ragged", op="grad", n=77, heads=6, d=201, x="fp32", dy="fp32", dx="fp32"),
        # a training step of the prompt's keys whose norm keeps its input in FP8: forward, then backward from the codes
        dict(name="checkpoint_prompt", op="checkpoint", n=131072, heads=1, d=128, fmt="fp8", x="bf16", dy="fp32",
             dx="bf16"),
        # the same of a shard's hidden states, kept in MXFP8
        dict(name="checkpoint_hidden", op="checkpoint", n=8192, heads=1, d=4096, fmt="mxfp8", x="bf16", dy="bf16",
             dx="bf16"),
        # a small batch of queries, eight heads of 96 each, kept in FP8
        dict(name="checkpoint_small", op="checkpoint", n=301, heads=8, d=96, fmt="fp8", x="bf16", dy="bf16", dx="bf16"),
        # one decoded token's queries behind an image: latency
        dict(name="axes_token", op="axes", n=1, heads=64, d=128, rot=128, first=0, layout="half", sections="16,24,24",
             cycle=False, restart=False, text=70000, high=30, wide=41, grad=False),
        # the queries of 8,192 video tokens: time, height and width in turn over the pairs
        dict(name="axes_video", op="axes", n=8192, heads=64, d=128, rot=64, first=64, layout="interleaved",
             sections="12,10,10", cycle=True, restart=False, text=211, high=24, wide=36, grad=False),
        # the gradient of an image's queries on its way to a bf16 projection: height and width with frequencies of
        # their own, odd token count, narrow heads
        dict(name="axes_gradient", op="axes", n=5003, heads=24, d=64, rot=64, first=0, layout="half", sections="16,16",
             cycle=False, restart=True, text=0, high=71, wide=71, grad=True),
        # the keys of a 131,072-token prompt of video rotated and written into an MXFP8 cache, and read back
        dict(name="axes_write", op="axes_write", n=131072, heads=1, d=128, rot=64, first=0, layout="half",
             sections="8,12,12", cycle=False, restart=False, text=33, high=45, wide=80, fmt="mxfp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_sections(rng, pairs):
    """Pairs of each of two or three axes."""
    if rng.random() < 0.3:
        return f"{pairs // 2},{pairs - pairs // 2}"
    a = pairs // 3 if rng.random() < 0.5 else pairs // 4
    b = min((pairs - a) // 2, pairs // 3)  # what fits in turn
    return f"{pairs - 2 * b},{b},{b}"


def draw(rng):
    op = rng.choice(["norm", "grad", "checkpoint", "axes", "axes_write"])
    if op in ("axes", "axes_write"):
        write = op == "axes_write"
        heads = rng.choice([1, 1, 4, 32]) if write else rng.choice([1, 4, 8, 24, 40, 64])
        d = 128 if write else rng.choice([64, 128])
        rot = rng.choice([d // 4, d // 2, d])
        c = dict(op=op, n=_log(rng, 1, max(2, min(1 << 17, (1 << 25) // (heads * d)))), heads=heads, d=d, rot=rot,
                 first=rng.choice([0, d - rot]), layout=rng.choice(["half", "interleaved"]),
                 sections=_draw_sections(rng, rot // 2), cycle=rng.random() < 0.5, restart=rng.random() < 0.3,
                 text=_log(rng, 1, 1 << 19), high=_log(rng, 1, 90), wide=_log(rng, 1, 90))
        if write:
            return dict(c, fmt=rng.choice(["bf16", "fp8", "mxfp8", "mxfp4"]))
        return dict(c, grad=rng.random() < 0.4)
    pick = lambda: rng.choice(["bf16", "bf16", "fp32"])  # noqa: E731
    if op == "checkpoint":
        d = 32 * _log(rng, 1, 256)
    else:
        d = rng.choice([64, 128, _log(rng, 8, 8192), 8 * _log(rng, 8, 1024)])
    heads = rng.choice([1, 1, 4, 24]) if d <= 256 else 1
    c = dict(op=op, n=_log(rng, 1, max(2, min(1 << 17, (1 << 25) // (heads * d)))), heads=heads, d=d, x=pick())
    if op == "norm":
        return dict(c, y=pick())
    if op == "grad":
        return dict(c, dy=pick(), dx=pick())
    return dict(c, fmt=rng.choice(["fp8", "mxfp8"]), dy=pick(), dx=pick())


def _shape(case):
    n, h, d = case["n"], case["heads"], case["d"]
    return (n, d) if h == 1 else (n, h, d)


def _sections(case):
    return tuple(int(x) for x in case["sections"].split(","))


def _axes(case):
    """The axis of every pair: the sections one behind the other, or in turn (axis a > 0 takes pairs a, a + A, a + 2 A,
    ..., the first axis the others)."""
    sections = _sections(case)
    A = len(sections)
    if not case["cycle"]:
        return [a for a, s in enumerate(sections) for _ in range(s)]
    axis = [0] * sum(sections)
    for a in range(1, A):
        for j in range(sections[a]):
            axis[a + j * A] = a
    return axis


def _frequencies(case):
    """Radians a position of every pair: one geometric series over all pairs, or one over each axis' own."""
    base = 10000.0 if case["d"] == 64 else 1000000.0
    axis, f = _axes(case), []
    for i, a in enumerate(axis):
        if case["restart"]:
            f.append(base ** (-axis[:i].count(a) / axis.count(a)))
        else:
            f.append(base ** (-i / len(axis)))
    return torch.tensor(f, device=DEV, dtype=torch.float64)


def _positions(case):
    """Positions [n][axes]: frames of high x wide tokens behind `text` tokens of text."""
    i = torch.arange(case["n"], device=DEV)
    hw = case["high"] * case["wide"]
    p = [i // hw, (i // case["wide"]) % case["high"], i % case["wide"]][3 - len(_sections(case)):]
    return (torch.stack(p, 1) + case["text"]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    op, n, h, d = case["op"], case["n"], case["heads"], case["d"]
    s = dict(case=dict(case))
    if op in ("norm", "grad", "checkpoint"):
        # rows of different sizes and offsets, as tokens have, with a weight near 1
        size, off = torch.exp(0.5 * normal(n, h, 1)), 0.3 * normal(n, h, 1)
        s["x"] = (normal(n, h, d) * size + off).to(DTYPES[case["x"]]).view(_shape(case))
        s["weight"], s["bias"] = 1 + 0.2 * normal(d), 0.1 * normal(d)
        if op != "norm":
            s["dy"] = (normal(n, h, d) / math.sqrt(d)).to(DTYPES[case["dy"]]).view(_shape(case))
        if op == "grad":  # kept by the forward pass
            s["stats"] = torch.cat(_statistics(s["x"].double()), -1).float()  # [..][2]: mean, reciprocal deviation
    else:
        grad = op == "axes" and case["grad"]
        s["x"] = (normal(n, h, d) * torch.exp(0.5 * normal(n, 1, 1))).to(torch.float32 if grad else torch.bfloat16)
        if op == "axes_write" and h == 1:
            s["x"] = s["x"].view(n, d)
        s["pos"], s["freq"] = _positions(case), _frequencies(case)
        s["axis"] = torch.tensor(_axes(case), device=DEV)
        if op == "axes_write":
            fmt, rows = case["fmt"], _shape(case)[:-1]
            s["codes"] = torch.zeros(rows + (d // 2 if fmt == "mxfp4" else d,), device=DEV,
                                     dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8)
            s["scale"] = None
            if fmt == "fp8":
                s["scale"] = torch.ones(n, device=DEV)
            elif fmt != "bf16":
                s["scale"] = torch.zeros(rows + (d // BLOCK,), device=DEV, dtype=torch.uint8)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The plan that a user's program keeps beside its inputs, and what its forward pass kept."""
    import exact_top_token_amd as hk
    c = s["case"]
    if c["op"] == "grad":
        s["saved"] = hk.NormSaved(s["x"], None, s["stats"], None)
    if c["op"] in ("axes", "axes_write"):
        s["plan"] = hk.Rotary(c["rot"], first=c["first"], layout=c["layout"], device=DEV, sections=_sections(c),
                              cycle=c["cycle"], restart=c["restart"], base=10000.0 if c["d"] == 64 else 1000000.0)


# ------------------------------------------------------------- plain forms

def _statistics(x):
    """Mean and reciprocal deviation of rows, in x's type."""
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    return mean, ((c * c).mean(-1, keepdim=True) + EPS) ** -0.5


def _norm_back(dy, x, mean, rstd, weight):
    """Gradients in 32 bits; mean and rstd [..][1]."""
    d = x.shape[-1]
    hat = (x - mean) * rstd
    g = dy * weight
    dx = rstd * (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True))
    return dx, (dy * hat).view(-1, d).sum(0), dy.reshape(-1, d).sum(0)


def _to_e4m3(v):
    """Values of E4M3, of 64-bit values: to nearest, ties to even, at most 448."""
    a = v.abs().clamp_max(448.0)
    # the power of two below, by its bits (exp2 may be off by a rounding, which moves ties), over the 8 steps to the next
    step = (a.clamp_min(2.0 ** -6).view(torch.int64) & (0x7ff << 52)).view(torch.float64) / 8
    return torch.copysign(torch.round(a / step) * step, v)


def _to_e2m1(v):
    a = v.abs().clamp_max(6.0)
    r = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return torch.copysign(r, v)


def _stored(y, fmt, over):
    """What rows y (32 bits) stand for once they are stored; an FP8 scale covers the last `over` axes."""
    if fmt == "bf16":
        return y.to(torch.bfloat16).float()
    if fmt == "fp8":
        amax = y.abs().amax(tuple(range(-over, 0)), keepdim=True)
        scale = (amax.double() / 448.0).float()  # a quotient rounded once: the codes of many ties hang on it
        scale = torch.where(amax > 0, scale.clamp_min(2.0 ** -126), torch.ones_like(amax))
        return _to_e4m3(y.double() / scale.double()).float() * scale
    b = y.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax)[1] - 1 - (8 if fmt == "mxfp8" else 2)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    f = ((e.long() + 1023) << 52).view(torch.float64)
    v = (_to_e4m3 if fmt == "mxfp8" else _to_e2m1)(b.double() / f)
    return (v * f).float().flatten(-2)


def _rotate(s, x):
    """Rows x [n][heads][d] in 32 bits; angles in 64."""
    c = s["case"]
    first, rot = c["first"], c["rot"]
    angle = s["pos"].double()[:, s["axis"]] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c.get("grad"):
        sin = -sin
    y = x.clone()
    part = x[..., first:first + rot]
    if c["layout"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        y[..., first:first + rot] = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        y[..., first:first + rot] = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return y


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "axes":
        return _rotate(s, s["x"].float()).to(torch.bfloat16)
    if op == "axes_write":
        y = _rotate(s, s["x"].view(c["n"], c["heads"], c["d"]).float())
        return _stored(y, c["fmt"], 2).to(torch.bfloat16).view(s["x"].shape)
    x = s["x"].float()
    if op == "grad":
        dx, dw, db = _norm_back(s["dy"].float(), x, s["stats"][..., :1], s["stats"][..., 1:], s["weight"])
        return {"dx": dx.to(DTYPES[c["dx"]]), "dweight": dw, "dbias": db}
    mean, rstd = _statistics(x)
    y = (x - mean) * rstd * s["weight"] + s["bias"]
    if op == "norm":
        return y.to(DTYPES[c["y"]])
    dx, dw, db = _norm_back(s["dy"].float(), _stored(x, c["fmt"], 1), mean, rstd, s["weight"])
    return {"y": y.to(s["x"].dtype), "dx": dx.to(DTYPES[c["dx"]]), "dweight": dw, "dbias": db}


def run(state):
    if not own:
        return _plain(state)
    import exact_top_token_amd as hk
    s, c = state, state["case"]
    op = c["op"]
    if op == "axes":
        return hk.rotary(s["x"], s["plan"], q_pos=s["pos"], backward=c["grad"], out_dtype=torch.bfloat16)
    if op == "axes_write":
        hk.cache_write(s["x"], s["codes"], s["scale"], fmt=c["fmt"], rotary=s["plan"], q_pos=s["pos"])
        return hk.cache_read(s["codes"], s["scale"], fmt=c["fmt"])
    if op == "norm":
        return hk.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=DTYPES[c["y"]])
    if op == "grad":
        return hk.layer_norm_backward(s["dy"], s["saved"], s["weight"], dx_dtype=DTYPES[c["dx"]])
    y, saved = hk.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, save=c["fmt"])
    return {"y": y, **hk.layer_norm_backward(s["dy"], saved, s["weight"], dx_dtype=DTYPES[c["dx"]])}


def work(case):
    op, n, h, d = case["op"], case["n"], case["heads"], case["d"]
    e, rows = n * h * d, n * h
    size = {"bf16": 2, "fp32": 4, "fp8": 1, "mxfp8": 1 + 1 / BLOCK, "mxfp4": 0.5 + 1 / BLOCK}
    if op in ("axes", "axes_write"):
        bytes_ = e * ((4 if case.get("grad") else 2) + 2) + 4 * n * len(_sections(case))
        if op == "axes_write":  # codes out, codes in again
            bytes_ += 2 * e * size[case["fmt"]]
        return {"bytes": bytes_, "flops": 3 * n * h * case["rot"] + (4 * e if op == "axes_write" else 0)}
    if op == "norm":
        return {"bytes": e * (size[case["x"]] + size[case["y"]]) + 8 * d, "flops": 8 * e}
    if op == "grad":
        return {"bytes": e * (size[case["x"]] + size[case["dy"]] + size[case["dx"]]) + 8 * rows + 12 * d, "flops": 14 * e}
    # forward: x in, y and the codes out; backward: codes and dy in, dx out
    return {"bytes": e * (2 * size[case["x"]] + 2 * size[case["fmt"]] + size[case["dy"]] + size[case["dx"]])
            + (16 + (8 if case["fmt"] == "fp8" else 0)) * rows + 20 * d, "flops": 24 * e}


# ------------------------------------------------- the definitions in 64 bits

def _nearest(v, table):
    """The nearest value of a table of magnitudes (ties to the even place), with v's sign."""
    t = torch.tensor(table, device=DEV, dtype=torch.float64)
    mid = (t[1:] + t[:-1]) / 2
    a = v.abs()
    lo = torch.bucketize(a, mid)
    hi = torch.bucketize(a, mid, right=True)
    return torch.where(lo == hi, t[lo], t[(lo + lo % 2).clamp_max(len(table) - 1)]) * torch.sign(v)


def _exact_stored(y, fmt):
    """What rows y [n][anything] in 64 bits stand for once stored, one FP8 scale a row."""
    e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1]
    if fmt == "bf16":
        return y
    if fmt == "fp8":
        top = y.abs().amax(1, keepdim=True)
        scale = torch.where(top > 0, (top / 448).float().double().clamp_min(2.0 ** -126), 1.0)
        return _nearest(y / scale, e4m3) * scale
    b = y.reshape(y.shape[0], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - (9 if fmt == "mxfp8" else 3), -127).clamp(-127, 127)
    scale = torch.tensor([2.0 ** k for k in range(-127, 128)], device=DEV, dtype=torch.float64)[e.long() + 127]
    return (_nearest(b / scale, e4m3 if fmt == "mxfp8" else [0, .5, 1, 1.5, 2, 3, 4, 6]) * scale).view(y.shape)


def _exact_rotated(s):
    c = s["case"]
    n, h, d, first, rot = (c[k] for k in ("n", "heads", "d", "first", "rot"))
    p = torch.stack([s["pos"][:, a].double() for a in _axes(c)], 1)
    turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), p * s["freq"])[:, None]
    if c.get("grad"):
        turn = turn.conj()
    y = s["x"].double().reshape(n, h, d).clone()
    part = y[..., first:first + rot]
    halves = c["layout"] == "half"
    pairs = part.reshape(n, h, 2, rot // 2).transpose(2, 3) if halves else part.reshape(n, h, rot // 2, 2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[..., first:first + rot] = (z.transpose(2, 3) if halves else z).reshape(n, h, rot)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "axes":
        return _exact_rotated(s)
    if op == "axes_write":
        return _exact_stored(_exact_rotated(s).flatten(1), case["fmt"]).view(s["x"].shape)
    x = s["x"].double().view(-1, d)
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    dev = torch.sqrt(var + EPS)
    out = {}
    w, b = s["weight"].double(), s["bias"].double()
    if op != "grad":
        out["y"] = ((x - mean) / dev * w + b).view(s["x"].shape)
        if op == "norm":
            return out["y"]
        x = _exact_stored(x, case["fmt"])
    c = x - mean
    dy = s["dy"].double().view(-1, d)
    g = dy * w
    out["dx"] = ((g - g.mean(1, keepdim=True)) / dev - c * ((g * c).mean(1, keepdim=True) / dev ** 3)).view(s["x"].shape)
    out["dweight"] = (dy * (c / dev)).sum(0)
    out["dbias"] = dy.sum(0)
    return out
