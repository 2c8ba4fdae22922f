"""Measured cases of the operators around the exact top-k selection: rotary positions, the quantised cache
(written and read back), the attention's mass at the selected entries, and the indexer's loss with its gradient.

Shapes follow the repository's workloads (64 indexer heads of 128, k = 2,048, 8,192 queries of a 1M context;
the 131,072-key problem; the 64-wide heads of the small one) or are generic.  With ``own`` false ``run``
computes an operator in elementary torch operations; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32                      # elements that share one E8M0 scale
EMAX = {"mxfp8": 8, "mxfp4": 2}  # exponent of the element format's largest value


def listed():
    return [
        # one decoded token's indexer queries near the end of a 1M context: latency
        dict(name="rotary_token", op="rotary", n=1, heads=64, d=128, rot=64, first=0, layout="half",
             scaling="yarn", pos=1048575, grad=False),
        # a context-parallel shard's queries: 8,192 tokens at the end of a 1M context
        dict(name="rotary_prompt", op="rotary", n=8192, heads=64, d=128, rot=64, first=64,
             layout="interleaved", scaling="yarn", pos=1040384, grad=False),
        # the gradient of the queries (fp32, from the indexer backward) on its way to a bf16 projection;
        # odd token count, narrow heads
        dict(name="rotary_gradient", op="rotary", n=5003, heads=24, d=64, rot=64, first=0, layout="half",
             scaling="linear", pos=131, grad=True),
        # one decoded token of each of 64 sequences rotated and written into an FP8 key cache, rows by slot
        dict(name="write_tokens_fp8", op="write", fmt="fp8", n=64, heads=1, d=128, rot=64, L=1048576,
             by_slot=True, pos=900000),
        # the indexer keys of a 131,072-token prompt rotated and written into an MXFP8 cache
        dict(name="write_prompt_mxfp8", op="write", fmt="mxfp8", n=131072, heads=1, d=128, rot=64, L=131072,
             by_slot=False, pos=0),
        # the queries of a shard rotated and quantised to MXFP4, 64 heads a token
        dict(name="write_queries_mxfp4", op="write", fmt="mxfp4", n=8192, heads=64, d=128, rot=128, L=8192,
             by_slot=False, pos=1040384),
        # a whole FP8 key cache of a 1M context decoded
        dict(name="read_context_fp8", op="read", fmt="fp8", rows=1048576, heads=1, d=128, L=1048576,
             by_slot=False),
        # the 2,048 selected keys of each of 9 decoded tokens read back from an MXFP8 cache; the last
        # rows of each list are padding
        dict(name="read_selected_mxfp8", op="read", fmt="mxfp8", rows=9 * 2048, heads=1, d=128, L=131072,
             by_slot=True),
        # the training target of a 2,048-query chunk of the 131,072-key problem: 64 heads on one key head
        dict(name="mass_shared_key", op="mass", n=2048, k=2048, A=64, G=1, d=128, L=131072, pos=129024,
             with_lse=False),
        # the first tokens of a short sequence: grouped key heads, rows shorter than k, the attention's
        # own normaliser at hand
        dict(name="mass_grouped", op="mass", n=301, k=500, A=32, G=4, d=64, L=4096, pos=0, with_lse=True),
        # the loss of a shard's 8,192 queries
        dict(name="loss_shard", op="loss", n=8192, k=2048, short=0.02),
        # the loss of a small batch with ragged rows
        dict(name="loss_ragged", op="loss", n=77, k=333, short=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "mass", "loss"])
    if op == "rotary":
        heads, d = rng.choice([1, 4, 8, 24, 40, 64]), rng.choice([64, 128])
        rot = rng.choice([d // 4, d // 2, d])
        return dict(op=op, n=_log(rng, 1, max(2, (1 << 26) // (heads * d))), heads=heads, d=d, rot=rot,
                    first=rng.choice([0, d - rot]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), pos=_log(rng, 1, 1 << 20),
                    grad=rng.random() < 0.4)
    if op == "write":
        heads = rng.choice([1, 1, 4, 32, 64])
        n = _log(rng, 1, min(1 << 17, (1 << 26) // (heads * 128)))
        return dict(op=op, fmt=rng.choice(["bf16", "fp8", "mxfp8", "mxfp4"]), n=n, heads=heads, d=128,
                    rot=rng.choice([0, 32, 64, 128]), L=n + _log(rng, 1, 4096), by_slot=rng.random() < 0.5,
                    pos=_log(rng, 1, 1 << 20))
    if op == "read":
        L = _log(rng, 64, 1 << 19)
        return dict(op=op, fmt=rng.choice(["bf16", "fp8", "mxfp8", "mxfp4"]), rows=_log(rng, 1, L), heads=1,
                    d=128, L=L, by_slot=rng.random() < 0.6)
    if op == "mass":
        A, G = rng.choice([(8, 1), (16, 2), (32, 4), (40, 8), (64, 1), (64, 8)])
        k = _log(rng, 2, 2048)
        d = rng.choice([64, 128, 192])
        L = _log(rng, 4096, 131072)
        n = _log(rng, 1, max(2, min(2048, (1 << 27) // (k * A * G))))
        pos = rng.choice([0, L - n]) if n > 8 else L - n
        return dict(op=op, n=n, k=k, A=A, G=G, d=d, L=L, pos=pos, with_lse=rng.random() < 0.5)
    return dict(op=op, n=_log(rng, 1, 8192), k=_log(rng, 2, 2048), short=rng.random())


def _frequencies(case):
    """Arguments of the rotary plan of a case."""
    s = case.get("scaling", "none")
    a = dict(base=10000.0 if case["d"] == 64 else 1000000.0, scaling=s)
    if s != "none":
        a.update(factor=32.0 if s == "yarn" else 4.0, original=32768)
    return a


def _slots(L, rows, by_slot, g, device, pad=0):
    """Cache rows of the tokens: distinct and in no order, some of them padding (-1)."""
    if not by_slot:
        return None
    s = torch.randperm(L, generator=g, device=device)[:rows].to(torch.int32)
    if pad:
        s[-pad:] = -1
    return s


def _width(fmt, d):
    return d // 2 if fmt == "mxfp4" else d


def _cache(fmt, L, heads, d):
    """An empty cache: codes and scales."""
    shape = (L, d) if heads == 1 else (L, heads, d)
    codes = torch.zeros(shape[:-1] + (_width(fmt, d),), device=DEV,
                        dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8)
    if fmt == "bf16":
        return codes, None
    if fmt == "fp8":
        return codes, torch.ones(L, device=DEV)
    return codes, torch.zeros(shape[:-1] + (d // BLOCK,), device=DEV, dtype=torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    op = case["op"]
    s = dict(case=dict(case))
    if op == "rotary":
        n, h, d = case["n"], case["heads"], case["d"]
        s["x"] = normal(n, h, d, dtype=torch.float32 if case["grad"] else torch.bfloat16)
        # positions near the end of the context in an order of their own (shards take theirs zigzag)
        s["pos"] = (case["pos"] + torch.randperm(n, generator=g, device=DEV)).to(torch.int32)
        s["freq"], s["attn"] = _plan_values(case["rot"], **_frequencies(case))
    elif op == "write":
        n, h, d, fmt = case["n"], case["heads"], case["d"], case["fmt"]
        # rows of different sizes, as tokens have
        size = torch.exp(0.5 * normal(n, 1, 1))
        s["x"] = (normal(n, h, d) * size).to(torch.bfloat16)
        if h == 1:
            s["x"] = s["x"].view(n, d)
        s["pos"] = (case["pos"] + torch.arange(n, device=DEV)).to(torch.int32)
        s["slots"] = _slots(case["L"], n, case["by_slot"], g, DEV)
        s["codes"], s["scale"] = _cache(fmt, case["L"], h, d)
        if case["rot"]:
            s["freq"], s["attn"] = _plan_values(case["rot"], **_frequencies(case))
    elif op == "read":
        L, d, fmt, rows = case["L"], case["d"], case["fmt"], case["rows"]
        if fmt == "bf16":
            s["codes"], s["scale"] = normal(L, d, dtype=torch.bfloat16), None
        else:
            codes = torch.randint(0, 256, (L, _width(fmt, d)), generator=g, device=DEV, dtype=torch.uint8)
            if fmt != "mxfp4":  # a cache holds no E4M3 NaN
                codes = torch.where((codes & 127) == 127, codes - 1, codes)
            s["codes"] = codes
            if fmt == "fp8":
                s["scale"] = torch.exp(normal(L)) / 448
            else:
                s["scale"] = torch.randint(110, 124, (L, d // BLOCK), generator=g, device=DEV, dtype=torch.uint8)
        s["slots"] = _slots(L, rows, case["by_slot"], g, DEV, pad=min(5, rows - 1))
    elif op == "mass":
        n, k, A, G, d, L = (case[x] for x in ("n", "k", "A", "G", "d", "L"))
        s["q"] = (2 * normal(n, A, d)).to(torch.bfloat16)
        s["keys"] = normal(L, G, d, dtype=torch.bfloat16)
        s["idx"] = _selected(n, k, case["pos"], g)
        s["lse"] = None
        if case["with_lse"]:
            s["lse"] = _lse(s)
    else:
        n, k = case["n"], case["k"]
        live = torch.full((n,), k, device=DEV)
        cut = torch.rand(n, generator=g, device=DEV) < case["short"]
        live = torch.where(cut, (torch.rand(n, generator=g, device=DEV) * (k + 1)).long(), live)
        dead = torch.arange(k, device=DEV) >= live[:, None]
        score = 2 * normal(n, k)
        s["score"] = torch.sort(score, dim=1, descending=True)[0].masked_fill(dead, -math.inf)
        mass = torch.exp(2 * normal(n, k)).masked_fill(dead, 0.0)
        s["mass"] = mass / mass.sum(1, keepdim=True).clamp_min(1e-30)
        s["weight"] = torch.rand(n, generator=g, device=DEV) / n
    if own:
        _plan(s)
    return s


def _plan(s):
    """The plan that a user's program keeps beside its inputs."""
    c = s["case"]
    if c["op"] in ("rotary", "write") and c["rot"]:
        import exact_top_token_amd as hk
        s["plan"] = hk.Rotary(c["rot"], first=c.get("first", 0), layout=c.get("layout", "half"), device=DEV,
                              **_frequencies(c))


def _plan_values(rot, base, scaling, factor=1.0, original=0):
    """Frequencies (64 bits, radians a position) and the factor on the rotated part."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    if scaling == "ntk":  # the base stretched so that the slowest frequency is divided by the factor
        base = base * factor ** (rot / max(rot - 2, 1))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":  # frequencies that turn often keep their speed, slow ones are divided, a ramp between
        def turns(r):  # the index whose frequency makes r turns in the original context
            return rot * math.log(original / (r * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1
    return f, 1.0


def _selected(n, k, pos, g):
    """Indices of the selection: query i sits at pos + i and sees the keys up to itself; distinct keys spread
    over its context in the order of their scores, -1 behind the end of a short context."""
    ctx = torch.arange(n, device=DEV)[:, None] + pos + (0 if pos else -1)  # pos 0: the first query sees nothing
    j = torch.arange(k, device=DEV)[None]
    step = (j + torch.rand((n, k), generator=g, device=DEV, dtype=torch.float64)) * ctx / k
    at = torch.where(ctx > k, step.long().clamp_max((ctx - 1).clamp_min(0)), j.expand(n, k))
    mix = torch.rand((n, k), generator=g, device=DEV).masked_fill(j >= ctx, 2.0).argsort(1)
    return torch.where(j < ctx, at.gather(1, mix), -1).to(torch.int32)


def _logits(s):
    """Logits [n][G][A/G][k] of the selected keys in 32 bits, -inf at padding."""
    q, keys, idx = s["q"].float(), s["keys"], s["idx"].long()
    n, A, d = q.shape
    G = keys.shape[1]
    rows = keys[idx.clamp_min(0)].float()                       # [n][k][G][d]
    rows = rows.permute(0, 2, 3, 1).contiguous()                # [n][G][d][k]
    x = torch.matmul(q.view(n, G, A // G, d), rows) * d ** -0.5
    return x.masked_fill((idx < 0)[:, None, None], -math.inf)


def _lse(s):
    x = _logits(s)
    return torch.logsumexp(x, -1).reshape(x.shape[0], -1)


# ------------------------------------------------------------- plain forms

def _rotate(x, pos, freq, attn, rot, first, layout, back):
    """x [n][H][d] in 32 bits; angles in 64."""
    angle = pos.double()[:, None] * freq
    cos, sin = (torch.cos(angle) * attn).float()[:, None], (torch.sin(angle) * attn).float()[:, None]
    if back:
        sin = -sin
    y = x.float().clone()
    part = x[..., first:first + rot].float()
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        y[..., first:first + rot] = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        y[..., first:first + rot] = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return y


def _to_e4m3(v):
    """E4M3 codes of 64-bit values: to nearest, ties to even, at most 448."""
    a = v.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    r = torch.copysign(torch.round(a / step) * step, v)
    return r.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _to_e2m1(v):
    a = v.abs().clamp_max(6.0)
    c = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    return c.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def _encode(y, fmt):
    """y [n][H][d] in 32 bits: codes and scales of a storage format."""
    n = y.shape[0]
    if fmt == "bf16":
        return y.to(torch.bfloat16), None
    if fmt == "fp8":
        amax = y.reshape(n, -1).abs().amax(1)
        scale = torch.where(amax > 0, (amax / 448.0).clamp_min(2.0 ** -126), torch.ones_like(amax))
        return _to_e4m3(y.double() / scale.double()[:, None, None]), scale
    b = y.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 1 - EMAX[fmt]
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    v = b.double() * torch.exp2(-e.double())[..., None]
    if fmt == "mxfp8":
        codes = _to_e4m3(v).flatten(-2)
    else:
        c = _to_e2m1(v).flatten(-2)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    return codes, (e + 127).to(torch.uint8)


def _decode(codes, scale, fmt):
    """Values of codes [rows][..][d] in 32 bits."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
        return v * scale.view((-1,) + (1,) * (v.dim() - 1))
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        m = (c & 7).float()
        v = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
        v = torch.where(c > 7, -v, v)
    f = torch.exp2(scale.double() - 127).float()
    return (v.unflatten(-1, (-1, BLOCK)) * f[..., None]).flatten(-2)


def _plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        y = _rotate(s["x"], s["pos"], s["freq"], s["attn"], c["rot"], c["first"], c["layout"], c["grad"])
        return y.to(torch.bfloat16)
    if c["op"] == "write":
        x = s["x"].view(c["n"], c["heads"], c["d"]).float()
        if c["rot"]:
            x = _rotate(x, s["pos"], s["freq"], s["attn"], c["rot"], 0, "half", False)
        codes, scale = _encode(x, c["fmt"])
        rows = slice(0, c["n"]) if s["slots"] is None else s["slots"].long()
        s["codes"][rows] = codes.view(s["codes"].shape[1:] if c["n"] == 0 else (c["n"],) + s["codes"].shape[1:])
        if scale is not None:
            s["scale"][rows] = scale.view((c["n"],) + s["scale"].shape[1:])
        back = _decode(s["codes"][rows], None if scale is None else s["scale"][rows], c["fmt"])
        return back.to(torch.bfloat16)
    if c["op"] == "read":
        if s["slots"] is None:
            rows = slice(0, c["rows"])
            return _decode(s["codes"][rows], None if s["scale"] is None else s["scale"][rows], c["fmt"]).to(torch.bfloat16)
        at = s["slots"].long()
        rows = at.clamp_min(0)
        v = _decode(s["codes"][rows], None if s["scale"] is None else s["scale"][rows], c["fmt"])
        return v.masked_fill((at < 0)[:, None], 0.0).to(torch.bfloat16)
    if c["op"] == "mass":
        x = _logits(s)
        n, G, R, k = x.shape
        lse = torch.logsumexp(x, -1) if s["lse"] is None else s["lse"].view(n, G, R)
        p = torch.exp(x - lse[..., None]).masked_fill((s["idx"] < 0)[:, None, None], 0.0)
        return p.sum((1, 2)) / (G * R)
    score, mass = s["score"], s["mass"]
    live = score != -math.inf
    t = torch.where(live, mass, 0.0)
    total = t.sum(1, keepdim=True)
    t = torch.where(total > 0, t / total, 0.0)
    logp = score - torch.logsumexp(score, 1, keepdim=True)
    term = torch.where(t > 0, t * (torch.log(t.clamp_min(1e-38)) - logp), 0.0)
    w = torch.where(total[:, 0] > 0, s["weight"], 0.0)
    grad = torch.where(live & (total > 0), torch.exp(logp) - t, 0.0) * w[:, None]
    return {"loss": term.sum(1) * w, "d_score": grad}


def run(state):
    if not own:
        return _plain(state)
    import exact_top_token_amd as hk
    s, c = state, state["case"]
    if c["op"] == "rotary":
        return hk.rotary(s["x"], s["plan"], q_pos=s["pos"], backward=c["grad"], out_dtype=torch.bfloat16)
    if c["op"] == "write":
        hk.cache_write(s["x"], s["codes"], s["scale"], fmt=c["fmt"], slots=s["slots"], rotary=s.get("plan"),
                       q_pos=s["pos"])
        return hk.cache_read(s["codes"], s["scale"], fmt=c["fmt"], slots=s["slots"], count=c["n"])
    if c["op"] == "read":
        return hk.cache_read(s["codes"], s["scale"], fmt=c["fmt"], slots=s["slots"], count=c["rows"])
    if c["op"] == "mass":
        return hk.attention_mass(s["q"], s["keys"], s["idx"], lse=s["lse"])
    loss, grad = hk.index_loss(s["score"], s["mass"], weight=s["weight"])
    return {"loss": loss, "d_score": grad}


def work(case):
    op = case["op"]
    bits = {"bf16": 16, "fp8": 8, "mxfp8": 8.25, "mxfp4": 4.25}
    if op == "rotary":
        e = case["n"] * case["heads"] * case["d"]
        return {"bytes": e * ((4 if case["grad"] else 2) + 2) + 4 * case["n"],
                "flops": 3 * case["n"] * case["heads"] * case["rot"]}
    if op == "write":  # rows in, codes out, codes in again, values out
        e = case["n"] * case["heads"] * case["d"]
        return {"bytes": e * (4 + 2 * bits[case["fmt"]] / 8) + 8 * case["n"],
                "flops": e * 4 + 3 * case["n"] * case["heads"] * case["rot"]}
    if op == "read":
        e = case["rows"] * case["heads"] * case["d"]
        return {"bytes": e * (2 + bits[case["fmt"]] / 8) + 8 * case["rows"], "flops": e}
    if op == "mass":
        n, k, A, G, d, L = (case[x] for x in ("n", "k", "A", "G", "d", "L"))
        rows = min(L, n * k)
        return {"bytes": 2 * n * A * d + 2 * rows * G * d + 8 * n * k, "flops": 2 * n * k * A * d}
    return {"bytes": 12 * case["n"] * case["k"] + 8 * case["n"], "flops": 12 * case["n"] * case["k"]}


# ------------------------------------------------- the definitions in 64 bits

def _exact_rotate(x, pos, freq, attn, rot, first, layout, back):
    turn = torch.polar(torch.full((1,), float(attn), device=DEV, dtype=torch.float64),
                       pos.double()[:, None] * freq)[:, None]
    if back:
        turn = turn.conj()
    y = x.double().clone()
    n, h, _ = y.shape
    p = y[..., first:first + rot]
    pairs = p.reshape(n, h, rot // 2, 2) if layout == "interleaved" else p.reshape(n, h, 2, rot // 2).transpose(2, 3)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[..., first:first + rot] = (z if layout == "interleaved" else z.transpose(2, 3)).reshape(n, h, rot)
    return y


def _nearest(v, table):
    """The nearest value of a table of magnitudes (ties to the even place), with v's sign."""
    t = torch.tensor(table, device=DEV, dtype=torch.float64)
    mid = (t[1:] + t[:-1]) / 2
    a = v.abs()
    lo = torch.bucketize(a, mid)
    hi = torch.bucketize(a, mid, right=True)
    return torch.where(lo == hi, t[lo], t[(lo + lo % 2).clamp_max(len(table) - 1)]) * torch.sign(v)


def _exact_quantised(y, fmt):
    """The values that a cache row stands for, from y in 64 bits."""
    e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1]
    if fmt == "bf16":
        return y
    if fmt == "fp8":
        top = y.abs().amax((1, 2), keepdim=True)
        scale = torch.where(top > 0, (top / 448).float().double().clamp_min(2.0 ** -126), 1.0)
        return _nearest(y / scale, e4m3) * scale
    b = y.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.floor(torch.log2(top.clamp_min(1e-300))) - EMAX[fmt]).clamp(-127, 127)
    scale = torch.pow(2.0, e)
    table = e4m3 if fmt == "mxfp8" else [0, .5, 1, 1.5, 2, 3, 4, 6]
    return (_nearest(b / scale, table) * scale).flatten(-2)


def _exact_codes(codes, fmt):
    """What each code stands for, from the formats' bit fields."""
    c = codes.to(torch.int64)
    if fmt == "mxfp4":
        c = torch.stack([c % 16, c // 16], -1).flatten(-2)
        t = [0, .5, 1, 1.5, 2, 3, 4, 6]
        t = t + [-x for x in t]
    else:
        t = [(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)]
        t = t + [-x for x in t]
    return torch.tensor(t, device=DEV, dtype=torch.float64)[c]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _exact_rotate(s["x"], s["pos"], s["freq"], s["attn"], case["rot"], case["first"], case["layout"], case["grad"])
    if op == "write":
        y = s["x"].double().view(case["n"], case["heads"], case["d"])
        if case["rot"]:
            y = _exact_rotate(y, s["pos"], s["freq"], s["attn"], case["rot"], 0, "half", False)
        v = _exact_quantised(y, case["fmt"])
        return v[:, 0] if case["heads"] == 1 else v
    if op == "read":
        at = torch.arange(case["rows"], device=DEV) if s["slots"] is None else s["slots"].long()
        c = s["codes"][at.clamp_min(0)]
        if case["fmt"] == "bf16":
            v = c.double()
        else:
            v = _exact_codes(c, case["fmt"])
            f = s["scale"][at.clamp_min(0)].double()
            v = v * (f[:, None] if case["fmt"] == "fp8" else torch.pow(2.0, f - 127).repeat_interleave(BLOCK, 1))
        return v * (at >= 0)[:, None]
    if op == "mass":
        q, keys, idx = s["q"].double(), s["keys"].double(), s["idx"].long()
        n, A, d = q.shape
        G = keys.shape[1]
        out = torch.zeros(idx.shape, device=DEV, dtype=torch.float64)
        for lo in range(0, n, 256):
            at = slice(lo, min(n, lo + 256))
            dead = (idx[at] < 0)[:, None]
            for h in range(G):
                rows = keys[idx[at].clamp_min(0), h]                                   # [q][k][d]
                x = torch.bmm(rows, q[at, h * (A // G):(h + 1) * (A // G)].transpose(1, 2).contiguous()) / math.sqrt(d)
                x = x.transpose(1, 2).masked_fill(dead, -math.inf)
                if s["lse"] is None:
                    top = x.amax(-1, keepdim=True).clamp_min(-1e300)
                    e = torch.exp(x - top)
                    p = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
                else:
                    p = torch.exp(x - s["lse"][at, h * (A // G):(h + 1) * (A // G), None].double())
                    p = p.masked_fill(dead, 0.0)
                out[at] += p.sum(1)
        return out / A
    score, mass = s["score"].double(), s["mass"].double()
    live = torch.isfinite(score)
    total = (mass * live).sum(1)
    t = torch.where(live & (total > 0)[:, None], mass / total[:, None], 0.0)
    e = torch.where(live, torch.exp(score - score.amax(1, keepdim=True).clamp_min(-1e300)), 0.0)
    p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    w = s["weight"].double() * (total > 0)
    loss = (torch.xlogy(t, t) - torch.where(t > 0, t * torch.log(p), 0.0)).sum(1)
    return {"loss": loss * w, "d_score": torch.where(live, p - t, 0.0) * w[:, None]}
