"""Layer norm, its checkpoints and positions of several axes as they are used together: a training step of the indexer
on video tokens, a decoded token, graphs that share a workspace, two host threads, other streams; and at their limits: more
rows than one launch holds, offsets past 32 bits."""
import threading

import numpy as np
import pytest
import torch

import datagen
import oracle
from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _room(gib):
    torch.cuda.empty_cache()  # what earlier tests left with torch
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def _rand(shape, seed, dtype=BF16, scale=1.0, offset=0.0):
    return (offset + scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def _video(n, text, high, wide):
    """Positions of n tokens: text, then frames of high x wide."""
    i = torch.arange(n) - text
    t = torch.stack([i // (high * wide), i // wide % high, i % wide], 1) + text
    return torch.where((i < 0)[:, None], torch.arange(n)[:, None].expand(n, 3), t).int().cuda()


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("save", ["x", "fp8", "mxfp8"])
def test_training_step(hk, save):
    """norm -> rotary by axes -> select -> replay -> mass -> loss -> backward -> transposed rotation -> norm's backward."""
    L, n, H, d, k = 600, 64, 8, 128, 96
    say(f"norm chain: training, {save}")
    plan = hk.Rotary(64, first=64, layout="interleaved", sections=(12, 10, 10), cycle=True)
    xk, xq = _rand((L, d), 1, offset=0.5), _rand((n, H, d), 2, scale=3.0)
    wk, bk, wq, bq = (_rand(d, 3 + i, FP32, 0.2 * d ** -0.5, o * d ** -0.5) for i, o in enumerate((1.0, 0.0, 1.0, 0.0)))
    w = torch.rand((n, H), generator=torch.Generator().manual_seed(7)).cuda()
    pos = _video(L, 40, 9, 13)
    nk, kept_k = hk.layer_norm(xk, wk, bk, eps=1e-6, save=save)
    nq, kept_q = hk.layer_norm(xq, wq, bq, eps=1e-6, save=save)
    key, q = hk.rotary(nk, plan, q_pos=pos), hk.rotary(nq, plan, q_pos=pos[L - n:])
    idx, score = hk.select(q, key, w, k)
    assert torch.equal(hk.replay(q, key, w, idx), score)
    mass = hk.attention_mass(_rand((n, 8, 64), 11, scale=2.0), _rand((L, 2, 64), 12), idx)
    loss, d_score = hk.index_loss(score, mass)
    g = hk.backward(q, key, w, idx, d_score)
    dk = hk.rotary(g["dk"], plan, q_pos=pos, backward=True)
    dq = hk.rotary(g["dq"], plan, q_pos=pos[L - n:], backward=True)
    gk = hk.layer_norm_backward(dk, kept_k, wk, dx_dtype=BF16)
    gq = hk.layer_norm_backward(dq, kept_q, wq, dx_dtype=BF16)
    # every new link against its definition on the link's own inputs, within 2^-16 of the largest value (some hundred
    # roundings of 2^-24) and a bf16 result's half step
    axis, f = plan.axis.cpu().numpy(), f64(plan.freq)

    def near(got, want, what):
        tol = 2.0 ** -16 * np.abs(want).max() + (2.0 ** -8 * np.abs(want) if got.dtype == BF16 else 0)
        assert (np.abs(f64(got) - want) <= tol).all(), what
    near(nk, op.layer_norm(f64(xk), f64(wk), f64(bk), 1e-6)[0], "keys normalised")
    near(nq, op.layer_norm(f64(xq), f64(wq), f64(bq), 1e-6)[0], "queries normalised")
    kw = dict(first=64, layout="interleaved", axis=axis)
    p = pos.cpu().numpy().astype(np.int64)
    near(key, op.rotary(f64(nk)[:, None], p, f, **kw)[:, 0], "keys rotated")
    near(q, op.rotary(f64(nq), p[L - n:], f, **kw), "queries rotated")
    near(dk, op.rotary(f64(g["dk"])[:, None], p, f, backward=True, **kw)[:, 0], "keys' gradient")
    near(dq, op.rotary(f64(g["dq"]), p[L - n:], f, backward=True, **kw), "queries' gradient")
    for x, kept, dy, weight, got in ((xk, kept_k, dk, wk, gk), (xq, kept_q, dq, wq, gq)):
        x64 = f64(x) if save == "x" else f64(hk.cache_read(kept.rows.reshape(-1, d), kept.scale.reshape(-1, *kept.scale.shape[x.dim() - 1:]),
                                                            fmt=save, dtype=FP32)).reshape(x.shape)
        st = f64(kept.stats)
        dx, dw, db = op.layer_norm_backward(f64(dy), x64, st[..., 0], st[..., 1], f64(weight))
        near(got["dx"], dx, "dx")
        near(got["dweight"], dw, "dweight")
        near(got["dbias"], db, "dbias")
    assert float(loss.sum()) > 0 and float(gk["dweight"].abs().max()) > 0


def test_the_step_s_slope(hk):
    """The gradient of the normalised, rotated and scored keys against differences of the fp64 chain: everything in fp32 but the
    scoring's bf16 operands, so the norm's and the rotation's part is checked with the scores' gradient taken as linear."""
    n, H, d = 40, 3, 64
    plan = hk.Rotary(32, first=16, sections=(6, 5, 5))
    x, w, b = _rand((n, H, d), 20, FP32), _rand(d, 21, FP32, 0.3, 1.0), _rand(d, 22, FP32)
    up = _rand((n, H, d), 23, FP32)
    pos = _video(n, 3, 4, 5)
    y, kept = hk.layer_norm(x, w, b, save="x")
    hk.rotary(y, plan, q_pos=pos, out=y)
    g = hk.layer_norm_backward(hk.rotary(up, plan, q_pos=pos, backward=True), kept, w)
    p, f, axis = pos.cpu().numpy().astype(np.int64), f64(plan.freq), plan.axis.cpu().numpy()
    rng = np.random.default_rng(24)
    for _ in range(5):
        v = [rng.standard_normal(s) for s in ((n, H, d), d, d)]

        def at(t):
            z = op.layer_norm(f64(x) + t * v[0], f64(w) + t * v[1], f64(b) + t * v[2], 1e-5)[0]
            return (f64(up) * op.rotary(z, p, f, first=16, axis=axis)).sum()
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        parts = [f64(g["dx"]) * v[0], f64(g["dweight"]) * v[1], f64(g["dbias"]) * v[2]]
        got, size = sum(t.sum() for t in parts), sum(np.abs(t).sum() for t in parts)
        assert abs(got - slope) <= 2.0 ** -18 * size + 1e-6 * abs(slope)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8", "mxfp4"])
def test_decode_step(hk, fmt):
    """A prompt normalised and written into a cache, then tokens one at a time; equal to all rows at once."""
    L, H, d, k, steps = 500, 8, 128, 64, 3
    say(f"norm chain: decode {fmt}")
    plan = hk.Rotary(128, sections=(16, 24, 24))
    x, w, b = _rand((L + steps, d), 30), _rand(d, 31, scale=0.1, offset=1.0), _rand(d, 32, scale=0.1)
    pos = _video(L + steps, 100, 6, 11)
    weights = torch.rand((1, H), generator=torch.Generator().manual_seed(33)).cuda()
    whole, whole_s = hk.quantize(hk.layer_norm(x, w, b), fmt, rotary=plan, q_pos=pos)
    codes, scale = torch.zeros_like(whole), None if whole_s is None else torch.zeros_like(whole_s)
    hk.cache_write(hk.layer_norm(x[:L], w, b), codes, scale, fmt=fmt, rotary=plan, q_pos=pos[:L])
    for t in range(steps):
        at = torch.tensor([L + t], dtype=torch.int32, device="cuda")
        p = pos[L + t:L + t + 1]
        hk.cache_write(hk.layer_norm(x[L + t:L + t + 1], w, b), codes, scale, fmt=fmt, slots=at, rotary=plan, q_pos=p)
        q, qs = hk.quantize(hk.layer_norm(_rand((1, H, d), 40 + t), w, b), fmt, rotary=plan, q_pos=p)
        kw = dict(q_pos=at, fmt=fmt, q_scale=qs)
        a, c = hk.select(q, codes, weights, k, k_scale=scale, **kw), hk.select(q, whole, weights, k, k_scale=whole_s, **kw)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1]) and int(a[0].max()) <= L + t
    assert torch.equal(codes, whole) and (scale is None or torch.equal(scale, whole_s))


class _Step:
    """A norm forward with a checkpoint, the rotation both ways and the norm's backward, in given or own memory."""

    def __init__(self, hk, seed, n, heads, d, save):
        self.hk, self.save = hk, save
        self.x, self.dy = _rand((n, heads, d), seed), _rand((n, heads, d), seed + 1, FP32)
        self.w, self.b = _rand(d, seed + 2, FP32, 0.2, 1.0), _rand(d, seed + 3, FP32)
        self.pos = _video(n, 5, 7, 9)
        self.plan = hk.Rotary(32, sections=(8, 8) if seed % 2 else (6, 5, 5))
        self.pos = self.pos[:, 3 - self.plan.axes:].contiguous()

    def run(self, workspace=None):
        hk = self.hk
        y, kept = hk.layer_norm(self.x, self.w, self.b, save=self.save)
        y = hk.rotary(y, self.plan, q_pos=self.pos)
        up = hk.rotary(self.dy, self.plan, q_pos=self.pos, backward=True)
        g = hk.layer_norm_backward(up, kept, self.w, dx_dtype=BF16, workspace=workspace)
        return y, kept.rows, kept.stats, up, g["dx"], g["dweight"], g["dbias"]


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs_that_share_a_workspace(hk):
    work = [_Step(hk, 50, 301, 4, 96, "fp8"), _Step(hk, 61, 1000, 1, 1100, "x"), _Step(hk, 72, 64, 2, 128, "mxfp8")]
    ws = torch.empty(max(hk.layer_norm_backward_workspace_bytes(s.dy) for s in work), dtype=torch.uint8, device="cuda")
    for s in work:
        s.run(ws)
    torch.cuda.synchronize()
    graphs, held = [], []
    for s in work:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            held.append((s.run(ws), s.run()))  # a shared workspace, and one of the graph's own memory
        graphs.append(gr)
    for rep in range(3):
        for i, s in enumerate(work):
            s.x.copy_(_rand(s.x.shape, 100 + 10 * rep + i, offset=float(rep)))
            s.dy.copy_(_rand(s.dy.shape, 200 + 10 * rep + i, FP32))
        want = [s.run() for s in work]
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for a, (b, c) in zip(want, held):
            assert _equal(a, b) and _equal(a, c), rep


def test_two_threads_and_other_streams(hk):
    work = [_Step(hk, 80, 700, 3, 128, "fp8"), _Step(hk, 91, 90, 1, 4096, "mxfp8")]
    alone = [s.run() for s in work]
    torch.cuda.synchronize()
    wrong, gate = [], threading.Barrier(2)

    def go(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gate.wait(60)
                for rep in range(6):
                    got = work[i].run()
                    stream.synchronize()
                    if not _equal(got, alone[i]):
                        wrong.append((i, rep))
        except Exception as e:  # a thread's failure is the test's
            wrong.append((i, repr(e)))
    threads = [threading.Thread(target=go, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_traced(hk):
    s = _Step(hk, 95, 50, 1, 64, "fp8")
    hk.trace_enable(True)
    try:
        s.run()
        t = hk.trace_read()
    finally:
        hk.trace_enable(False)
    assert t["layer_norm"][0] == 1 and t["layer_norm_backward"][0] == 1 and t["rotary"][0] == 2


# ------------------------------------------------------------------- limits

def test_the_most_rows(hk):
    """2^31 - 1 rows of one element: each is its own mean, so y is the bias and dx is 0; dbias of a sum that stays small."""
    _room(40)
    n = (1 << 31) - 1
    say("norm: the most rows")
    x = torch.empty((n, 1), dtype=BF16, device="cuda").fill_(1.5)
    x[::7] = -3.0
    b = torch.full((1,), 0.75, device="cuda")
    y = hk.layer_norm(x, None, b)
    assert bool((y == 0.75).all())
    stats = torch.zeros((n, 2), device="cuda")
    stats[:, 1] = 1.0
    del y
    dy = torch.zeros((n, 1), dtype=BF16, device="cuda")
    dy[-3:], dy[0] = 1.0, 4.0
    r = hk.layer_norm_backward(dy, hk.NormSaved(x, None, stats, None))
    # h is x itself with these statistics: dweight = sum dy x, and g - mean(g) - h mean(g h) = -x^2 dy
    tail = x[-3:].float().sum().item()
    assert r["dbias"].item() == 7.0 and r["dweight"].item() == tail + 4.0 * x[0].item()
    assert r["dx"][0].item() == -4.0 * 9.0 and not r["dx"][1:-3].any() and bool((r["dx"][-3:] == -(x[-3:] ** 2)).all())


@pytest.mark.parametrize("d", [128, 100, 2048])
def test_offsets_past_32_bits(hk, d):
    """Rows whose places in their buffers pass 2^31 elements, by token and by head strides."""
    _room(60)
    say(f"norm: far rows, d={d}")
    step = (1 << 31) + 64
    base = torch.empty(3 * step + d, dtype=BF16, device="cuda")
    w, b = _rand(d, 1, FP32), _rand(d, 2, FP32)
    near, dy = _rand((2, 2, d), 3), _rand((2, 2, d), 4, BF16)
    want, saved = hk.layer_norm(near, w, b, save="x")
    grads = hk.layer_norm_backward(dy, saved, w)
    for strides in ((step, 2 * step, 1), (2 * step, step, 1)):
        far = base.as_strided((2, 2, d), strides)
        far.copy_(near)
        y, s = hk.layer_norm(far, w, b, save="x")
        assert torch.equal(y, want) and torch.equal(s.stats, saved.stats)
        r = hk.layer_norm_backward(dy, s, w)
        assert all(torch.equal(r[name], grads[name]) for name in grads)
        r = hk.layer_norm_backward(far, saved, w)  # far rows as the gradient
        assert torch.equal(r["dx"], hk.layer_norm_backward(near, saved, w)["dx"])
        hk.layer_norm(near, w, b, out=far)
        assert torch.equal(far, want)
        hk.layer_norm_backward(dy, saved, w, out={"dx": far}, want=())
        assert torch.equal(far, grads["dx"])


def test_a_checkpoint_past_32_bits(hk):
    """More than 2^32 elements: codes, scales and rows at their far ends."""
    _room(60)
    n, d = 600000, 8192
    say("norm: a checkpoint of 4.9G elements")
    x = torch.empty((n, d), dtype=BF16, device="cuda")
    part = _rand((1000, d), 5)
    for i in range(0, n, 1000):
        x[i:i + 1000] = part
    for fmt in ("fp8", "mxfp8"):
        y, saved = hk.layer_norm(x, save=fmt)
        small, ref = hk.layer_norm(part, save=fmt)
        for i in (0, 262000, 524000, n - 1000):
            at = slice(i, i + 1000)
            assert torch.equal(y[at], small) and torch.equal(saved.rows[at], ref.rows) and torch.equal(saved.scale[at], ref.scale)
            assert torch.equal(saved.stats[at], ref.stats)
        r = hk.layer_norm_backward(y, saved, want=("dx",), out={"dx": y})
        want = hk.layer_norm_backward(small, ref, want=("dx",))["dx"]
        for i in (0, 262000, 524000, n - 1000):
            assert torch.equal(r["dx"][i:i + 1000], want)
        del y, saved, r
