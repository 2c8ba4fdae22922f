"""The operators together with the selection, as they are used: a training step
of the indexer, a decoded token, and a step recorded in a graph."""
import numpy as np
import pytest
import torch

import datagen
import oracle
from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rand(shape, seed, scale=1.0, dtype=torch.bfloat16):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def _inputs64(q, k, w):
    """The oracle's view of a bf16 problem on the GPU."""
    L, n, H, d = k.shape[0], q.shape[0], q.shape[1], q.shape[2]
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    return datagen.Inputs("chain", L, n, H, d, 0, "bf16", bits(q), bits(k), w.cpu().numpy())


def test_training_step(hk):
    """rotary -> select -> replay -> attention mass -> loss -> backward -> transposed rotation."""
    L, n, H, d, k, A = 600, 64, 16, 128, 96, 8
    say(f"chain: training L={L} n={n} H={H} d={d} k={k}")
    plan = hk.Rotary(64, layout="half", scaling="yarn", factor=4.0, original=256)
    xq, xk = _rand((n, H, d), 1, d ** -0.5), _rand((L, d), 2, d ** -0.5)
    w = torch.rand((n, H), generator=torch.Generator().manual_seed(3)).cuda()
    aq, ak = _rand((n, A, 64), 4, 2.0), _rand((L, 2, 64), 5)
    q = hk.rotary(xq, plan, q_start=L - n)
    key = hk.rotary(xk, plan)
    idx, score = hk.select(q, key, w, k)
    again = hk.replay(q, key, w, idx)
    assert torch.equal(again, score)
    mass = hk.attention_mass(aq, ak, idx)
    loss, d_score = hk.index_loss(again, mass)
    g = hk.backward(q, key, w, idx, d_score)
    dxq = hk.rotary(g["dq"], plan, q_start=L - n, backward=True, out_dtype=torch.bfloat16)
    dxk = hk.rotary(g["dk"], plan, backward=True)
    torch.cuda.synchronize()
    # every link against its definition on the link's own inputs
    inp = _inputs64(q, key, w)
    ref = oracle.replay(inp, idx.cpu().numpy())
    assert np.abs(score.double().cpu().numpy() - ref).max() < 1e-4 * (np.abs(ref).max() + 1)
    p64 = op.attention_mass(aq.double().cpu().numpy(), ak.double().cpu().numpy(), idx.cpu().numpy(), 0.125)
    m = mass.double().cpu().numpy()
    # logits below 40 in size and 64 products each: within 4 * 64 * 40 * 2^-24 * (|q||k| over |q.k|, below 8)
    assert np.abs(m - p64).max() <= 4 * 64 * 40 * 8 * 2.0 ** -24 * p64.max()
    rl, rg = op.index_loss(again.double().cpu().numpy(), m)
    # fp32 sums over 96 entries of terms below 20: 20 * (96 + 100) roundings
    assert np.abs(loss.double().cpu().numpy() - rl).max() <= 20 * 196 * 2.0 ** -24
    assert np.abs(d_score.double().cpu().numpy() - rg).max() <= 200 * 2.0 ** -24
    rgrad = oracle.backward(inp, idx.cpu().numpy(), d_score.cpu().numpy())
    for name in ("dq", "dw", "dk"):
        r = rgrad[name]
        assert np.abs(g[name].double().cpu().numpy() - r).max() <= 1e-3 * np.abs(r).max(), name
    f = plan.freq.cpu().numpy()
    want = op.rotary(g["dk"].double().cpu().numpy()[:, None], np.arange(L), f, gain=plan.gain, backward=True)[:, 0]
    assert np.abs(dxk.double().cpu().numpy() - want).max() <= 2.0 ** -20 * plan.gain * np.abs(want).max() * 2
    want = op.rotary(g["dq"].double().cpu().numpy(), np.arange(L - n, L), f, gain=plan.gain, backward=True)
    assert np.all(np.abs(dxq.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * np.abs(want).max())
    # the gradient points uphill: the chain's own loss along it (fp64, same selection)
    assert float(loss.sum()) > 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8", "mxfp4"])
def test_decode_step(hk, fmt):
    """A prompt written into a cache, then tokens one at a time: the keys at
    slots, the query quantised, the selection over the cache; equal to the selection over
    the same rows quantised at once."""
    L, H, d, k, steps = 700, 16, 128, 64, 3
    say(f"chain: decode {fmt}")
    plan = hk.Rotary(64, first=64, layout="interleaved")
    x = _rand((L + steps, d), 7)
    w = torch.rand((1, H), generator=torch.Generator().manual_seed(8)).cuda()
    whole, whole_s = hk.quantize(x, fmt, rotary=plan)
    codes, scale = torch.zeros_like(whole), None if whole_s is None else torch.zeros_like(whole_s)
    hk.cache_write(x[:L], codes, scale, fmt=fmt, rotary=plan)
    for t in range(steps):
        at = torch.tensor([L + t], dtype=torch.int32, device="cuda")
        hk.cache_write(x[L + t:L + t + 1], codes, scale, fmt=fmt, slots=at, rotary=plan, q_pos=at)
        xq = _rand((1, H, d), 20 + t)
        q, qs = hk.quantize(xq, fmt, rotary=plan, q_pos=at)
        kw = dict(q_pos=at, fmt=fmt, q_scale=qs)
        idx, score = hk.select(q, codes, w, k, k_scale=scale, **kw)
        i2, s2 = hk.select(q, whole, w, k, k_scale=whole_s, **kw)
        assert torch.equal(idx, i2) and torch.equal(score, s2)
        assert int(idx.max()) <= L + t
        kept = hk.cache_read(codes, scale, fmt=fmt, slots=idx[0], dtype=torch.float32).double()
        qv = hk.cache_read(q, qs, fmt=fmt, dtype=torch.float32).double()[0]
        ref = (torch.relu(kept @ qv.t()) * w[0].double()).sum(1)
        assert (ref - score[0].double()).abs().max() <= 1e-4 * (ref.abs().max() + 1)
    assert torch.equal(codes, whole) and (scale is None or torch.equal(scale, whole_s))


def test_training_step_in_a_graph(hk):
    """The whole chain recorded once, two graphs that share one workspace replayed in turn,
    eager calls and changed inputs between."""
    L, n, H, d, k, A = 500, 20, 8, 64, 40, 8
    plan = hk.Rotary(32)
    xq, xk = _rand((n, H, d), 31), _rand((L, d), 32)
    w = torch.rand((n, H), generator=torch.Generator().manual_seed(33)).cuda()
    aq, ak = _rand((n, A, 64), 34), _rand((L, 1, 64), 35)
    bufs = dict(q=torch.empty_like(xq), key=torch.empty_like(xk),
                idx=torch.zeros((n, k), dtype=torch.int32, device="cuda"), sc=torch.zeros((n, k), device="cuda"),
                mass=torch.zeros((n, k), device="cuda"), loss=torch.zeros(n, device="cuda"),
                grad=torch.zeros((n, k), device="cuda"), st=torch.zeros(8, dtype=torch.int32, device="cuda"))
    ws = torch.empty(hk.select_workspace_bytes(xq, xk, w, k), dtype=torch.uint8, device="cuda")
    need = max(hk.attention_mass_workspace_bytes(aq, ak, bufs["idx"]), 256)
    mws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(b):
        hk.rotary(xq, plan, q_start=L - n, out=b["q"])
        hk.rotary(xk, plan, out=b["key"])
        hk.select_async(b["q"], b["key"], w, k, workspace=ws, out=(b["idx"], b["sc"]), status=b["st"])
        hk.attention_mass(aq, ak, b["idx"], workspace=mws, out=b["mass"])
        hk.index_loss(b["sc"], b["mass"], out=(b["loss"], b["grad"]))
    step(bufs)
    torch.cuda.synchronize()
    other = {name: t.clone() for name, t in bufs.items()}
    graphs = []
    for b in (bufs, other):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(b)
        graphs.append(gr)
    for rep in range(3):
        xq.copy_(_rand((n, H, d), 50 + rep))
        aq.copy_(_rand((n, A, 64), 60 + rep))
        want = {name: t.clone() for name, t in bufs.items()}
        step(want)
        torch.cuda.synchronize()
        for gr, b in zip(graphs, (bufs, other)):
            gr.replay()
        torch.cuda.synchronize()
        for b in (bufs, other):
            for name in want:
                assert torch.equal(b[name], want[name]), (rep, name)
