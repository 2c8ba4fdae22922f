"""Calls at the edges of what the operators around the selection allow: slices of one buffer, far positions,
plans of a model's own, values at the ends of their range."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotary_between_slices_of_one_buffer(hk, dtype):
    """One slice of a fused projection rotated into another: the result of separate buffers, and every other
    element as it was."""
    n, h, d = 37, 3, 64
    plan = hk.Rotary(32, first=16)
    for shape, x_at, y_at in (((n, h, 200), np.s_[..., :d], np.s_[..., d:2 * d]), ((n, h, 200), np.s_[..., 136:], np.s_[..., 3:3 + d]),
                              ((n, 3 * h, d), np.s_[:, :h], np.s_[:, 2 * h:]), ((n, 2, h, d), np.s_[:, 1], np.s_[:, 0])):
        say(f"rotary between slices: {shape} {dtype}")
        fused = _rand(shape, 3, dtype)
        before = fused.clone()
        want = hk.rotary(fused[x_at].contiguous(), plan, q_start=70)
        hk.rotary(fused[x_at], plan, q_start=70, out=fused[y_at])
        assert torch.equal(fused[y_at], want)
        before[y_at] = want
        assert torch.equal(fused, before)


def test_rotary_angles_at_the_ends_of_int32(hk):
    """Cosines and sines themselves (rows of ones and zeros, fp32) at positions up to 2^31, where one rounding of
    a product in 64 bits is 3 * 2^-24 of a radian.  In units of 2^-24: the turn's rounding to fp32, 2 pi 2^-26:
    1.58; 2 pi as fp32 and its product, 1.47 of an angle up to pi/4: 1.16; the cosine's polynomial 0.42 left off,
    its terms 0.6, its last rounding 0.5 (the sine's less): 1.52.  4.26 together."""
    far = 2 ** 31 - 1 - np.arange(600) * 977
    pos = np.concatenate([far, -far - 1, 2 ** 30 + np.arange(300), 2 ** 20 + np.arange(100), np.arange(100)])
    for plan in (hk.Rotary(64), hk.Rotary(128, base=1000000.0, layout="interleaved"),
                 hk.Rotary(64, scaling="linear", factor=3.0), hk.Rotary(64, scaling="ntk", factor=7.0)):
        half = plan.dim // 2
        x = np.zeros((len(pos), 2, plan.dim), np.float32)  # (1, 0) gives (cos, sin), (0, 1) gives (-sin, cos)
        a, b = (np.s_[:half], np.s_[half:]) if plan.layout == "half" else (np.s_[0::2], np.s_[1::2])
        x[:, 0, a] = 1
        x[:, 1, b] = 1
        y = hk.rotary(torch.from_numpy(x).cuda(), plan, q_pos=torch.from_numpy(pos.astype(np.int32)).cuda())
        ref = op.rotary(x.astype(np.float64), pos, plan.freq.cpu().numpy(), layout=plan.layout)
        err = np.abs(y.double().cpu().numpy() - ref)
        say(f"rotary angles: largest error {err.max() / U:.2f} * 2^-24")
        assert err.max() <= 4.26 * U, (np.argwhere(err > 4.26 * U)[0], err.max() / U)
        assert np.array_equal(y[:, 1, b].cpu().numpy(), y[:, 0, a].cpu().numpy())


def test_rotary_with_a_gain_and_frequencies_of_its_own(hk):
    f = np.geomspace(3.0, 1e-6, 16)
    x, pos = _rand((40, 3, 64), 4, torch.float32), np.arange(5000, 5040)
    for kw in (dict(gain=1.0, scaling="yarn", factor=40.0, original=4096), dict(freq=f), dict(freq=torch.from_numpy(f).cuda(), gain=-0.75)):
        plan = hk.Rotary(32, first=8, **kw)
        y = hk.rotary(x, plan, q_start=5000).double().cpu().numpy()
        x64 = x.double().cpu().numpy()
        freq = f if "freq" in kw else plan.freq.cpu().numpy()
        gain = kw.get("gain", 1.0)
        ref = op.rotary(x64, pos, freq, first=8, gain=gain)
        # 2^-21 gain (|a| + |b|), as derived in test_gpu_rotary.py
        both = 2.0 ** -21 * abs(gain) * (np.abs(x64[..., 8:24]) + np.abs(x64[..., 24:40]))
        assert np.all(np.abs(y - ref)[..., 8:40] <= np.concatenate([both, both], -1))
        assert np.array_equal(y[..., :8], x64[..., :8]) and np.array_equal(y[..., 40:], x64[..., 40:])


@pytest.mark.parametrize("k", [40, 61, 700, 1999, 2048])
def test_index_loss_of_live_entries_at_the_lowest_score(hk, k):
    """A score of the type's lowest value is live: with mass there the loss is t * 3.4e38 an entry, and finite.
    t: a sum of k terms in k/64 + 6 steps, a reciprocal and a product; a term two more roundings; the terms' sum the
    same steps again, and the weight's product."""
    low = torch.finfo(torch.float32).min
    score, mass = torch.zeros(3, k), torch.ones(3, k)
    score[:, -5:] = low
    score[1, :3] = torch.tensor([4.0, -20.0, 30.0])
    score[2] = -1e30
    score[2, 7:] = low
    mass[2, 7:-1] = 0.0
    weight = torch.tensor([0.125, 1.0, 0.25])
    loss, grad = hk.index_loss(score.cuda(), mass.cuda(), weight=weight.cuda())
    rl, rg = op.index_loss(score.numpy(), mass.numpy(), weight.numpy())
    assert np.isfinite(rl).all() and (rl > 1e34).all()
    steps = 2 * (k / 64 + 6) + 6
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= steps * U * rl)
    # p: the exponential of an exact 0, -24, 26 or nothing below 2^-23 of itself, its row's sum, reciprocal, product
    p = rg / weight[:, None].numpy() + mass.numpy() / mass.sum(1, keepdim=True).numpy()
    tol = ((k / 64 + 6 + 100) * p + (k / 64 + 10) / 7) * U
    assert np.all(np.abs(grad.double().cpu().numpy() - rg) <= tol)


@pytest.mark.parametrize("k", [5, 64, 700, 2047, 2048])
def test_index_loss_of_masses_whose_sum_passes_fp32(hk, k):
    """Finite masses, an infinite sum: the same bits as from the masses times 2^-40 (a power of two moves no
    rounding).  An infinity itself shows, in its row alone."""
    g = torch.Generator().manual_seed(k)
    score = torch.randn((5, k), generator=g)
    mass = torch.rand((5, k), generator=g) * 1e38 + 2e38
    mass[1, 2:] = 3.0
    score[2, k // 2:] = -float("inf")
    mass[2, k // 2:] = float("inf")  # no part of the row
    assert torch.isinf(mass.sum(1)[[0, 1, 3]]).all()
    loss, grad = hk.index_loss(score.cuda(), mass.cuda())
    small = torch.where(torch.isinf(mass), mass, mass * 2.0 ** -40)
    l2, g2 = hk.index_loss(score.cuda(), small.cuda())
    assert torch.isfinite(loss).all() and torch.equal(loss, l2) and torch.equal(grad, g2)
    rl, rg = op.index_loss(score.numpy(), mass.numpy())
    # t and p within their row's sum (k/64 + 6 steps) and 100 roundings
    assert np.all(np.abs(grad.double().cpu().numpy() - rg) <= (k / 64 + 106) * U)
    mass[3, 1] = float("inf")
    l3, g3 = hk.index_loss(score.cuda(), mass.cuda())
    keep = [0, 1, 2, 4]
    assert torch.isnan(l3[3]) and torch.equal(l3[keep], loss[keep]) and torch.equal(g3[keep], grad[keep])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rotary_of_every_scaling_by_the_oracle_s_own_plan(hk, scaling, layout):
    dim, base, factor, original, first = 64, 500000.0, 8.0, 8192, 32
    plan = hk.Rotary(dim, first=first, layout=layout, base=base, scaling=scaling, factor=factor, original=original)
    freq, gain = op.rotary_plan(dim, base, scaling, factor, original)
    x = _rand((200, 3, 128), 11, torch.float32)
    pos = np.random.default_rng(4).integers(0, 1 << 17, 200)
    y = hk.rotary(x, plan, q_pos=torch.from_numpy(pos.astype(np.int32)).cuda()).double().cpu().numpy()
    x64 = x.double().cpu().numpy()
    ref = op.rotary(x64, pos, freq, first=first, layout=layout, gain=gain)
    # 2^-21 gain (|a| + |b|), as derived in test_gpu_rotary.py, which leaves room for the plans' 1e-13 of 2^17 radians
    part = np.abs(x64[..., first:first + dim])
    both = part + (np.roll(part, dim // 2, -1) if layout == "half" else part.reshape(200, 3, -1, 2)[..., ::-1].reshape(part.shape))
    assert np.all(np.abs(y - ref)[..., first:first + dim] <= 2.0 ** -21 * gain * both)
    assert np.array_equal(y[..., :first], x64[..., :first]) and np.array_equal(y[..., first + dim:], x64[..., first + dim:])


def test_the_training_step_s_gradient_is_its_loss_s_slope(hk):
    """rotary -> select -> replay -> attention mass -> loss -> backward -> transposed rotation: the loss in
    64 bits (the selection and the mass fixed) rises along the gradients of the rows before the rotation
    and of the weights as steeply as those gradients are long."""
    L, n, H, d, k, A = 500, 24, 16, 128, 80, 8
    plan = hk.Rotary(64, first=32, layout="interleaved", scaling="yarn", factor=4.0, original=256)
    rand = lambda shape, seed, f=1.0: (f * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()  # noqa: E731
    xq, xk = rand((n, H, d), 1, 0.3), rand((L, d), 2, 0.3)
    w = torch.rand((n, H), generator=torch.Generator().manual_seed(3)).cuda()
    q, key = hk.rotary(xq, plan, q_start=L - n), hk.rotary(xk, plan)
    idx, score = hk.select(q, key, w, k)
    mass = hk.attention_mass(rand((n, A, 64), 4, 2.0), rand((L, 2, 64), 5), idx)
    _, d_score = hk.index_loss(hk.replay(q, key, w, idx), mass)
    g = hk.backward(q, key, w, idx, d_score)
    dxq = hk.rotary(g["dq"], plan, q_start=L - n, backward=True)
    dxk = hk.rotary(g["dk"], plan, backward=True)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    q0, k0, w0, m0, at = host(q), host(key), host(w), host(mass), idx.cpu().numpy()
    live = at >= 0

    def loss(q, key, w):
        dots = np.maximum(np.matmul(key[at], q.transpose(0, 2, 1)), 0.0)  # [n][k][H]
        s = np.where(live, (dots * w[:, None]).sum(-1), -np.inf)
        return op.index_loss(s, m0)[0].sum()

    freq = plan.freq.cpu().numpy()
    turn = lambda v, pos: op.rotary(v, pos, freq, first=32, layout="interleaved", gain=plan.gain)  # noqa: E731
    zero = (0 * q0, 0 * k0, 0 * w0)
    for name, grad, move, raw in (("dq", host(dxq), lambda v: (turn(v, np.arange(L - n, L)), zero[1], zero[2]), host(g["dq"])),
                                  ("dk", host(dxk), lambda v: (zero[0], turn(v[:, None], np.arange(L))[:, 0], zero[2]), host(g["dk"])),
                                  ("dw", host(g["dw"]), lambda v: (zero[0], zero[1], v), host(g["dw"]))):
        length = np.sqrt((grad ** 2).sum())
        u = move(grad / length)
        h = 1e-5
        up, down = (loss(q0 + t * u[0], k0 + t * u[1], w0 + t * u[2]) for t in (h, -h))
        slope = (up - down) / (2 * h)
        say(f"slope along {name}: {slope:.6f}, length {length:.6f}")
        # the backward's results lie within 1e-3 of their largest (test_gpu_operators_chain.py), here summed over the unit direction;
        # the difference itself 1e-9 of the loss over 2 h, and ReLU's corners h of the slope
        tol = 1e-3 * np.abs(raw).max() * plan.gain * np.abs(grad).sum() / length + 1e-9 * abs(up) / h + 10 * h * length
        assert slope > 0 and abs(slope - length) <= tol


def test_rotary_cosines_and_sines_are_rounded_little_more_than_once(hk):
    """In units of 2^-24, at any position: the rest of the nearest quarter turn as fp32, pi/2 2^-26, moves a cosine below
    0.71 by 0.28; its polynomial r^2 Q, up to 0.29, three roundings relative to it, 0.88; the last rounding 0.5.  The
    sine: 0.37, r P up to 0.08 four roundings, 0.31, the last 0.5, what the polynomial leaves off 0.04.  1.67 at most.
    Frequencies above a turn a position, and negative ones, among them."""
    rng = np.random.default_rng(9)
    pos = np.concatenate([rng.integers(-2 ** 31, 2 ** 31, 1500), np.arange(500), [2 ** 31 - 1, -2 ** 31]])
    odd = np.concatenate([rng.uniform(-9, 9, 40), np.pi / 2 * np.arange(1, 9), np.geomspace(1e-12, 10, 16)])
    for plan in (hk.Rotary(64), hk.Rotary(64, base=1000000.0, scaling="yarn", factor=32.0, original=32768, gain=1.0), hk.Rotary(128, freq=odd)):
        half = plan.dim // 2
        x = np.zeros((len(pos), 1, plan.dim), np.float32)
        x[..., :half] = 1  # gives (cos, sin)
        y = hk.rotary(torch.from_numpy(x).cuda(), plan, q_pos=torch.from_numpy(pos.astype(np.int32)).cuda())
        # the reference's own mantissa of 64 bits: three roundings of 4.3e9 turns, 0.08
        ref = op.rotary(x.astype(np.float64), pos, plan.freq.cpu().numpy())
        err = np.abs(y.double().cpu().numpy() - ref)
        say(f"rotary cosines and sines: largest error {err.max() / U:.2f} * 2^-24")
        assert err.max() <= 1.75 * U, (np.argwhere(err > 1.75 * U)[0], err.max() / U)
