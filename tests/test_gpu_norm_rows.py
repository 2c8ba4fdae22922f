"""Layer norm of rows where its arithmetic is at its limits, against the fp64 definition: constant rows of every size, whose mean
times rstd may pass fp32, on widths that leave some of a row's places empty.  u = 2^-24; tolerances of the two passes are those that
test_gpu_layer_norm derives."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as op
from test_gpu_layer_norm import check_backward, check_forward

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rand(shape, seed, dtype=FP32, scale=1.0, offset=0.0):
    return (offset + scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def f64(t):
    return t.double().cpu().numpy()


def _off_16_bytes(t):
    off = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    return off.copy_(t)


# 128, 1,024: every place of a row is taken; the others leave some empty
@pytest.mark.parametrize("d", [3, 24, 96, 100, 128, 201, 576, 1024, 1100, 5120, 7168])
def test_the_gradient_of_constant_rows_of_any_size(hk, d):
    """h is 0 in all of a constant row, so dx is rstd (g - mean(g)) and the row adds nothing to dweight, however far
    mean * rstd lies beyond fp32.  The statistics are the definition's: c and eps^(-1/2)."""
    say(f"norm: the gradient of constant rows, d={d}")
    top = 0.9 * 2.0 ** 127 / d  # the row's sum stays below 2^128
    x = torch.tensor([1.0, -1e6, 1e20, -1e-3 * top, top, 7.25, 0.0])[:, None].expand(7, d).contiguous()
    w, dy = _rand(d, 1, FP32, 0.2, 1.0), _rand((7, d), 2, FP32, d ** -0.5)
    for dtype in (FP32, BF16):
        rows = x.to(dtype).cuda()
        for eps in (1e-5, 1e-12):
            stats = torch.stack([rows[:, 0].float(), torch.full((7,), eps ** -0.5, device="cuda")], 1)
            for r, g in ((rows, dy), (_off_16_bytes(rows), dy), (rows, dy.to(BF16)), (rows, _off_16_bytes(dy))):
                got = hk.layer_norm_backward(g, hk.NormSaved(r, None, stats, None), w, dx_dtype=FP32)
                check_backward(got, g, f64(rows), stats, w)
                assert not got["dweight"].any()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8"])
@pytest.mark.parametrize("d", [32, 96, 544, 5120])
def test_the_gradient_of_constant_rows_from_a_checkpoint(hk, d, fmt):
    """Rows of 7 * 2^k: their checkpoints hold them exactly (448 of 2^(k - 6))."""
    k = 123 - int(np.ceil(np.log2(d)))  # 7 * 2^k * d is below 2^126
    x = torch.tensor([7.0 * 2.0 ** k, -7.0 * 2.0 ** (k - 20), 7.0, 0.0])[:, None].expand(4, d).contiguous().cuda()
    codes, scale = hk.quantize(x, fmt)
    stats = torch.stack([x[:, 0], torch.full((4,), 1000.0, device="cuda")], 1)
    w, dy = _rand(d, 3, FP32, 0.2, 1.0), _rand((4, d), 4, FP32, d ** -0.5)
    for g in (dy, dy.to(BF16), _off_16_bytes(dy)):
        got = hk.layer_norm_backward(g, hk.NormSaved(codes, scale, stats, fmt), w, dx_dtype=FP32)
        check_backward(got, g, f64(x), stats, w, coded=True)
        assert not got["dweight"].any()


# ----------------------------------------------------------------- forward

def _constants(d, seed):
    """Rows of one value each, of sizes from 1e-3 to 2^127 / d, among rows of their own values."""
    rng = np.random.default_rng(seed)
    size = np.array([1e-3, 1.0, 1e3, 1e6, 1e9, 1e15, 1e25, 0.5 * 2.0 ** 127 / d])
    c = (np.repeat(size, 12) * rng.uniform(1, 2, 96) * rng.choice([-1, 1], 96)).astype(np.float32)
    x = torch.from_numpy(c)[:, None].expand(96, d).clone()
    x[::4] = torch.from_numpy(rng.standard_normal((24, d)).astype(np.float32))
    flat = torch.ones(96, dtype=torch.bool)
    flat[::4] = d == 1
    return x, flat


# 41, 55, 107 and 3,993: d times the rounded 1 / d is not 1 after rounding
@pytest.mark.parametrize("d", [1, 3, 24, 41, 55, 64, 96, 107, 128, 160, 201, 576, 1000, 1536, 2056, 3993, 5120, 7168, 8191, 8192])
def test_constant_rows_of_any_size_give_the_bias(hk, d):
    """Deviations are 0 exactly: y is the bias, the mean the value, rstd eps^(-1/2) (the instruction's 2^-23, a rounding of eps), and
    NaN without eps.  The rows of normal numbers between them are the definition's."""
    say(f"norm: constant rows, d={d}")
    w, b = _rand(d, 5, FP32, 0.2, 1.0), _rand(d, 6)
    for dtype in (FP32, BF16):
        x, flat = _constants(d, d)
        x = x.to(dtype).cuda()
        saves = ["x"] + (["fp8", "mxfp8"] if d % 32 == 0 else [])
        for rows in (x, _off_16_bytes(x), x.view(32, 3, d)):
            for save in saves:
                for eps in (1e-5, 1e-12):
                    y, saved = hk.layer_norm(rows, w, b, eps=eps, out_dtype=FP32, save=save)
                    y, st = y.reshape(96, d), saved.stats.reshape(96, 2)
                    assert torch.equal(y[flat], b.expand(int(flat.sum()), d))
                    assert torch.equal(st[flat, 0], x[flat, 0].float())
                    assert float((st[flat, 1].double() * eps ** 0.5 - 1).abs().max()) <= 2.0 ** -22
                    if d > 1:
                        check_forward(y[~flat], st[~flat], x[~flat], w, b, eps)
        y = hk.layer_norm(x, w, b, eps=0.0, out_dtype=FP32)
        assert torch.isnan(y[flat]).all() and torch.isfinite(y[~flat]).all()
        # both passes together
        y, saved = hk.layer_norm(x, w, b, eps=1e-6, save="x")
        dy = _rand((96, d), 7, FP32, d ** -0.5)
        got = hk.layer_norm_backward(dy, saved, w)
        check_backward(got, dy, f64(x), saved.stats, w)
        assert torch.isfinite(got["dx"]).all() and torch.isfinite(got["dweight"]).all()


@pytest.mark.parametrize("d", [96, 128, 1100, 5120])
def test_rows_far_from_zero(hk, d):
    """Rows of deviations of size 1 about 2^10 .. 2^22, their first element among the others, far from them, or next to the mean.  A shift m0
    within 2^-18 of the mean (2^-19 of itself from a value, 17 roundings) leaves the mean of the deviations below 2^-18 |mean|, whose
    square is taken from that of the deviations: rstd is off by 28 u of 1 + 2 (2^-18 mean)^2 / var, of var here about 1."""
    say(f"norm: rows far from zero, d={d}")
    base = _rand((39, d), 8)
    base[0::3, 0] = 30.0
    base[1::3, 0] = 0.0
    off = 2.0 ** torch.arange(10, 23).repeat_interleave(3).double().cuda()
    x = (base.double() + off[:, None]).float()
    x64 = f64(x)
    y, saved = hk.layer_norm(x, eps=1e-6, save="x")
    mean, var = x64.mean(1, keepdims=True), x64.var(1, keepdims=True)
    rstd = (var + 1e-6) ** -0.5
    ratio = 1 + 2 * (2.0 ** -18 * mean) ** 2 / var
    st = f64(saved.stats)
    assert (np.abs(st[:, 1:] / rstd - 1) <= 32 * U * ratio).all()
    assert (np.abs(st[:, :1] - mean) <= U * np.abs(mean) + 56 * U * (2.0 ** -18 * mean + var ** 0.5)).all()
    # a deviation is off by 2 u of itself and of the shift, the deviations' mean by 50 u of theirs, y by rstd's error and three roundings
    c = np.abs(x64 - mean)
    tol = rstd * (2 * U * (c + 2.0 ** -18 * mean) + 52 * U * (c.mean(1, keepdims=True) + 2.0 ** -18 * mean)) + c * rstd * U * (32 * ratio + 3)
    assert (np.abs(f64(y) - (x64 - mean) * rstd) <= tol).all()


# ------------------------------------------- the gradient far from zero

@pytest.mark.parametrize("d", [96, 128, 1100, 5120])
@pytest.mark.parametrize("offset", [0.0, 2.0 ** 10, 2.0 ** 15, 2.0 ** 18])
def test_the_gradient_of_rows_far_from_zero(hk, d, offset):
    """Against the derivative with the mean and deviation of x in 64 bits.  The mean is kept in fp32, off by u |mean| (and 52 u of the
    deviations' mean size), so h is off by that times rstd; rstd, off by 32 u, is in h and in dx."""
    say(f"norm: the gradient far from zero, d={d}, {offset}")
    x, w, dy = _rand((64, d), 9, FP32, offset=offset), _rand(d, 10, FP32, 0.2, 1.0), _rand((64, d), 11, FP32, d ** -0.5)
    _, saved = hk.layer_norm(x, w, eps=1e-6, save="x")
    got = hk.layer_norm_backward(dy, saved, w)
    x64, dy64, w64 = f64(x), f64(dy), f64(w)
    mean, rstd = x64.mean(1), (x64.var(1) + 1e-6) ** -0.5
    dx, dw, db = op.layer_norm_backward(dy64, x64, mean, rstd, w64)
    r, a = rstd[:, None], np.abs(dy64)
    dev = np.abs(x64 - mean[:, None])
    h, g = dev * r, a * np.abs(w64)
    eh = r * (1.001 * U * np.abs(mean)[:, None] + 52 * U * dev.mean(1, keepdims=True)) + 34 * U * h
    row = lambda t: t.mean(1, keepdims=True)  # noqa: E731
    size = g + row(g) + h * row(g * h)
    tol = r * (eh * row(g * h) + (h + eh) * row(g * eh) + (32 + 60) * U * size)
    assert (np.abs(f64(got["dx"]) - dx) <= tol).all()
    chain = 155 + 64 / 256
    assert (np.abs(f64(got["dweight"]) - dw) <= U * chain * (a * h).sum(0) + (a * eh).sum(0)).all()
    assert (np.abs(f64(got["dbias"]) - db) <= U * chain * a.sum(0)).all()
