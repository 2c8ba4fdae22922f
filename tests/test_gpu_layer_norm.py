"""Layer norm and its 8-bit checkpoints against the fp64 definition (oracle.operators).

Tolerances, with u = 2^-24 and at most N = 48 additions one behind the other in a row's sum (24 or 32 of a thread,
6 over lanes, 8 over waves).  Forward: m0 is a number; c = x - m0 is off by u |c|, its mean by (N + 2) u mean|c|, so a
deviation by u (2 |c| + 50 mean|c|); the variance is off by 56 u of var + mean(c)^2 and its inverse root by half that and 3 u
(the instruction's 2^-23, a rounding): 31 u where mean(c)^2 is small; product, weight and sum 3 u more.  |c| is at most
|x - mean| + 48 u mean|x|.  Backward, from statistics given in fp32: h is off by eh = 2 u |h| (u |x| rstd more
where x is a code times an fp32 scale), g = dy w by u |g|, the means by (N + 3) u of the means of the sizes, and three
roundings of each of the three terms.  Sums over rows: a thread's rows one behind the other (at most rows / 256 + 1), then at most 150
additions, each off by u of the sum of the sizes, and 4 u of each product.  A result in bf16 adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import datagen
import oracle
from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rand(shape, seed, dtype=FP32, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (offset + scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def _rows(n, heads, d, seed, dtype):
    """Rows of different sizes and offsets."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, d), generator=g) * torch.exp(torch.randn((n, heads, 1), generator=g))
    return (x + torch.randn((n, heads, 1), generator=g)).to(dtype).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def _params(w, b, d):
    return (np.ones(d) if w is None else f64(w)), (np.zeros(d) if b is None else f64(b))


def _half_step(t, ref, tol):
    return tol + (2.0 ** -8 * (np.abs(ref) + tol) if t.dtype == BF16 else 0.0)


def _close(got, ref, tol, what):
    err = np.abs(f64(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[0], err[bad][0], tol[bad][0], ref[bad][0])


def check_forward(y, stats, x, w, b, eps):
    x64 = f64(x)
    w64, b64 = _params(w, b, x64.shape[-1])
    ref, mean, rstd = op.layer_norm(x64, w64, b64, eps)
    c = np.abs(x64 - mean[..., None]) + 48 * U * np.abs(x64).mean(-1, keepdims=True)
    cm = c.mean(-1, keepdims=True)
    tol = U * (np.abs(w64) * rstd[..., None] * (2 * c + 50 * cm) + 34 * np.abs(ref - b64) + 2 * np.abs(ref))
    _close(y, ref, _half_step(y, ref, tol), "y")
    if stats is not None:
        _close(stats[..., 0], mean, U * (2 * np.abs(mean) + 52 * cm[..., 0]), "mean")
        _close(stats[..., 1], rstd, 32 * U * rstd, "rstd")


def check_backward(res, dy, x64, stats, w, coded=False):
    """res: the gradients; x64: the rows that the backward read."""
    dy64, st = f64(dy), f64(stats)
    d = x64.shape[-1]
    w64, _ = _params(w, None, d)
    mean, rstd = st[..., 0], st[..., 1]
    dx, dw, db = op.layer_norm_backward(dy64, x64, mean, rstd, w64)
    r = rstd[..., None]
    h = np.abs(x64 - mean[..., None]) * r
    eh = U * (2 * h + (np.abs(x64) * r if coded else 0.0))
    g = np.abs(dy64 * w64)
    row = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    gm, ghm = row(g), row(g * h)
    if res.get("dx") is not None:
        tol = r * (5 * U * g + 56 * U * gm + eh * ghm + h * (row(g * eh) + 58 * U * ghm)) + U * np.abs(dx)
        _close(res["dx"], dx, _half_step(res["dx"], dx, tol), "dx")
    axes = tuple(range(x64.ndim - 1))
    chain = 151 + int(np.prod(x64.shape[:-1])) / 256
    a = np.abs(dy64)
    if res.get("dweight") is not None:
        _close(res["dweight"], dw, U * (chain + 4) * (a * h).sum(axes) + (a * eh).sum(axes), "dweight")
    if res.get("dbias") is not None:
        _close(res["dbias"], db, U * chain * a.sum(axes), "dbias")


SHAPES = [  # n, heads, d: every number of threads and pieces a row, whole and partial pieces, one row and many
    (1, 1, 128), (1, 64, 128), (7, 3, 64), (300, 1, 128), (2049, 1, 128), (33, 5, 32), (5, 2, 16), (9, 1, 8), (4, 3, 1), (6, 1, 2),
    (3, 1, 7), (19, 2, 100), (5, 4, 201), (17, 1, 256), (11, 1, 512), (6, 1, 520), (5, 1, 576), (9, 1, 1000), (4, 1, 1024),
    (3, 1, 1537), (5, 1, 2048), (3, 1, 2056), (7, 1, 2560), (2, 1, 4096), (3, 1, 5120), (2, 1, 6144), (3, 1, 7168), (2, 1, 8191),
    (600, 1, 8192), (1, 1, 8192), (40000, 1, 24),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_both_passes_match_the_definition(hk, shape):
    n, heads, d = shape
    say(f"layer norm {shape}")
    types = [(BF16, BF16, FP32), (FP32, FP32, FP32), (BF16, FP32, None), (FP32, BF16, BF16)] if n * d < 100000 else [(BF16, BF16, FP32)]
    for tx, ty, tw in types:
        x = _rows(n, heads, d, n + d, tx)
        w = None if tw is None else _rand(d, 1, tw, 0.2, 1.0)
        b = None if tw is None else _rand(d, 2, tw, 0.1)
        y, saved = hk.layer_norm(x, w, b, eps=1e-6, out_dtype=ty, save="x")
        assert y.dtype == ty and saved.rows is x and saved.fmt is None and saved.stats.shape == (n, heads, 2)
        check_forward(y, saved.stats, x, w, b, 1e-6)
        assert torch.equal(hk.layer_norm(x, w, b, eps=1e-6, out_dtype=ty), y)
        for tg, tdx in ((BF16, None), (FP32, BF16), (FP32, None), (BF16, FP32)):
            dy = _rand((n, heads, d), 3, tg, d ** -0.5)
            res = hk.layer_norm_backward(dy, saved, w, dx_dtype=tdx)
            assert set(res) == {"dx", "dweight", "dbias"} and res["dx"].dtype == (tdx or tg)
            check_backward(res, dy, f64(x), saved.stats, w)


def test_two_axes_equal_three(hk):
    x, w, b = _rows(21, 1, 128, 4, BF16), _rand(128, 5), _rand(128, 6)
    dy = _rand((21, 1, 128), 7)
    y3, s3 = hk.layer_norm(x, w, b, save="x")
    y2, s2 = hk.layer_norm(x[:, 0], w, b, save="x")
    assert torch.equal(y2, y3[:, 0]) and torch.equal(s2.stats, s3.stats[:, 0])
    a, c = hk.layer_norm_backward(dy, s3, w), hk.layer_norm_backward(dy[:, 0], s2, w)
    assert torch.equal(a["dx"][:, 0], c["dx"]) and torch.equal(a["dweight"], c["dweight"])


def test_the_gradient_is_the_slope(hk):
    """dx, dweight and dbias against differences of the fp64 definition along random directions: with a step of 1e-5 the
    third derivative's share is below 1e-8 of a slope whose rows are of size 1, the result's own roundings 2^-20 of its parts."""
    n, heads, d = 6, 2, 96
    x, w, b = _rand((n, heads, d), 8), _rand(d, 9, FP32, 0.3, 1.0), _rand(d, 10)
    dy = _rand((n, heads, d), 11)
    _, saved = hk.layer_norm(x, w, b, eps=1e-5, save="x")
    res = hk.layer_norm_backward(dy, saved, w)
    rng = np.random.default_rng(12)
    for _ in range(8):
        vx, vw, vb = rng.standard_normal((n, heads, d)), rng.standard_normal(d), rng.standard_normal(d)

        def at(t):
            return (f64(dy) * op.layer_norm(f64(x) + t * vx, f64(w) + t * vw, f64(b) + t * vb, 1e-5)[0]).sum()
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        parts = [(f64(res["dx"]) * vx), (f64(res["dweight"]) * vw), (f64(res["dbias"]) * vb)]
        got, size = sum(p.sum() for p in parts), sum(np.abs(p).sum() for p in parts)
        assert abs(got - slope) <= 2.0 ** -18 * size + 1e-6 * abs(slope)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_offsets_and_sizes_of_rows(hk, dtype):
    """Rows far from zero, small and large rows, constant rows: an offset does not reach the deviations."""
    d = 128
    base = _rand((8, d), 13)
    x = torch.stack([base[0], base[1] + 1000, base[2] * 1e-3 + 30, base[3] * 1e15, base[4] * 1e-18, base[5] * 0 + 7.25,
                     base[6] * 0, torch.where(torch.arange(d, device="cuda") == 5, 1e6, base[7])]).to(dtype)
    w, b = _rand(d, 14, FP32, 0.2, 1.0), _rand(d, 15)
    for eps in (1e-6, 1e-12):
        y, saved = hk.layer_norm(x, w, b, eps=eps, out_dtype=FP32, save="x")
        check_forward(y, saved.stats, x, w, b, eps)
        assert torch.equal(y[5], b) and torch.equal(y[6], b)
        dy = _rand((8, d), 16)
        check_backward(hk.layer_norm_backward(dy, saved, w), dy, f64(x), saved.stats, w)
    # an offset of fp32 rows that their sum cannot hold to the size of the deviations
    if dtype == FP32:
        x = (base + 2.0 ** 15).contiguous()
        y = hk.layer_norm(x, eps=1e-6)
        check_forward(y, None, x, None, None, 1e-6)


def test_without_eps(hk):
    d = 64
    x = _rand((5, d), 17) * torch.tensor([1.0, 1e-20, 1e-19, 1e10, 0.0], device="cuda")[:, None]
    y, saved = hk.layer_norm(x, eps=0.0, save="x")
    # rows whose squares are subnormal (1e-40) carry fewer bits: within 2^-140 of 1e-40 a square, 2^-7 of the sum
    x64 = f64(x)
    ref, _, _ = op.layer_norm(x64[:4], 1.0, 0.0, 0.0)
    got = f64(y)
    for i, rel in ((0, 1e-5), (1, 2.0 ** -6), (2, 2.0 ** -12), (3, 1e-5)):
        assert np.abs(got[i] - ref[i]).max() <= rel * np.abs(ref[i]).max(), i
    assert np.isnan(got[4]).all()


def test_rows_that_are_not_finite_stay_alone(hk):
    d = 200
    x = _rand((40, d), 18, BF16)
    clean, saved0 = hk.layer_norm(x, save="x")
    bad = x.clone()
    bad[3, 7], bad[11, 0], bad[39, d - 1] = float("inf"), float("nan"), float("-inf")
    y, saved = hk.layer_norm(bad, save="x")
    rows = torch.tensor([3, 11, 39])
    assert torch.isnan(y[rows]).all()
    keep = torch.ones(40, dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(y[keep], clean[keep]) and torch.equal(saved.stats[keep], saved0.stats[keep])
    dy = _rand((40, d), 19)
    dx, dx0 = (hk.layer_norm_backward(dy, s, want=("dx",))["dx"] for s in (saved, saved0))
    assert torch.equal(dx[keep], dx0[keep]) and torch.isnan(dx[rows]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 96, 1100])
def test_strides_alignment_and_in_place(hk, dtype, d):
    n, h = 13, 3
    base, w, b = _rows(n, h, d, 20, dtype), _rand(d, 21, BF16, 0.2, 1.0), _rand(d, 22, BF16)
    dy = _rand((n, h, d), 23, dtype)
    want, saved = hk.layer_norm(base, w, b, save="x")
    check_forward(want, saved.stats, base, w, b, 1e-5)
    grads = hk.layer_norm_backward(dy, saved, w)
    check_backward(grads, dy, f64(base), saved.stats, w)

    def views(t):
        fused = torch.full((n, h, 3 * d), 2.0, dtype=dtype, device="cuda")
        fused[..., d:2 * d] = t
        swapped = t.transpose(0, 1).contiguous().transpose(0, 1)
        off = torch.empty(n * h * d + 1, dtype=dtype, device="cuda")[1:].view(n, h, d)
        off.copy_(t)
        return fused[..., d:2 * d], swapped, off
    for x, g in zip(views(base), views(dy)):
        y, s = hk.layer_norm(x, w, b, save="x")
        assert torch.equal(y, want) and torch.equal(s.stats, saved.stats)
        r = hk.layer_norm_backward(g, s, w)
        # the same order of additions however the rows lie
        for name in grads:
            assert torch.equal(r[name], grads[name]), name
        out = torch.empty((n, h, d + 5), dtype=dtype, device="cuda").fill_(3.0)
        hk.layer_norm(x, w, b, out=out[..., 5:])
        assert torch.equal(out[..., 5:], want) and bool((out[..., :5] == 3.0).all())
        hk.layer_norm_backward(g, s, w, out={"dx": out[..., 5:]}, want=())
        assert torch.equal(out[..., 5:], grads["dx"]) and bool((out[..., :5] == 3.0).all())
    # in place: the result over x, dx over dy and over x; what lies beside the rows stays
    fused, _, _ = views(base)
    hk.layer_norm(fused, w, b, out=fused)
    assert torch.equal(fused, want) and bool((fused._base[..., :d] == 2.0).all()) and bool((fused._base[..., 2 * d:] == 2.0).all())
    g = dy.clone()
    r = hk.layer_norm_backward(g, saved, w, out={"dx": g})
    assert torch.equal(g, grads["dx"]) and torch.equal(r["dweight"], grads["dweight"])
    kept = saved._replace(rows=base.clone())
    r = hk.layer_norm_backward(dy, kept, w, out={"dx": kept.rows})
    assert torch.equal(kept.rows, grads["dx"]) and torch.equal(r["dbias"], grads["dbias"])
    # x and dy broadcast over heads and tokens
    one, g1 = base[:, :1], dy[:1]
    y, s = hk.layer_norm(one.expand(n, h, d), w, b, save="x")
    assert torch.equal(y, want[:, :1].expand(n, h, d))
    r = hk.layer_norm_backward(g1.expand(n, h, d), s, w)
    check_backward(r, g1.expand(n, h, d), f64(one.expand(n, h, d)), s.stats, w)


def test_some_gradients(hk):
    x, w, dy = _rows(50, 2, 72, 24, BF16), _rand(72, 25), _rand((50, 2, 72), 26)
    _, saved = hk.layer_norm(x, w, save="x")
    every = hk.layer_norm_backward(dy, saved, w)
    for want in (("dx",), ("dweight",), ("dbias",), ("dweight", "dbias"), ("dx", "dbias"), ()):
        got = hk.layer_norm_backward(dy, saved, w, want=want)
        assert set(got) == set(want) and all(torch.equal(got[k], every[k]) for k in want)
    none = hk.layer_norm_backward(dy, saved, None)
    check_backward(none, dy, f64(x), saved.stats, None)
    assert torch.equal(none["dweight"], every["dweight"])


def test_no_rows(hk):
    for shape in ((0, 64), (0, 3, 64)):
        x = torch.empty(shape, device="cuda")
        for save in ("x", "fp8", "mxfp8"):
            y, saved = hk.layer_norm(x, save=save)
            assert y.shape == shape
            r = hk.layer_norm_backward(x, saved, out={"dweight": torch.full((64,), 5.0, device="cuda")})
            assert r["dx"].shape == shape and not r["dweight"].any() and not r["dbias"].any()


@pytest.mark.parametrize("d", [64, 128, 201, 576, 1024, 4096, 8192])
def test_few_rows(hk, d):
    """Around the number of rows up to which one workgroup writes the sums itself; each of the sums alone."""
    w = _rand(d, 50, FP32, 0.2, 1.0)
    at_once = max(1, 512 // max(1, 1 << max(0, (d + 7) // 8 - 1).bit_length()))
    seen = set()
    for n in sorted({1, 2, 3, 4, 5, *(k * at_once + e for k in (1, 2, 4, 8, 32) for e in (-1, 0, 1))} - {0}):
        x, dy = _rows(n, 1, d, n, BF16)[:, 0], _rand((n, d), n + 1)
        _, saved = hk.layer_norm(x, w, save="x")
        seen.add(hk.layer_norm_backward_workspace_bytes(dy) == 0)
        res = hk.layer_norm_backward(dy, saved, w)
        check_backward(res, dy, f64(x), saved.stats, w)
        for name in ("dweight", "dbias"):
            assert torch.equal(hk.layer_norm_backward(dy, saved, w, want=(name,))[name], res[name]), (n, name)
        # results in the middle of other memory: nothing beside them is written
        room = torch.full((3, d + 3), 7.0, device="cuda")
        out = {"dweight": room[2, 1:d + 1], "dbias": room[0, 2:d + 2]}
        hk.layer_norm_backward(dy, saved, w, want=(), out=out)
        assert torch.equal(out["dweight"], res["dweight"]) and torch.equal(out["dbias"], res["dbias"])
        assert bool((room[1] == 7.0).all()) and int((room == 7.0).sum()) >= (d + 3) + 6
    assert seen == {True, False}


def test_sums_far_apart(hk):
    """dweight and dbias more than 2^31 floats apart, either first, dx over dy."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    d = 96
    base = torch.empty((1 << 31) + 4 * d, device="cuda")
    x, w, dy = _rows(20, 2, d, 51, BF16), _rand(d, 52), _rand((20, 2, d), 53)
    _, saved = hk.layer_norm(x, w, save="x")
    want = hk.layer_norm_backward(dy, saved, w)
    lo, hi = base[:d], base[-d:]
    for a, b in ((lo, hi), (hi, lo)):
        g = dy.clone()
        r = hk.layer_norm_backward(g, saved, w, out={"dweight": a, "dbias": b, "dx": g})
        assert all(torch.equal(r[name], want[name]) for name in want)


def test_sums_of_many_rows(hk):
    """131,072 rows whose gradients cancel: the sums stay within their roundings."""
    n, d = 131072, 64
    x = _rows(n, 1, d, 27, BF16)[:, 0]
    dy = _rand((n, d), 28)
    dy[1::2] = -dy[0::2]
    x[1::2] = x[0::2]
    _, saved = hk.layer_norm(x, save="x")
    r = hk.layer_norm_backward(dy, saved, want=("dweight", "dbias"))
    check_backward(r, dy, f64(x), saved.stats, None)
    again = hk.layer_norm_backward(dy, saved, want=("dweight", "dbias"))
    assert torch.equal(r["dweight"], again["dweight"]) and torch.equal(r["dbias"], again["dbias"])


# ------------------------------------------------------------- checkpoints

FMT_SHAPES = [(1, 1, 32), (1, 1, 128), (3, 2, 64), (301, 8, 96), (2500, 1, 128), (5, 1, 544), (7, 1, 1024), (4, 1, 2080), (3, 1, 4096),
              (5, 1, 5120), (2, 1, 8192)]


def _decoded(saved):
    """The rows that a checkpoint stands for, by the storage formats' own decoders."""
    lead, d = saved.rows.shape[:-1], saved.rows.shape[-1]
    codes = saved.rows.cpu().numpy().reshape(-1, d)
    if saved.fmt == "fp8":
        v = oracle.decode_e4m3(codes).astype(np.float64) * saved.scale.cpu().numpy().reshape(-1, 1).astype(np.float64)
    else:
        e = saved.scale.cpu().numpy().reshape(-1, d // 32).astype(np.int64) - 127
        v = oracle.decode_e4m3(codes).astype(np.float64) * np.repeat(np.ldexp(1.0, e), 32, axis=1)
    return v.reshape(*lead, d)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8"])
@pytest.mark.parametrize("shape", FMT_SHAPES)
def test_checkpoints(hk, shape, fmt):
    n, heads, d = shape
    say(f"checkpoint {shape} {fmt}")
    w, b = _rand(d, 30, FP32, 0.2, 1.0), _rand(d, 31)
    for dtype in (BF16, FP32):
        x = _rows(n, heads, d, 32 + d, dtype)
        if n > 2:
            x[2] = 0
            x[1, 0, 0] = 2.0 ** 7
        y, saved = hk.layer_norm(x, w, b, save=fmt)
        plain, kept = hk.layer_norm(x, w, b, save="x")
        assert torch.equal(y, plain) and torch.equal(saved.stats, kept.stats) and saved.fmt == fmt
        # the codes are the cache's own: each row a cache row
        codes, scale = hk.quantize(x.reshape(-1, d), fmt)
        assert torch.equal(saved.rows.reshape(-1, d), codes) and torch.equal(saved.scale.reshape(scale.shape), scale)
        x64 = _decoded(saved)
        for tg, tdx in ((BF16, None), (FP32, BF16), (FP32, None)):
            dy = _rand((n, heads, d), 33, tg, d ** -0.5)
            res = hk.layer_norm_backward(dy, saved, w, dx_dtype=tdx)
            check_backward(res, dy, x64, saved.stats, w, coded=fmt == "fp8")
        # rows off 16 bytes give the same
        off = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1:].view(x.shape)
        off.copy_(x)
        y2, s2 = hk.layer_norm(off, w, b, save=fmt)
        assert torch.equal(y2, y) and torch.equal(s2.rows, saved.rows) and torch.equal(s2.scale, saved.scale)
        goff = torch.empty(dy.numel() + 1, device="cuda")[1:].view(dy.shape)
        goff.copy_(dy)
        r2 = hk.layer_norm_backward(goff, s2, w)
        assert all(torch.equal(r2[k], res[k]) for k in res)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8"])
def test_a_checkpoint_s_gradient_is_near_the_input_s(hk, fmt):
    """E4M3 is off by 2^-4 of a value (and of the smallest by half its step); an MX block's scale leaves its largest value
    between 256 and 512 steps of which 448 can be held, so what lies above is off by up to 64 / 512 = 2^-3.  The difference of
    dx is bounded by the definition's own change and is not zero."""
    n, d = 64, 256
    x, w = _rows(n, 1, d, 40, BF16)[:, 0], _rand(d, 41, FP32, 0.2, 1.0)
    dy = _rand((n, d), 42)
    _, a = hk.layer_norm(x, w, save="x")
    _, c = hk.layer_norm(x, w, save=fmt)
    diff = f64(hk.layer_norm_backward(dy, c, w)["dx"]) - f64(hk.layer_norm_backward(dy, a, w)["dx"])
    st = f64(a.stats)
    v = _decoded(c)
    rel = 2.0 ** -4 if fmt == "fp8" else 2.0 ** -3
    assert (np.abs(v - f64(x)) <= rel * np.abs(f64(x)) + 2.0 ** -10 * np.abs(f64(x)).max(1, keepdims=True)).all()
    e = np.abs(v - f64(x)) * st[:, 1:]
    h, g = np.abs(f64(x) - st[:, :1]) * st[:, 1:], np.abs(f64(dy) * f64(w))
    bound = st[:, 1:] * (e * (g * (h + e)).mean(1, keepdims=True) + h * (g * e).mean(1, keepdims=True))
    assert (np.abs(diff) <= bound * 1.001 + 2.0 ** -16 * st[:, 1:] * (g + g.mean(1, keepdims=True) + h * (g * h).mean(1, keepdims=True))).all()
    assert np.abs(diff).max() > 0


def test_given_buffers_are_filled(hk):
    n, d = 37, 160
    x, w = _rows(n, 1, d, 43, BF16)[:, 0], _rand(d, 44)
    for fmt, st, shape in (("fp8", FP32, (n,)), ("mxfp8", torch.uint8, (n, d // 32))):
        y, ref = hk.layer_norm(x, w, save=fmt)
        # in larger buffers, whose other rows stay
        codes = torch.full((n + 2, d), 99, dtype=torch.uint8, device="cuda")
        scale = torch.full((n + 2,) + shape[1:], 3, dtype=st, device="cuda")
        stats = torch.full((n + 2, 2), 5.0, device="cuda")
        mine = hk.NormSaved(codes[1:-1], scale[1:-1], stats[1:-1], fmt)
        if fmt == "mxfp8":  # scales are 4-byte aligned
            mine = mine._replace(scale=torch.zeros((n, d // 32), dtype=st, device="cuda"))
        y2, got = hk.layer_norm(x, w, save=mine)
        assert got is mine and torch.equal(y2, y) and torch.equal(mine.rows, ref.rows) and torch.equal(mine.scale, ref.scale)
        assert torch.equal(mine.stats, ref.stats)
        assert bool((codes[[0, -1]] == 99).all()) and bool((stats[[0, -1]] == 5.0).all())
        if fmt == "fp8":
            assert bool((scale[[0, -1]] == 3).all())
