"""FP8 cache rows that hold an infinity: the row's scale is infinite and all of it reads as NaN, so that no number of such a row passes for
one; the other rows are as without it."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rows(n, heads, d, dtype):
    x = torch.randn((n, heads, d), generator=torch.Generator().manual_seed(n + d)).to(dtype)
    x[:, :, ::5] = 0  # zeros too must not read as numbers
    bad = x.clone()
    bad[1, 0, 0], bad[4, heads - 1, d - 1], bad[n - 1, 0, 7] = INF, -INF, INF
    bad[n - 2], bad[n - 2, 0, 3] = 0, INF  # nothing else in the row
    return x.cuda(), bad.cuda(), [1, 4, n - 2, n - 1]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,heads,d", [(9, 1, 32), (70, 1, 128), (33, 4, 64), (7, 1, 1056), (8, 1, 8192)])
def test_rows_with_an_infinity_read_as_nan(hk, n, heads, d, dtype):
    say(f"fp8 infinity {n} x {heads} x {d} {dtype}")
    x, bad, rows = _rows(n, heads, d, dtype)
    keep = [i for i in range(n) if i not in rows]
    if heads == 1:
        x, bad = x[:, 0], bad[:, 0]
    plan = hk.Rotary(32)
    for kw in ({}, dict(rotary=plan, q_start=3)):
        codes, scale = hk.quantize(x, "fp8", **kw)
        c, s = hk.quantize(bad, "fp8", **kw)
        assert torch.isinf(s[rows]).all()
        assert torch.equal(c[keep], codes[keep]) and torch.equal(s[keep], scale[keep])
        for out in (BF16, FP32):
            got = hk.cache_read(c, s, fmt="fp8", dtype=out)
            assert torch.isnan(got[rows]).all() and torch.isfinite(got[keep]).all()
    # a norm's checkpoint is the same rows, each (token, head) by itself
    _, saved = hk.layer_norm(bad, save="fp8")
    flat, fs = hk.quantize(bad.reshape(-1, d), "fp8")
    assert torch.equal(saved.rows.reshape(-1, d), flat) and torch.equal(saved.scale.reshape(-1), fs)
    assert int(torch.isinf(fs).sum()) == 4


def test_the_largest_finite_rows(hk):
    """Next to an infinity: the largest numbers, and the smallest ones, keep the quotient's scale."""
    top = torch.tensor([torch.finfo(FP32).max, 2.0 ** 127, 448.0, 447.99997, 2.0 ** -117, 2.0 ** -126, 2.0 ** -149, 0.0])
    x = torch.zeros((8, 32))
    x[:, 5] = top
    codes, scale = hk.quantize(x.cuda(), "fp8")
    want = torch.where(top > 0, (top.double() / 448).float().clamp_min(2.0 ** -126), 1.0)
    assert torch.equal(scale.cpu(), want)
