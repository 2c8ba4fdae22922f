"""Layer norm of rows where its arithmetic is at its limits, against the fp64 definition: constant rows of every size, whose mean
times rstd may pass fp32, on widths that leave some of a row's places empty.  u = 2^-24; tolerances of the two passes are those that
test_gpu_layer_norm derives."""
import numpy as np
import pytest
import torch

from gpu_util import say
from test_gpu_layer_norm import check_backward

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
