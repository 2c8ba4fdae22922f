"""Plans of several axes without positions: a token sits at q_start + i on every axis, near and far, in every kernel that rotates."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 31) - 4096])
def test_tokens_without_positions(hk, layout, start):
    say(f"axes without positions, {layout}, from {start}")
    one, many = hk.Rotary(64, first=32, layout=layout), hk.Rotary(64, first=32, layout=layout, sections=(12, 10, 10), cycle=True)
    g = torch.Generator().manual_seed(1)
    for n, heads in ((1, 1), (2500, 1), (300, 5)):
        x = torch.randn((n, heads, 128), generator=g).bfloat16().cuda()
        off = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        off.copy_(x)
        for rows in (x, off, x.float()):
            want = hk.rotary(rows, one, q_start=start)
            assert torch.equal(hk.rotary(rows, many, q_start=start), want)
            pos = (start + torch.arange(n)).int()[:, None].expand(n, 3).contiguous().cuda()
            assert torch.equal(hk.rotary(rows, many, q_pos=pos), want)
            for fmt in ("bf16", "fp8", "mxfp8", "mxfp4"):
                a, b = hk.quantize(rows, fmt, rotary=one, q_start=start), hk.quantize(rows, fmt, rotary=many, q_start=start)
                assert torch.equal(a[0], b[0]) and (a[1] is None or torch.equal(a[1], b[1]))
