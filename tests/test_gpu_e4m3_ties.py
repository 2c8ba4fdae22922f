"""FP8 rows next to the ties of E4M3: codes and scales against the exact quotient's, bit for bit.  The 64-bit quotient of two
24-bit numbers does not round onto a number of 5 bits unless it is one, so a tie is seen as one there."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _definition(x):
    top = x.float().abs().amax(1, keepdim=True)
    scale = (top.double() / 448).float()
    scale = torch.where(top > 0, scale.clamp_min(2.0 ** -126), torch.ones_like(scale))
    q = x.double() / scale.double()
    a = q.abs().clamp_max(448.0)
    # the power of two below, by its bits, over eight steps
    step = (a.clamp_min(2.0 ** -6).view(torch.int64) & (0x7ff << 52)).view(torch.float64) / 8
    v = torch.copysign(torch.round(a / step) * step, q)
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8), scale[:, 0]


def _rows(kind, n, g):
    def ints(lo, hi):
        return torch.randint(lo, hi, (n, 128), generator=g, device="cuda").double()
    if kind == "whole numbers":  # with 448 among them every odd half of a step is met
        x = ints(-448, 449)
        x[:, 0] = 448
        return x
    if kind == "sevenths":  # the largest a multiple of 7: ties of bf16 rows
        x = ints(-256, 257)
        x[:, 5] = 7 * torch.randint(19, 37, (n,), generator=g, device="cuda").double()
        return x
    if kind == "small":  # down to codes below the normal ones and to zeros
        return torch.randn((n, 128), generator=g, device="cuda").double() * torch.exp(-16 * torch.rand((n, 128), generator=g, device="cuda").double())
    return torch.randn((n, 128), generator=g, device="cuda").double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["whole numbers", "sevenths", "small", "normal"])
def test_codes_next_to_ties(hk, kind, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    for scale in (0, -126, -118, -60, -1, 1, 37, 110):
        say(f"ties: {kind} {dtype} 2^{scale}")
        x = (_rows(kind, 6000, g) * 2.0 ** scale).to(dtype)
        x[17] = 0
        codes, s = hk.quantize(x, "fp8")
        want, ws = _definition(x)
        assert torch.equal(s, ws)
        assert torch.equal(codes, want), (codes != want).nonzero()[0]


def test_scales_next_to_a_power_of_two(hk):
    """fp32 rows whose scale has every kind of significand, elements at every tie of it and one step beside."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n = 20000
    top = (1 + torch.rand(n, 1, generator=g, device="cuda").double()) * 448
    x = torch.zeros((n, 128), device="cuda")
    scale = (top.float().double() / 448).float().double()
    ties = torch.cat([(2 * torch.arange(8, device="cuda") + 17) / 32 * 2.0 ** e for e in range(-6, 9)])[:-1].double()  # above 448 none
    at = ties[torch.randint(0, len(ties) - 1, (n, 128), generator=g, device="cuda")] * scale
    x = at.float()  # the tie itself or next to it
    bits = x.view(torch.int32) + torch.randint(-1, 2, (n, 128), generator=g, device="cuda", dtype=torch.int32)
    x = bits.view(torch.float32).clamp_max(448.0)
    x[:, 0] = top[:, 0].float()
    codes, s = hk.quantize(x, "fp8")
    want, ws = _definition(x)
    assert torch.equal(s, ws) and torch.equal(codes, want)
