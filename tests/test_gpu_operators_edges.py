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
