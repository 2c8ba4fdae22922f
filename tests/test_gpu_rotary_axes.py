"""Rotary positions of several axes against the fp64 definition (oracle.operators), in hk.rotary, hk.cache_write
and hk.quantize.  The tolerance of a rotated element is test_gpu_rotary.py's: 2^-21 gain (|a| + |b|), and half a step of a bf16 result.
Codes are compared with those of the rotation's own fp32 result."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _positions(n, axes, seed, top=1 << 20):
    return torch.randint(0, top, (n, axes), generator=torch.Generator().manual_seed(seed)).int()


def _check(y, x, pos, plan, axis, backward=False):
    x64, f = x.double().cpu().numpy(), plan.freq.cpu().numpy()
    ref = op.rotary(x64, np.asarray(pos).astype(np.int64), f, first=plan.first, layout=plan.layout, gain=plan.gain,
                    backward=backward, axis=axis)
    i, half = np.arange(plan.dim // 2), plan.dim // 2
    ia, ib = ((plan.first + i, plan.first + half + i) if plan.layout == "half"
              else (plan.first + 2 * i, plan.first + 2 * i + 1))
    tol = np.zeros_like(ref)
    tol[..., ia] = tol[..., ib] = 2.0 ** -21 * plan.gain * (np.abs(x64[..., ia]) + np.abs(x64[..., ib]))
    if y.dtype == BF16:
        tol += 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    bad = err > tol
    assert not bad.any(), (np.argwhere(bad)[0], err[bad][0], tol[bad][0])


PLANS = [  # n, heads, d, dim, first, sections, cycle, restart
    (1, 64, 128, 128, 0, (16, 24, 24), False, False), (300, 4, 128, 64, 64, (12, 10, 10), True, False), (33, 24, 64, 64, 0, (16, 16), False, True),
    (7, 1, 576, 64, 512, (11, 11, 10), True, True), (1000, 2, 64, 32, 16, (4, 4, 4, 4), True, False), (5, 3, 100, 36, 7, (6, 6, 6), False, False),
    (3, 2, 17, 6, 3, (1, 1, 1), False, True), (4, 2, 4096, 1024, 2048, (170, 171, 171), False, False), (9, 1, 64, 32, 0, (1,) * 16, True, False),
    (2, 5, 32, 10, 2, (3, 2), True, False),
]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", PLANS)
def test_matches_the_definition(hk, case, layout):
    n, heads, d, dim, first, sections, cycle, restart = case
    say(f"axes {case} {layout}")
    plan = hk.Rotary(dim, first=first, layout=layout, sections=sections, cycle=cycle, restart=restart, scaling="yarn", factor=4.0,
                     original=4096)
    axis = plan.axis.cpu().numpy()
    assert [int((axis == a).sum()) for a in range(len(sections))] == list(sections)
    pos = _positions(n, len(sections), d)
    for tin, tout in ((BF16, BF16), (FP32, FP32), (FP32, BF16), (BF16, FP32)):
        x = _rand((n, heads, d), tin, n + d)
        for back in (False, True):
            _check(hk.rotary(x, plan, q_pos=pos.cuda(), backward=back, out_dtype=tout), x, pos, plan, axis, back)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_equal_positions_are_the_one_axis_rotation(hk, layout):
    """A text token's positions are the same on every axis; rows of any alignment, one and several axes: the same bits."""
    n, h, d = 50, 3, 128
    one = hk.Rotary(64, first=32, layout=layout, scaling="ntk", factor=4.0)
    x = _rand((n, h, d), BF16, 1)
    pos = _positions(n, 1, 2)
    want = hk.rotary(x, one, q_pos=pos[:, 0].contiguous().cuda())
    off = torch.empty(x.numel() + 1, dtype=BF16, device="cuda")[1:].view(x.shape)
    off.copy_(x)
    for cycle in (False, True):
        many = hk.Rotary(64, first=32, layout=layout, scaling="ntk", factor=4.0, sections=(12, 10, 10), cycle=cycle)
        p3 = pos.expand(n, 3).contiguous().cuda()
        for v in (x, off):
            assert torch.equal(hk.rotary(v, many, q_pos=p3), want)
        # without positions a token sits at q_start + i on every axis
        assert torch.equal(hk.rotary(x, many, q_start=99), hk.rotary(x, one, q_start=99))
    single = hk.Rotary(64, first=32, layout=layout, scaling="ntk", factor=4.0, sections=(32,))
    assert single.axes == 1 and single.axis is None
    assert torch.equal(hk.rotary(x, single, q_pos=pos[:, 0].contiguous().cuda()), want)


def test_one_axis_alone_turns(hk):
    """Positions of 0 on the other axes leave their pairs as they are."""
    plan = hk.Rotary(64, layout="half", sections=(12, 10, 10))
    axis = plan.axis.cpu().numpy()
    x = _rand((20, 2, 64), FP32, 3)
    for a in range(3):
        pos = torch.zeros((20, 3), dtype=torch.int32)
        pos[:, a] = torch.arange(1, 21)
        y = hk.rotary(x, plan, q_pos=pos.cuda())
        still = np.concatenate([axis != a, axis != a])
        assert torch.equal(y.cpu()[..., still], x.cpu()[..., still])
        assert not bool((y.cpu()[..., ~still] == x.cpu()[..., ~still]).all())


def test_far_and_negative_positions(hk):
    plan = hk.Rotary(64, sections=(16, 16), cycle=True)
    ends = [0, 1, (1 << 31) - 1, -1, -(1 << 31), (1 << 24) + 1]
    pos = torch.tensor([[a, b] for a in ends for b in ends], dtype=torch.int32)
    x = _rand((len(pos), 2, 64), FP32, 5)
    _check(hk.rotary(x, plan, q_pos=pos.cuda()), x, pos, plan, plan.axis.cpu().numpy())


def test_the_transpose_is_the_adjoint(hk):
    """<R x, y> = <x, R^T y> over the whole batch: both sums of products of fp32 results, each off by 2^-21 (|a| + |b|)."""
    plan = hk.Rotary(64, layout="interleaved", sections=(12, 10, 10), cycle=True, scaling="yarn", factor=8.0, original=1024)
    x, y = _rand((40, 4, 64), FP32, 6), _rand((40, 4, 64), FP32, 7)
    pos = _positions(40, 3, 8).cuda()
    a = (hk.rotary(x, plan, q_pos=pos).double() * y.double()).sum()
    b = (x.double() * hk.rotary(y, plan, q_pos=pos, backward=True).double()).sum()
    assert abs(float(a - b)) <= 2 * 2.0 ** -21 * plan.gain * 4 * float((x.abs().double() * y.abs().double()).sum() + 40 * 4 * 64)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_written_into_a_cache(hk, fmt, layout):
    """A write rotates as hk.rotary does, in fp32 and not rounded in between."""
    for n, heads, d, dim, first, sections in ((70, 1, 128, 64, 0, (8, 12, 12)), (9, 64, 128, 128, 0, (16, 24, 24)), (5, 3, 96, 32, 64, (8, 8)),
                                              (6, 2, 64, 20, 3, (4, 3, 3))):
        plan = hk.Rotary(dim, first=first, layout=layout, sections=sections)
        x = _rand((n, heads, d), BF16, 9)
        pos = _positions(n, len(sections), 10).cuda()
        turned = hk.rotary(x, plan, q_pos=pos, out_dtype=FP32)
        want, ws = hk.quantize(turned, fmt)
        got, gs = hk.quantize(x, fmt, rotary=plan, q_pos=pos)
        assert torch.equal(got, want) and (ws is None or torch.equal(gs, ws))
        # by slot, among other rows
        slots = torch.randperm(3 * n, generator=torch.Generator().manual_seed(11))[:n].int().cuda()
        codes = torch.zeros((3 * n,) + got.shape[1:], dtype=got.dtype, device="cuda")
        scale = None if gs is None else torch.zeros((3 * n,) + gs.shape[1:], dtype=gs.dtype, device="cuda")
        hk.cache_write(x, codes, scale, fmt=fmt, slots=slots, rotary=plan, q_pos=pos)
        assert torch.equal(codes[slots.long()], want)
        rest = torch.ones(3 * n, dtype=torch.bool, device="cuda")
        rest[slots.long()] = False
        assert not codes[rest].any()


def test_an_axis_that_does_not_exist_is_the_last(hk):
    plan = hk.Rotary(32, sections=(8, 8))
    x, pos = _rand((10, 2, 32), FP32, 12), _positions(10, 2, 13).cuda()
    want = hk.rotary(x, plan, q_pos=pos)
    plan.axis[8:] = torch.tensor([2, -1, 1 << 30, -(1 << 31), 1, 7, 2, 1], dtype=torch.int32, device="cuda")
    assert torch.equal(hk.rotary(x, plan, q_pos=pos), want)


def test_many_tokens_and_graphs(hk):
    """More tokens than one tile, recorded and replayed with new positions."""
    plan = hk.Rotary(128, sections=(16, 24, 24))
    x = _rand((5003, 2, 128), BF16, 14)
    pos = _positions(5003, 3, 15).cuda()
    out = torch.empty_like(x)
    hk.rotary(x, plan, q_pos=pos, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hk.rotary(x, plan, q_pos=pos, out=out)
    for seed in range(3):
        pos.copy_(_positions(5003, 3, 20 + seed))
        want = hk.rotary(x, plan, q_pos=pos)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    _check(out, x, pos.cpu(), plan, plan.axis.cpu().numpy())
