"""Rotary positions against the fp64 definition (oracle.operators).

Tolerance of an fp32 result, per rotated element y = g (a c - b s): the cosine
and sine carry their argument's rounding (2^-26 of a turn: 2 pi 2^-26 < 2^-23.3)
and at most 2 ulp of the function (2^-23 below 1), the gain's rounding and
product 2 * 2^-24, and the two products and their sum at most 3 * 2^-24 of
|a| + |b|: together below 2^-21 g (|a| + |b|).  A bf16 result adds half a
bf16 step (2^-8 of the value).  Elements outside the rotated part are copied: exact in
their own type, half a step into a shorter one."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _check(y, x, pos, plan, backward=False):
    """y against the definition on x (both tensors [n][heads][d])."""
    x64 = x.double().cpu().numpy()
    pos = np.asarray(pos)
    f = plan.freq.cpu().numpy()
    ref = op.rotary(x64, pos, f, first=plan.first, layout=plan.layout, gain=plan.gain, backward=backward)
    half = plan.dim // 2
    i = np.arange(half)
    ia, ib = ((plan.first + i, plan.first + half + i) if plan.layout == "half"
              else (plan.first + 2 * i, plan.first + 2 * i + 1))
    tol = np.zeros_like(ref)
    both = 2.0 ** -21 * plan.gain * (np.abs(x64[..., ia]) + np.abs(x64[..., ib]))
    tol[..., ia] = both
    tol[..., ib] = both
    if y.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    bad = err > tol
    assert not bad.any(), (np.argwhere(bad)[0], err[bad][0], tol[bad][0])
    if y.dtype == x.dtype:  # what is not rotated is copied
        keep = np.ones(x.shape[-1], bool)
        keep[ia] = keep[ib] = False
        assert np.array_equal(y.double().cpu().numpy()[..., keep], x64[..., keep])


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


SHAPES = [  # n, heads, d, dim, first
    (1, 64, 128, 64, 0), (1, 1, 64, 64, 0), (7, 3, 128, 128, 0), (33, 1, 128, 64, 64), (5, 40, 192, 64, 128),
    (300, 8, 64, 32, 16), (2, 129, 64, 16, 48), (1000, 1, 576, 64, 512), (3, 2, 4096, 1024, 2048),
    (3, 5, 100, 36, 7), (17, 2, 6, 2, 3), (4, 1, 2, 2, 0), (9, 3, 1000, 600, 1),
]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotary_matches_the_definition(hk, shape, layout):
    n, heads, d, dim, first = shape
    say(f"rotary: {shape} {layout}")
    plan = hk.Rotary(dim, first=first, layout=layout, scaling="yarn", factor=4.0, original=4096)
    for tin, tout in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                      (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        x = _rand((n, heads, d), tin, n + d)
        pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(d)).int()
        for back in (False, True):
            y = hk.rotary(x, plan, q_pos=pos.cuda(), backward=back, out_dtype=tout)
            assert y.dtype == tout
            _check(y, x, pos.numpy(), plan, back)


def test_far_and_negative_positions(hk):
    """At the ends of int32 the angle keeps its precision (64-bit reduction)."""
    plan = hk.Rotary(64)
    pos = np.array([0, 1, (1 << 24) + 1, (1 << 31) - 1, -1, -(1 << 31)], dtype=np.int32)
    x = _rand((6, 2, 64), torch.float32, 5)
    y = hk.rotary(x, plan, q_pos=torch.from_numpy(pos).cuda())
    _check(y, x, pos.astype(np.int64), plan)
    y = hk.rotary(x[:4], plan, q_start=(1 << 31) - 4)
    _check(y, x[:4], np.arange((1 << 31) - 4, 1 << 31), plan)


def test_positions_by_start_equal_explicit_ones(hk):
    plan = hk.Rotary(64, scaling="linear", factor=2.0)
    x = _rand((1025, 2, 64), torch.bfloat16, 6)
    a = hk.rotary(x, plan, q_start=77)
    b = hk.rotary(x, plan, q_pos=torch.arange(77, 77 + 1025, dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_alignment_and_in_place(hk, layout, dtype):
    plan = hk.Rotary(32, first=16, layout=layout)
    n, h, d = 19, 3, 64
    pos = torch.arange(5, 5 + n, dtype=torch.int32)
    base = _rand((n, h, d), dtype, 8)
    want = hk.rotary(base, plan, q_pos=pos.cuda())
    _check(want, base, pos.numpy(), plan)
    # a slice of a fused projection, heads before tokens, one element off 16-byte alignment
    fused = _rand((n, h, 3 * d), dtype, 9)
    fused[..., d:2 * d] = base
    swapped = base.transpose(0, 1).contiguous().transpose(0, 1)
    off = torch.empty(n * h * d + 1, dtype=dtype, device="cuda")[1:].view(n, h, d)
    off.copy_(base)
    for x in (fused[..., d:2 * d], swapped, off):
        assert torch.equal(hk.rotary(x, plan, q_pos=pos.cuda()), want)
        out = torch.empty_like(off)
        hk.rotary(x, plan, q_pos=pos.cuda(), out=out)
        assert torch.equal(out, want)
    # into a strided destination, whose other elements stay
    wide = torch.full((n, h, d + 7), 3.0, dtype=dtype, device="cuda")
    hk.rotary(base, plan, q_pos=pos.cuda(), out=wide[..., 7:])
    assert torch.equal(wide[..., 7:], want) and bool((wide[..., :7] == 3.0).all())
    # in place, also within the fused rows
    x = fused[..., d:2 * d]
    before = fused.clone()
    hk.rotary(x, plan, q_pos=pos.cuda(), out=x)
    assert torch.equal(x, want)
    assert torch.equal(fused[..., :d], before[..., :d]) and torch.equal(fused[..., 2 * d:], before[..., 2 * d:])
    # x broadcast over heads
    one = base[:, :1]
    y = hk.rotary(one.expand(n, h, d), plan, q_pos=pos.cuda())
    assert torch.equal(y, hk.rotary(one.contiguous(), plan, q_pos=pos.cuda()).expand(n, h, d))
    # two axes
    assert torch.equal(hk.rotary(base[:, 1], plan, q_pos=pos.cuda()), want[:, 1])
    # nothing
    assert hk.rotary(base[:0], plan).shape == (0, h, d)
    with pytest.raises(hk.HytopkError):  # rows of the result that share elements
        hk.rotary(base, plan, out=torch.empty_like(base[:1]).expand(n, h, d))
    with pytest.raises(hk.HytopkError):
        hk.rotary(fused[..., :d], plan, out=fused[..., 8:d + 8])


def test_backward_is_the_gradient(hk):
    """<g, R x> = <R^T g, x> for the kernel's own results, and the definition's gradient."""
    for layout in ("half", "interleaved"):
        plan = hk.Rotary(64, first=32, layout=layout, scaling="yarn", factor=8.0, original=1024)
        x, g = _rand((50, 4, 128), torch.float32, 10), _rand((50, 4, 128), torch.float32, 11)
        y, dx = hk.rotary(x, plan, q_start=900), hk.rotary(g, plan, q_start=900, backward=True)
        _check(dx, g, np.arange(900, 950), plan, True)
        a = (g.double() * y.double()).sum().item()
        b = (dx.double() * x.double()).sum().item()
        # each side's results are off by at most 2^-21 g (|a| + |b|) an element
        s = 2.0 ** -21 * plan.gain * 2 * 2 * (g.double().norm() * x.double().norm()).item()
        assert abs(a - b) <= s


def test_rotary_in_a_graph_and_on_another_stream(hk):
    plan = hk.Rotary(64)
    x = _rand((40, 8, 64), torch.bfloat16, 12)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hk.rotary(x, plan, q_pos=pos, out=y)
    side.synchronize()
    want = y.clone()
    assert torch.equal(hk.rotary(x, plan, q_pos=pos), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hk.rotary(x, plan, q_pos=pos, out=y)
    for rep in range(3):
        x.copy_(_rand((40, 8, 64), torch.bfloat16, 20 + rep))
        pos.add_(1000)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, hk.rotary(x, plan, q_pos=pos))
