"""The quantised cache: rows written in the four storage formats and read back.

Without a rotation the codes and scales are compared bit for bit with the
generator's quantisers (rounding of the exact quotient), and what is read back
with the codes' exact values.  With one, the values read back lie within half a
step of the format of the fp64 rotation, plus the rotation's own error (2^-21 gain (|a| + |b|),
derived in test_gpu_rotary.py)."""
import numpy as np
import pytest
import torch

import datagen
import oracle
from gpu_util import say
from oracle import operators as op

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "fp8", "mxfp8", "mxfp4"]


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _rows(n, heads, d, seed, dtype=torch.bfloat16):
    """Rows of very different sizes, some of them zero, with signed zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, heads, d)) * np.exp2(rng.integers(-20, 20, size=(n, 1, 1)))
    x[rng.random((n, heads, d)) < 0.05] = -0.0
    if n > 2:
        x[n // 2] = 0.0
    if d >= 64:
        x[0, 0, 32:64] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _reference(x32: np.ndarray, fmt: str):
    if fmt == "bf16":
        return datagen.f32_to_bf16_bits(x32), None
    if fmt == "fp8":
        return datagen.quantize_e4m3_per_row(x32)
    return datagen.quantize_mx(x32, fmt)


def _codes(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def _values(codes: np.ndarray, scale, fmt: str) -> np.ndarray:
    if fmt == "bf16":
        return oracle.decode_bf16(codes)
    if fmt == "fp8":
        v = oracle.decode_e4m3(codes)
        return v * scale.astype(np.float64).reshape((-1,) + (1,) * (v.ndim - 1))
    return oracle.decode_mx(codes, scale, fmt)


def _empty(fmt, L, heads, d, fill=0x55):
    codes = torch.full((L, heads, d // 2 if fmt == "mxfp4" else d), fill, dtype=torch.uint8, device="cuda")
    if fmt == "bf16":
        codes = torch.full((L, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    scale = {"bf16": None, "fp8": torch.full((L,), 9.0, device="cuda")}.get(
        fmt, torch.full((L, heads, d // 32), 99, dtype=torch.uint8, device="cuda"))
    return codes, scale


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 1, 128), (5, 1, 32), (64, 1, 128), (33, 1, 96), (7, 64, 128), (3, 3, 160),
                                   (20, 2, 64), (2, 1, 8192), (9, 5, 320), (1500, 1, 128), (6, 1, 576), (5, 64, 96),
                                   (3, 40, 160), (2, 13, 576), (9000, 4, 32), (70, 32, 128)])
def test_codes_equal_the_reference_quantiser(hk, fmt, shape):
    say(f"cache: {fmt} {shape}")
    n, heads, d = shape
    for dtype in (torch.bfloat16, torch.float32):
        x = _rows(n, heads, d, n + d, dtype)
        codes, scale = hk.quantize(x.cuda(), fmt)
        rc, rs = _reference(x.float().numpy(), fmt)
        if rs is not None:
            assert np.array_equal(scale.cpu().numpy(), rs)
        assert np.array_equal(_codes(codes), rc)
        exact = _values(rc, rs, fmt)
        f32 = hk.cache_read(codes, scale, fmt=fmt, dtype=torch.float32)
        assert np.array_equal(f32.cpu().numpy(), exact.astype(np.float32))
        b16 = hk.cache_read(codes, scale, fmt=fmt)
        assert np.array_equal(_codes(b16), datagen.f32_to_bf16_bits(exact.astype(np.float32)))


def test_every_code_is_read_and_ties_round_to_even(hk):
    """All 256 E4M3 codes and E2M1 pairs decode to their values; every midpoint
    between neighbouring magnitudes rounds to the even code."""
    codes = torch.arange(256, dtype=torch.uint8).view(2, 128).cuda()
    one = torch.ones(2, device="cuda")
    v = hk.cache_read(codes, one, fmt="fp8", dtype=torch.float32).cpu().numpy()
    ref = (np.arange(256) & 127)
    nan = ref == 127
    assert np.isnan(v.reshape(-1)[nan]).all()
    assert np.array_equal(v.reshape(-1)[~nan], oracle.decode_e4m3(np.arange(256, dtype=np.uint8)[~nan]))
    sc = torch.full((1, 4), 127, dtype=torch.uint8, device="cuda")
    for part in codes.cpu().numpy().reshape(4, 64):
        c = torch.from_numpy(part.copy()).view(1, 64).cuda()
        v = hk.cache_read(c, sc, fmt="mxfp4", dtype=torch.float32).cpu().numpy()
        assert np.array_equal(v, oracle.decode_mx(part.reshape(1, 64), sc.cpu().numpy(), "mxfp4"))
    # scale bytes at their ends: 2^-127 (subnormal in fp32), 2^127, and NaN
    sc = torch.tensor([[0, 254, 255, 127]], dtype=torch.uint8, device="cuda")
    c = torch.full((1, 64), 0x31, dtype=torch.uint8, device="cuda")  # 0.5, 1.5
    v = hk.cache_read(c, sc, fmt="mxfp4", dtype=torch.float32).cpu().numpy()[0]
    assert v[0] == np.float32(2.0 ** -128) and v[33] == np.float32(1.5 * 2.0 ** 127)
    assert np.isnan(v[64:96]).all() and v[97] == 1.5
    # midpoints, and the fp32 neighbours on both sides of them, under a scale of 1 (amax 448)
    t = oracle.decode_e4m3(np.arange(127, dtype=np.uint8))
    mid = ((t[1:] + t[:-1]) / 2).astype(np.float32)
    x = np.concatenate([[448.0], mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), -mid])
    x = np.resize(np.concatenate([x, np.zeros(-len(x) % 32)]), (-(-len(x) // 32)) * 32).astype(np.float32)
    for scale in (1.0, 0.37, 3.0):
        row = torch.from_numpy((x * np.float32(scale))[None, :]).cuda()
        codes, sc = hk.quantize(row, "fp8")
        rc, rs = datagen.quantize_e4m3_per_row(row.cpu().numpy())
        assert np.array_equal(sc.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
    b = np.zeros((2, 32), np.float32)
    b[0, :15] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5]
    b[1, :8] = [7.9, 6.9, -7.9, 4.999, 5.001, .2499, .2501, 4]
    codes, sc = hk.quantize(torch.from_numpy(b).cuda(), "mxfp4")
    rc, rs = datagen.quantize_mx(b, "mxfp4")
    assert np.array_equal(sc.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)


def test_scales_at_the_ends_of_the_range(hk):
    """Rows of subnormals and of the largest finite values."""
    tiny = np.float32(2.0 ** -149)
    x = np.zeros((4, 32), np.float32)
    x[0, 0] = tiny
    x[1, :2] = [3.0e38, -1.0e30]
    x[2, :2] = [2.0 ** -126, 2.0 ** -140]
    x[3, 5] = -1.0e-30
    codes, scale = hk.quantize(torch.from_numpy(x).cuda(), "fp8")
    s = scale.cpu().numpy()
    # amax / 448 would be subnormal or 0 in rows 0 and 2: the smallest normal scale instead
    want = np.maximum(np.abs(x).max(1) / np.float32(448), np.float32(2.0 ** -126))
    assert np.array_equal(s, want)
    q = x.astype(np.float64) / want[:, None].astype(np.float64)
    assert np.array_equal(codes.cpu().numpy(), datagen.f32_to_e4m3(q))
    for fmt in ("mxfp8", "mxfp4"):
        codes, scale = hk.quantize(torch.from_numpy(x).cuda(), fmt)
        rc, rs = datagen.quantize_mx(x, fmt)
        assert np.array_equal(scale.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [5, 40, 1024, 1025, 3000])
def test_slots_padding_repeats_and_other_rows(hk, fmt, n):
    """Rows go to their slots; padding and slots outside the cache write nothing; of
    repeated slots the last row is kept; every other cache row stays."""
    L, heads, d = 4000, 1 if n > 100 else 2, 64
    rng = np.random.default_rng(n)
    slots = rng.permutation(L)[:n].astype(np.int32)
    slots[rng.random(n) < 0.3] = slots[0]                    # many rows of one slot
    slots[rng.random(n) < 0.1] = -1
    slots[rng.random(n) < 0.05] = L
    slots[rng.random(n) < 0.05] = np.iinfo(np.int32).min
    x = _rows(n, heads, d, 3)
    codes, scale = _empty(fmt, L, heads, d)
    before = codes.clone(), None if scale is None else scale.clone()
    hk.cache_write(x.cuda(), codes, scale, fmt=fmt, slots=torch.from_numpy(slots).cuda())
    rc, rs = _reference(x.float().numpy(), fmt)
    want_c, want_s = _codes(before[0]).copy(), None if scale is None else before[1].cpu().numpy()
    for i in range(n):
        if 0 <= slots[i] < L:
            want_c[slots[i]] = rc[i]
            if scale is not None:
                want_s[slots[i]] = rs[i]
    assert np.array_equal(_codes(codes), want_c)
    if scale is not None:
        assert np.array_equal(scale.cpu().numpy(), want_s)
    # read back by slot: padding reads as zeros
    v = hk.cache_read(codes, scale, fmt=fmt, slots=torch.from_numpy(slots).cuda(), dtype=torch.float32)
    ok = (slots >= 0) & (slots < L)
    ref = np.zeros((n, heads, d), np.float32)
    ref[ok] = _values(want_c, want_s, fmt).astype(np.float32)[slots[ok]]
    assert np.array_equal(v.cpu().numpy(), ref)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_by_start_and_both_ends_of_the_cache(hk, fmt):
    codes, scale = _empty(fmt, 300, 1, 128)
    x = _rows(300, 1, 128, 4)
    for a, b in ((0, 1), (1, 130), (130, 299), (299, 300)):
        hk.cache_write(x[a:b].cuda(), codes, scale, fmt=fmt, start=a)
    rc, rs = _reference(x.float().numpy(), fmt)
    assert np.array_equal(_codes(codes), rc)
    full = hk.cache_read(codes, scale, fmt=fmt)
    assert torch.equal(hk.cache_read(codes, scale, fmt=fmt, start=299), full[299:])
    assert torch.equal(hk.cache_read(codes, scale, fmt=fmt, start=3, count=200), full[3:203])
    with pytest.raises(hk.HytopkError):
        hk.cache_write(x[:2].cuda(), codes, scale, fmt=fmt, start=299)
    with pytest.raises(hk.HytopkError):
        hk.cache_read(codes, scale, fmt=fmt, start=1, count=300)
    assert hk.cache_read(codes, scale, fmt=fmt, count=0).shape == (0, 1, 128)
    hk.cache_write(x[:0].cuda(), codes, scale, fmt=fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", [(50, 1, 128, 64, 0), (9, 64, 128, 128, 0), (11, 2, 96, 36, 3), (300, 1, 64, 32, 32),
                                   (4, 1, 2048, 1024, 512), (11, 2, 96, 64, 16), (5, 64, 96, 64, 32), (3, 40, 160, 64, 0),
                                   (70, 32, 128, 64, 64), (2, 32, 256, 256, 0), (4100, 4, 32, 16, 0), (9, 3, 256, 16, 240)])
def test_rotated_rows(hk, fmt, layout, shape):
    n, heads, d, dim, first = shape
    say(f"cache: {fmt} rotated {shape} {layout}")
    plan = hk.Rotary(dim, first=first, layout=layout, scaling="yarn", factor=4.0, original=2048)
    x = _rows(n, heads, d, 5)
    pos = np.random.default_rng(6).integers(0, 1 << 20, n).astype(np.int32)
    codes, scale = hk.quantize(x.cuda(), fmt, rotary=plan, q_pos=torch.from_numpy(pos).cuda())
    x64 = x.double().numpy()
    y = op.rotary(x64, pos, plan.freq.cpu().numpy(), first=first, layout=layout, gain=plan.gain)
    half = dim // 2
    i = np.arange(half)
    ia, ib = (first + i, first + half + i) if layout == "half" else (first + 2 * i, first + 2 * i + 1)
    rot = np.zeros_like(y)
    rot[..., ia] = rot[..., ib] = 2.0 ** -21 * plan.gain * (np.abs(x64[..., ia]) + np.abs(x64[..., ib]))
    v = _values(_codes(codes), None if scale is None else scale.cpu().numpy(), fmt)
    a = np.abs(y)
    if fmt == "bf16":
        tol = 2.0 ** -8 * (a + rot) + rot
    elif fmt == "fp8":
        # scale: that of the row's largest value, to that value's error and a rounding
        top, err = a.max((1, 2)), rot.max((1, 2))
        s = scale.cpu().numpy().astype(np.float64)
        ref = np.where(top > 0, np.maximum(top / 448, 2.0 ** -126), 1.0)
        assert np.all(np.abs(s - ref) <= 2.0 ** -23 * ref + err / 448)
        tol = np.maximum(2.0 ** -4 * (a + rot), 2.0 ** -10 * s[:, None, None]) + rot + 448 * np.abs(s - ref)[:, None, None]
    else:
        emax, largest = (8, 448.0) if fmt == "mxfp8" else (2, 6.0)
        blk = lambda z: z.reshape(n, heads, d // 32, 32)  # noqa: E731
        top, err = blk(a).max(-1), blk(rot).max(-1)
        s = np.exp2(scale.cpu().numpy().astype(np.float64) - 127)
        lo = np.exp2(np.floor(np.log2(np.maximum(top - err, 2.0 ** -149))) - emax)
        hi = np.exp2(np.floor(np.log2(np.maximum(top + err, 2.0 ** -149))) - emax)
        live = top > 0
        assert np.all((s >= np.maximum(lo, 2.0 ** -127)) & (s <= hi) | ~live)
        unit = np.repeat(s, 32, -1).reshape(y.shape)
        step = np.maximum(2.0 ** -4 * (a + rot), 2.0 ** -10 * unit) if fmt == "mxfp8" else \
            np.maximum(2.0 ** -2 * (a + rot), 0.25 * unit)
        tol = np.maximum(step, a + rot - largest * unit) + rot
    assert np.all(np.abs(v - y) <= tol), np.argwhere(np.abs(v - y) > tol)[0]


def test_strided_and_unaligned_rows(hk):
    """A slice of a fused projection, head-major rows, rows off 16-byte alignment."""
    plan = hk.Rotary(32, first=32)
    base = _rows(21, 3, 64, 7).cuda()
    fused = torch.zeros(21, 3, 200, dtype=torch.bfloat16, device="cuda")
    fused[..., 72:136] = base
    off = torch.zeros(21 * 3 * 64 + 3, dtype=torch.bfloat16, device="cuda")[3:].view(21, 3, 64)
    off.copy_(base)
    for fmt in FORMATS:
        want = hk.quantize(base, fmt, rotary=plan, q_start=50)
        for x in (fused[..., 72:136], base.transpose(0, 1).contiguous().transpose(0, 1), off):
            got = hk.quantize(x, fmt, rotary=plan, q_start=50)
            assert torch.equal(got[0], want[0]) and (want[1] is None or torch.equal(got[1], want[1]))
    with pytest.raises(hk.HytopkError):  # rows that lie in the cache itself
        hk.cache_write(base, base.view(torch.bfloat16), fmt="bf16")


def test_long_rows_by_slot(hk):
    """Rows of 8,192 elements (several pieces a thread, or a workgroup of 1,024): slots, padding
    and repeats, few rows and many."""
    for fmt in FORMATS:
        for heads, d, n in ((64, 128, 40), (64, 128, 1100), (64, 96, 30)):
            x = _rows(n, heads, d, 17)
            L = 1200
            slots = np.random.default_rng(n).integers(-2, L, n).astype(np.int32)
            codes, scale = _empty(fmt, L, heads, d)
            want_c, want_s = _codes(codes).copy(), None if scale is None else scale.cpu().numpy().copy()
            hk.cache_write(x.cuda(), codes, scale, fmt=fmt, slots=torch.from_numpy(slots).cuda())
            rc, rs = _reference(x.float().numpy(), fmt)
            for i in range(n):
                if slots[i] >= 0:
                    want_c[slots[i]] = rc[i]
                    if rs is not None:
                        want_s[slots[i]] = rs[i]
            assert np.array_equal(_codes(codes), want_c), (fmt, heads, d, n)
            assert scale is None or np.array_equal(scale.cpu().numpy(), want_s)


def test_rows_behind_32_bit_offsets(hk):
    """A cache of more than 2^32 bytes: rows at its end keep their places."""
    L = (1 << 25) + 77
    codes = torch.zeros((L, 128), dtype=torch.uint8, device="cuda")
    scale = torch.ones(L, device="cuda")
    x = _rows(3, 1, 128, 8)[:, 0]
    slots = torch.tensor([L - 1, 5, 1 << 25], dtype=torch.int32, device="cuda")
    hk.cache_write(x.cuda(), codes, scale, slots=slots)
    rc, rs = _reference(x.float().numpy(), "fp8")
    assert np.array_equal(codes[slots.long()].cpu().numpy(), rc)
    assert int((codes != 0).any(1).sum()) == int((rc != 0).any(1).sum())
    v = hk.cache_read(codes, scale, slots=slots, dtype=torch.float32)
    assert np.array_equal(v.cpu().numpy(), _values(rc, rs, "fp8").astype(np.float32))
    tail = hk.cache_read(codes, scale, start=L - 2, dtype=torch.float32)
    assert np.array_equal(tail[1].cpu().numpy(), v[0].cpu().numpy())


@pytest.mark.parametrize("n", [12, 2000])
def test_write_and_read_in_a_graph(hk, n):
    """Recorded with its workspace (n = 2000: rows by slot with repeats), replayed with
    other rows and slots, eager work between the replays."""
    L = 4096
    plan = hk.Rotary(64)
    x = _rows(n, 1, 128, 9)[:, 0].cuda()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    codes, scale = (t[:, 0].contiguous() for t in _empty("mxfp8", L, 1, 128))
    ws = torch.empty(max(hk.cache_write_workspace_bytes(codes, scale, n, fmt="mxfp8"), 1), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((n, 128), dtype=torch.bfloat16, device="cuda")

    def step(c, s, o):
        hk.cache_write(x, c, s, fmt="mxfp8", slots=slots, rotary=plan, q_pos=pos, workspace=ws)
        hk.cache_read(c, s, fmt="mxfp8", slots=slots, out=o)
    step(codes, scale, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(codes, scale, out)
    for rep in range(3):
        x.copy_(_rows(n, 1, 128, 30 + rep)[:, 0])
        g = np.random.default_rng(rep)
        slots.copy_(torch.from_numpy(g.integers(-3, L, n).astype(np.int32)))
        pos.add_(777)
        c2, s2, o2 = codes.clone(), scale.clone(), out.clone()
        graph.replay()
        torch.cuda.synchronize()
        step(c2, s2, o2)
        assert torch.equal(codes, c2) and torch.equal(scale, s2) and torch.equal(out, o2)
