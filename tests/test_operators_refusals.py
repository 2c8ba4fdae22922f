"""Refusals of the operators around the selection, each by its own reason: every buffer has memory of its
own, a call has one fault, and the message is checked with the status, so that a case fails when its
check is gone.  No call gets past the checks: each one also has the fault that the library looks for last, so a
missing check shows as that one's message and nothing is launched."""
import ctypes

import pytest

import exact_top_token_amd as hk

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
BF16, FP32 = 0, 1


def at(i):
    """The i-th buffer's address: 16 GiB apart."""
    return (i + 1) << 34


CODES, SCALE, X, SLOTS, POS, FREQ, WS, OUT = (at(i) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    return hk.load_library()


def refused(lib, rc, status, words):
    assert rc == status, (rc, lib.hytopk_last_error())
    assert words in lib.hytopk_last_error().decode()


def write(lib, n=2000, L=1 << 20, dtype=hk.FP8_E4M3, heads=1, d=128, codes=CODES, scale=CODES + 256, x=X, ts=None,
          hs=None, xtype=BF16, slots=SLOTS, start=0, freq=FREQ, dim=64, first=0, pos=POS, ws=WS, ws_bytes=1 << 30):
    c = hk.Cache(codes, scale, L, heads, d, dtype, 0)
    r = hk.RowsArray(x, heads * d if ts is None else ts, d if hs is None else hs, xtype, 0)
    p = hk.RotaryPlan(freq, 1.0, dim, first, 0, 0)
    return lib.hytopk_cache_write(ctypes.byref(c), n, ctypes.byref(r), slots, start,
                                  ctypes.byref(p) if freq else None, pos, 0, ws, ws_bytes, None)


def test_a_write_s_last_check_is_that_codes_and_scales_lie_apart(lib):
    for kw in (dict(), dict(n=4, ws=None), dict(freq=None, pos=None), dict(slots=None, ws=None), dict(scale=CODES + (128 << 20) - 4),
               dict(scale=CODES - (4 << 20) + 4), dict(dtype=hk.MXFP8_E4M3, scale=CODES + (128 << 20) - 4),
               dict(dtype=hk.MXFP4_E2M1, scale=CODES + (64 << 20) - 4), dict(dtype=hk.MXFP4_E2M1, scale=CODES - (4 << 20) + 4)):
        refused(lib, write(lib, **kw), EINVAL, "codes and scales overlap")
    # scales apart: the next fault before it shows
    for scale in (CODES + (128 << 20), CODES - (4 << 20)):
        refused(lib, write(lib, scale=scale, slots=CODES), EINVAL, "overlap the cache")


# the claim workspace of more than 1,024 rows by slot: 4 L bytes
@pytest.mark.parametrize("kw", [
    dict(slots=WS + (4 << 20) - 4), dict(slots=WS - 4 * 2000 + 4), dict(x=WS + 1024), dict(x=WS - 2 * 128 * 2000 + 2),
    dict(pos=WS + 64), dict(freq=WS + (4 << 20) - 8), dict(freq=WS - 8 * 32 + 8),
])
def test_a_write_s_workspace_lies_apart_from_what_it_reads(lib, kw):
    refused(lib, write(lib, **kw), EINVAL, "the workspace overlaps")


def test_a_workspace_that_is_not_used_may_lie_anywhere(lib):
    for kw in (dict(n=1024, slots=WS), dict(slots=None, x=WS), dict(n=4, pos=WS)):
        refused(lib, write(lib, **kw), EINVAL, "codes and scales overlap")
    # one that only touches what is read is fine
    for kw in (dict(slots=WS + (4 << 20)), dict(slots=WS - 8000), dict(x=WS + (4 << 20)), dict(freq=WS - 256)):
        refused(lib, write(lib, **kw), EINVAL, "codes and scales overlap")


def rotary(lib, n=4, heads=3, d=64, x=(X, None, None, BF16), y=(OUT, None, None, BF16), dim=32, first=0, layout=0, gain=1.0,
           freq=None, pos=None, start=0):
    """x, y: (address, token stride, head stride, type); the plan lies over y's first row (the last check)."""
    rows = [None if r is None else hk.RowsArray(r[0], heads * d if r[1] is None else r[1], d if r[2] is None else r[2], r[3], 0)
            for r in (x, y)]
    p = hk.RotaryPlan((y[0] & ~7) if freq is None else freq, gain, dim, first, layout, 0)
    return lib.hytopk_rotary(ctypes.byref(p), n, heads, d, *(r if r is None else ctypes.byref(r) for r in rows), pos, start, 0, None)


def test_rotary_s_last_check_is_that_y_lies_apart_from_plan_and_positions(lib):
    for kw in (dict(), dict(x=(OUT, None, None, BF16)), dict(x=(X, None, 0, FP32)), dict(x=(X, 0, 0, BF16)), dict(n=1)):
        refused(lib, rotary(lib, **kw), EINVAL, "the positions or the plan")


SLICES = [  # n, heads, d, x, y of one buffer (offset in elements, token stride, head stride), whether they share memory
    (9, 3, 64, (0, 600, 200), (64, 600, 200), False), (9, 3, 64, (0, 600, 200), (136, 600, 200), False),
    (9, 3, 64, (0, 600, 200), (63, 600, 200), True), (9, 3, 64, (0, 600, 200), (137, 600, 200), True),
    (9, 3, 64, (136, 600, 200), (0, 600, 200), False), (9, 3, 64, (137, 600, 200), (0, 600, 200), True),
    # neighbouring heads of a projection, one slot apart, in the next token's slice
    (9, 3, 64, (0, 576, 64), (192, 576, 64), False), (9, 3, 64, (0, 576, 64), (384, 576, 64), False),
    (9, 3, 64, (0, 576, 64), (191, 576, 64), True), (9, 3, 64, (0, 576, 64), (385, 576, 64), True),
    (9, 3, 64, (0, 576, 64), (192 + 576, 576, 64), False), (9, 3, 64, (0, 576, 64), (128, 576, 64), True),
    # heads before tokens
    (9, 3, 64, (0, 128, 2000), (64, 128, 2000), False), (9, 3, 64, (0, 128, 2000), (65, 128, 2000), True),
    (9, 3, 64, (0, 64, 2000), (9 * 64, 64, 2000), False), (9, 3, 64, (0, 64, 2000), (8 * 64, 64, 2000), True),
    # one axis alone
    (9, 1, 64, (0, 128, 5), (64, 128, 7), False), (1, 3, 64, (0, 5, 128), (64, 7, 128), False),
    # other strides: taken as whole extents
    (9, 3, 64, (0, 600, 200), (64, 600, 190), True), (9, 3, 64, (0, 600, 0), (64, 600, 100), True),
    (9, 3, 64, (0, 600, 200), (8 * 600 + 2 * 200 + 64, 600, 190), False),
]


@pytest.mark.parametrize("elem", [BF16, FP32])
@pytest.mark.parametrize("case", SLICES)
def test_rotary_between_slices_of_one_buffer(lib, case, elem):
    n, heads, d, x, y, shared = case
    size = 4 if elem == FP32 else 2
    rows = [(X + size * r[0], r[1], r[2], elem) for r in (x, y)]
    cells = [{r[0] + i * r[1] + h * r[2] + e for i in range(n) for h in range(heads) for e in range(d)} for r in (x, y)]
    assert shared or not cells[0] & cells[1]
    if x[1:] == y[1:]:
        assert bool(cells[0] & cells[1]) == shared
    refused(lib, rotary(lib, n, heads, d, *rows), EINVAL, "x and y overlap" if shared else "the positions or the plan")


def test_rotary_between_slices_of_two_types(lib):
    """fp32 rows of 256 bytes and bf16 rows of 128 in cells of 384."""
    for off, shared in ((0, True), (254, True), (256, False), (258, True), (256 + 384, False), (256 - 384, False)):
        x, y = (X, 96 * 3, 96, FP32), (X + off, 2 * 96 * 3, 2 * 96, BF16)
        refused(lib, rotary(lib, x=x, y=y), EINVAL, "x and y overlap" if shared else "the positions or the plan")


def test_a_plan_with_a_gain_or_frequencies_of_its_own():
    """YaRN of a model that takes the factor elsewhere, and frequencies that no scaling here gives."""
    import numpy as np
    import torch
    kw = dict(scaling="yarn", factor=40.0, original=4096, device="cpu")
    one, usual = hk.Rotary(64, gain=1.0, **kw), hk.Rotary(64, **kw)
    assert one.gain == 1.0 and one._plan.gain == 1.0 and torch.equal(one.freq, usual.freq)
    assert abs(usual.gain - (0.1 * np.log(40.0) + 1)) < 1e-15
    assert hk.Rotary(64, gain=0, device="cpu").gain == 0.0
    f = np.geomspace(2.0, 1e-7, 32)
    for own in (f, list(f), torch.from_numpy(f)):
        p = hk.Rotary(64, first=64, layout="interleaved", freq=own, gain=0.5, device="cpu")
        assert p.freq.dtype == torch.float64 and np.array_equal(p.freq.numpy(), f)
        assert (p.gain, p.dim, p.first, p.layout) == (0.5, 64, 64, "interleaved")
        assert p._plan.freq == p.freq.data_ptr()
    mine = torch.from_numpy(f.copy())
    kept = hk.Rotary(64, freq=mine, device="cpu")
    mine.zero_()
    assert kept.gain == 1.0 and np.array_equal(kept.freq.numpy(), f)  # a copy: the plan does not change with it
    assert np.array_equal(hk.Rotary(64, freq=f.astype(np.float32), device="cpu").freq.numpy(), f.astype(np.float32).astype(np.float64))
    for bad in (dict(freq=f[:31]), dict(freq=f[None]), dict(freq=f * np.inf), dict(freq=np.append(f[:31], np.nan)),
                dict(freq=f, scaling="linear", factor=2.0), dict(gain=float("nan")), dict(gain=float("inf"))):
        with pytest.raises(ValueError):
            hk.Rotary(64, device="cpu", **bad)
    with pytest.raises(hk.HytopkError):
        hk.Rotary(63, freq=f, device="cpu")
