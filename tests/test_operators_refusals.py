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


ROTARY = [  # arguments, status, a part of the message
    (dict(dim=63), EINVAL, "must be even"), (dict(dim=0), EINVAL, "must be even"), (dict(dim=66), EINVAL, "outside the head"),
    (dict(first=-2), EINVAL, "outside the head"), (dict(first=34), EINVAL, "outside the head"),
    (dict(layout=2), EINVAL, "unknown rotary layout"), (dict(layout=-1), EINVAL, "unknown rotary layout"),
    (dict(freq=FREQ + 4), EINVAL, "8-byte aligned"), (dict(gain=float("nan")), EINVAL, "gain must be finite"),
    (dict(gain=float("-inf")), EINVAL, "gain must be finite"), (dict(gain=1e39), EINVAL, "gain must be finite"),
    (dict(dim=1026, d=2048), EUNSUPPORTED, "rotary dim > 1024"),
    (dict(n=-1), EINVAL, "n must be >= 0"), (dict(heads=0), EINVAL, "heads, d > 0"), (dict(d=0, dim=2), EINVAL, "heads, d > 0"),
    (dict(n=1 << 31), EUNSUPPORTED, "n >= 2^31"), (dict(heads=1 << 20, d=1 << 11), EUNSUPPORTED, "heads * d >= 2^31"),
    (dict(x=None), EINVAL, "rows are NULL"), (dict(x=(0, None, None, BF16)), EINVAL, "rows data is NULL"),
    (dict(x=(X, None, None, 2)), EINVAL, "unknown rows dtype"), (dict(x=(X, None, None, -1)), EINVAL, "unknown rows dtype"),
    (dict(x=(X + 1, None, None, BF16)), EINVAL, "aligned to their element"),
    (dict(x=(X + 2, None, None, FP32)), EINVAL, "aligned to their element"),
    (dict(x=(X, -1, None, BF16)), EINVAL, "strides must be >= 0"), (dict(x=(X, None, -1, BF16)), EINVAL, "strides must be >= 0"),
    (dict(x=(X, 1 << 62, None, BF16)), EINVAL, "more memory than exists"),
    (dict(y=(OUT, 1 << 62, None, BF16)), EINVAL, "more memory than exists"),
    (dict(y=(OUT, None, None, 7)), EINVAL, "unknown rows dtype"), (dict(y=(OUT + 1, None, None, BF16)), EINVAL, "aligned to their element"),
    (dict(y=(OUT, None, 0, BF16)), EINVAL, "rows of y overlap"), (dict(y=(OUT, None, 63, BF16)), EINVAL, "rows of y overlap"),
    (dict(y=(OUT, 191, None, BF16)), EINVAL, "rows of y overlap"), (dict(y=(OUT, 64, 255, BF16)), EINVAL, "rows of y overlap"),
    (dict(y=(X + 64, None, None, BF16)), EINVAL, "x and y overlap"), (dict(y=(X, None, None, FP32)), EINVAL, "x and y overlap"),
    (dict(y=(X, 600, None, BF16)), EINVAL, "x and y overlap"),
    (dict(start=-1), EINVAL, "positions q_start"), (dict(start=(1 << 31) - 3), EINVAL, "positions q_start"),
    (dict(pos=POS + 2), EINVAL, "q_pos must be 4-byte"), (dict(pos=OUT + 4 * 3 * 64 * 2 - 4, freq=FREQ), EINVAL, "the positions or the plan"),
    (dict(start=(1 << 31) - 4), EINVAL, "the positions or the plan"), (dict(pos=POS, start=-1), EINVAL, "the positions or the plan"),
    (dict(y=(OUT, 64, 256, BF16)), EINVAL, "the positions or the plan"), (dict(d=1030, dim=1024), EINVAL, "the positions or the plan"),
]


@pytest.mark.parametrize("kw,status,words", ROTARY)
def test_rotary_refuses_for_its_reason(lib, kw, status, words):
    refused(lib, rotary(lib, **kw), status, words)


def test_rotary_refuses_a_plan_without_frequencies(lib):
    p, r = hk.RotaryPlan(None, 1.0, 32, 0, 0, 0), hk.RowsArray(X, 192, 64, BF16, 0)
    call = lambda plan: lib.hytopk_rotary(plan, 4, 3, 64, ctypes.byref(r), ctypes.byref(r), None, 0, 0, None)  # noqa: E731
    refused(lib, call(ctypes.byref(p)), EINVAL, "rotary freq is NULL")
    refused(lib, call(None), EINVAL, "rotary plan is NULL")


WRITE = [
    (dict(codes=None), EINVAL, "cache codes are NULL"), (dict(codes=CODES + 8), EINVAL, "codes must be 16-byte"),
    (dict(scale=None), EINVAL, "need scales"), (dict(scale=SCALE + 2), EINVAL, "scales must be 4-byte"),
    (dict(L=0), EINVAL, "L, heads and d"), (dict(heads=0), EINVAL, "L, heads and d"), (dict(d=0), EINVAL, "L, heads and d"),
    (dict(dtype=4), EINVAL, "unknown dtype"), (dict(dtype=-1), EINVAL, "unknown dtype"), (dict(L=1 << 31), EUNSUPPORTED, "L >= 2^31"),
    (dict(d=100), EUNSUPPORTED, "multiples of 32"), (dict(d=16), EUNSUPPORTED, "multiples of 32"),
    (dict(heads=65), EUNSUPPORTED, "heads * d > 8192"), (dict(n=-1), EINVAL, "n must be >= 0"), (dict(n=1 << 31), EUNSUPPORTED, "n >= 2^31"),
    (dict(slots=SLOTS + 1), EINVAL, "slots must be 4-byte"), (dict(slots=None, start=-1), EINVAL, "outside the cache"),
    (dict(slots=None, start=(1 << 20) - 1999), EINVAL, "outside the cache"), (dict(slots=None, n=(1 << 20) + 1), EINVAL, "outside the cache"),
    (dict(x=None), EINVAL, "rows data is NULL"), (dict(x=X + 1), EINVAL, "aligned to their element"), (dict(xtype=2), EINVAL, "unknown rows dtype"),
    (dict(ts=-1), EINVAL, "strides must be >= 0"), (dict(dim=130), EINVAL, "outside the head"), (dict(dim=0), EINVAL, "must be even"),
    (dict(pos=POS + 2), EINVAL, "q_pos must be 4-byte"), (dict(freq=FREQ + 4), EINVAL, "8-byte aligned"),
    (dict(x=CODES + (128 << 20) - 2), EINVAL, "x overlaps the cache"), (dict(x=CODES - 2000 * 256 + 2), EINVAL, "x overlaps the cache"),
    (dict(x=SCALE, scale=SCALE + 4096), EINVAL, "x overlaps the cache"), (dict(ws=None), EWORKSPACE, "workspace is NULL"),
    (dict(ws=WS + 128), EWORKSPACE, "256-byte aligned"), (dict(ws_bytes=(4 << 20) - 1), EWORKSPACE, "too small"),
    (dict(slots=CODES + 4), EINVAL, "overlap the cache"), (dict(pos=CODES + 4), EINVAL, "overlap the cache"),
    (dict(freq=CODES + 8), EINVAL, "overlap the cache"), (dict(ws=CODES + 256), EINVAL, "overlap the cache"),
    (dict(slots=None, start=(1 << 20) - 2000), EINVAL, "codes and scales overlap"), (dict(ws_bytes=4 << 20), EINVAL, "codes and scales overlap"),
    (dict(ts=0, hs=0), EINVAL, "codes and scales overlap"), (dict(freq=None, pos=POS + 2), EINVAL, "codes and scales overlap"),
]


@pytest.mark.parametrize("kw,status,words", WRITE)
def test_cache_write_refuses_for_its_reason(lib, kw, status, words):
    refused(lib, write(lib, **kw), status, words)


def read(lib, n=100, L=1 << 20, dtype=hk.FP8_E4M3, heads=1, d=128, codes=CODES, scale=SCALE, slots=OUT + 1024, start=0,
         out=OUT, out_type=BF16):
    """The slots lie in the result (the last check)."""
    c = hk.Cache(codes, scale, L, heads, d, dtype, 0)
    return lib.hytopk_cache_read(ctypes.byref(c), n, slots, start, out, out_type, None)


READ = [
    (dict(), EINVAL, "out overlaps the slots"), (dict(slots=OUT + 100 * 256 - 4), EINVAL, "out overlaps the slots"),
    (dict(slots=OUT + 100 * 512 - 4, out_type=FP32), EINVAL, "out overlaps the slots"), (dict(slots=OUT - 396), EINVAL, "out overlaps the slots"),
    (dict(dtype=hk.BF16, scale=None), EINVAL, "out overlaps the slots"),
    (dict(codes=None), EINVAL, "cache codes are NULL"), (dict(codes=CODES + 8), EINVAL, "codes must be 16-byte"), (dict(scale=None), EINVAL, "need scales"),
    (dict(scale=SCALE + 1), EINVAL, "scales must be 4-byte"), (dict(L=0), EINVAL, "L, heads and d"), (dict(dtype=9), EINVAL, "unknown dtype"),
    (dict(d=48), EUNSUPPORTED, "multiples of 32"), (dict(heads=65), EUNSUPPORTED, "heads * d > 8192"), (dict(n=-1), EINVAL, "n must be >= 0"),
    (dict(n=1 << 31), EUNSUPPORTED, "n >= 2^31"), (dict(slots=OUT + 1026), EINVAL, "slots must be 4-byte"),
    (dict(slots=None, start=-1), EINVAL, "outside the cache"), (dict(slots=None, start=(1 << 20) - 99), EINVAL, "outside the cache"),
    (dict(out=None), EINVAL, "out is NULL"), (dict(out=OUT + 8), EINVAL, "out must be 16-byte"), (dict(out_type=2), EINVAL, "unknown rows dtype"),
    (dict(out=CODES + (128 << 20) - 16), EINVAL, "out overlaps the cache"), (dict(out=SCALE - 100 * 256 + 16), EINVAL, "out overlaps the cache"),
    (dict(slots=None, start=(1 << 20) - 100, out=CODES), EINVAL, "out overlaps the cache"),
]


@pytest.mark.parametrize("kw,status,words", READ)
def test_cache_read_refuses_for_its_reason(lib, kw, status, words):
    refused(lib, read(lib, **kw), status, words)


Q, K, IDX, LSE, MASS, MWS = (at(i + 20) for i in range(6))
OVER = "must not overlap the inputs"


def mass(lib, L=1000, n=4, heads=64, key_heads=1, d=128, k=100, scale=0.1, q=Q, keys=K, idx=IDX, lse=LSE, out=IDX + 16, ws=MWS,
         ws_bytes=1 << 30):
    """The mass lies over the indices (the last check)."""
    a = hk.Attention(L, n, heads, key_heads, d, k, scale, 0)
    return lib.hytopk_attention_mass(ctypes.byref(a), q, keys, idx, lse, out, ws, ws_bytes, None)


MASS_CASES = [
    (dict(), EINVAL, OVER), (dict(lse=None), EINVAL, OVER), (dict(ws=None, ws_bytes=0), EINVAL, OVER), (dict(heads=1024, key_heads=2), EINVAL, OVER),
    (dict(L=0), EINVAL, "L must be > 0"), (dict(n=-1), EINVAL, "n >= 0"), (dict(heads=0), EINVAL, "key_heads must divide"),
    (dict(key_heads=0), EINVAL, "key_heads must divide"), (dict(key_heads=3), EINVAL, "key_heads must divide"), (dict(key_heads=-1), EINVAL, "key_heads must divide"),
    (dict(k=0), EINVAL, "k must be > 0"), (dict(k=2049), EUNSUPPORTED, "k > 2048"), (dict(d=100), EUNSUPPORTED, "d must be 64"), (dict(d=0), EUNSUPPORTED, "d must be 64"),
    (dict(scale=float("nan")), EINVAL, "softmax_scale must be finite"), (dict(scale=3e38), EINVAL, "softmax_scale must be finite"),
    (dict(L=1 << 31), EUNSUPPORTED, "L >= 2^31"), (dict(n=1 << 24), EUNSUPPORTED, "n >= 2^24"), (dict(n=1 << 23, d=512), EUNSUPPORTED, "n >= 2^24, or 2^23"),
    (dict(heads=1025), EUNSUPPORTED, "heads > 1024"),
    (dict(q=None), EINVAL, "must be non-NULL"), (dict(keys=None), EINVAL, "must be non-NULL"), (dict(idx=None), EINVAL, "must be non-NULL"),
    (dict(out=None), EINVAL, "must be non-NULL"), (dict(q=Q + 8), EINVAL, "q and k must be 16-byte"), (dict(keys=K + 2), EINVAL, "q and k must be 16-byte"),
    (dict(idx=IDX + 2), EINVAL, "4-byte aligned"), (dict(lse=LSE + 2), EINVAL, "4-byte aligned"), (dict(out=IDX + 18), EINVAL, "4-byte aligned"),
    (dict(lse=None, ws=None), EWORKSPACE, "workspace is NULL"), (dict(lse=None, ws=MWS + 4), EWORKSPACE, "256-byte aligned"),
    (dict(lse=None, n=1, ws_bytes=1), EWORKSPACE, "too small"),
    (dict(out=Q + 2 * 4 * 64 * 128 - 4), EINVAL, OVER), (dict(out=K - 1596), EINVAL, OVER), (dict(out=LSE + 4), EINVAL, OVER),
    (dict(out=MASS, lse=None, ws=MASS - 256, n=1, k=2000), EINVAL, OVER), (dict(out=MASS, lse=None, ws=Q, n=1, k=2000), EINVAL, OVER),
    (dict(out=MASS, lse=None, ws=K, n=1, k=2000), EINVAL, OVER), (dict(out=MASS, lse=None, ws=IDX, n=1, k=2000), EINVAL, OVER),
]


@pytest.mark.parametrize("kw,status,words", MASS_CASES)
def test_attention_mass_refuses_for_its_reason(lib, kw, status, words):
    refused(lib, mass(lib, **kw), status, words)


SCORE, TARGET, WEIGHT, LOSS, GRAD = (at(i + 30) for i in range(5))


def index_loss(lib, n=4, k=100, score=SCORE, target=TARGET, weight=WEIGHT, loss=TARGET + 1584, grad=GRAD):
    """The loss lies over the target (the last check)."""
    return lib.hytopk_index_loss(n, k, score, target, weight, loss, grad, None)


LOSS_CASES = [
    (dict(), EINVAL, "loss overlaps"), (dict(grad=None), EINVAL, "loss overlaps"), (dict(weight=None), EINVAL, "loss overlaps"),
    (dict(grad=SCORE), EINVAL, "loss overlaps"), (dict(grad=TARGET), EINVAL, "loss overlaps"), (dict(loss=SCORE - 12), EINVAL, "loss overlaps"),
    (dict(loss=WEIGHT + 12), EINVAL, "loss overlaps"), (dict(loss=GRAD + 1596), EINVAL, "loss overlaps"),
    (dict(n=-1), EINVAL, "n must be >= 0"), (dict(k=0), EINVAL, "k > 0"), (dict(k=2049), EUNSUPPORTED, "k > 2048"), (dict(n=1 << 31), EUNSUPPORTED, "n >= 2^31"),
    (dict(score=None), EINVAL, "score and mass must be non-NULL"), (dict(target=None), EINVAL, "score and mass must be non-NULL"),
    (dict(loss=None, grad=None), EINVAL, "both NULL"), (dict(score=SCORE + 2), EINVAL, "4-byte aligned"), (dict(target=TARGET + 2), EINVAL, "4-byte aligned"),
    (dict(weight=WEIGHT + 1), EINVAL, "4-byte aligned"), (dict(loss=LOSS + 3), EINVAL, "4-byte aligned"), (dict(grad=GRAD + 2), EINVAL, "4-byte aligned"),
    (dict(grad=SCORE + 16), EINVAL, "d_score overlaps an input"), (dict(grad=TARGET - 16), EINVAL, "d_score overlaps an input"),
    (dict(grad=WEIGHT - 1596), EINVAL, "d_score overlaps an input"),
]


@pytest.mark.parametrize("kw,status,words", LOSS_CASES)
def test_index_loss_refuses_for_its_reason(lib, kw, status, words):
    refused(lib, index_loss(lib, **kw), status, words)


def test_empty_rows_have_no_strides_to_refuse():
    """A tensor without elements is contiguous whatever its strides say (those from numpy are all 0)."""
    import numpy as np
    import torch
    empty = torch.from_numpy(np.zeros((0, 3, 64), np.float32))
    assert empty.stride() == (0, 0, 0)
    hk.operators._rows_array(empty, "x")
    with pytest.raises(ValueError):
        hk.operators._rows_array(torch.zeros(64, 3, 2).transpose(0, 2), "x")
