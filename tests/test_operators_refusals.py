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
