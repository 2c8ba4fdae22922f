"""Refusals of the layer norm and of rotary plans of several axes, without a GPU, each by its own reason: every buffer has
memory of its own, a call has one fault, and the message is checked with the status.  No call gets past the checks: each one
also has the fault that the library looks for last."""
import ctypes

import pytest
import torch

import exact_top_token_amd as hk
from oracle import operators as op

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
BF16, FP32 = 0, 1


def at(i):
    """The i-th buffer's address: 16 GiB apart."""
    return (i + 1) << 34


X, Y, W, B, STATS, CODES, SCALE, DY, DX, DW, DB, WS, FREQ, POS = (at(i) for i in range(14))
LAST_FWD, LAST_BACK = "overlap each other, x or the parameters", "the gradients or the workspace overlap"


@pytest.fixture(scope="module")
def lib():
    return hk.load_library()


def refused(lib, rc, status, words):
    assert rc == status, (rc, lib.hytopk_last_error())
    assert words in lib.hytopk_last_error().decode()


def rows(addr, heads, d, dtype=BF16, ts=None, hs=None):
    return hk.RowsArray(addr, heads * d if ts is None else ts, d if hs is None else hs, dtype, 0)


def by(x):
    return None if x is None else ctypes.byref(x)


def forward(lib, n=5, heads=3, d=64, x=dict(), y=dict(), w=W, b=W, dtype=FP32, eps=1e-5, stats=STATS, save=None, norm=True):
    """With stats over the weight, which is looked for last."""
    a = None if x is None else rows(**{"addr": X, "heads": heads, "d": d, **x})
    c = None if y is None else rows(**{"addr": Y, "heads": heads, "d": d, **y})
    p = hk.Norm(w, b, dtype, eps) if norm else None
    if stats == STATS:
        stats = w
    return lib.hytopk_layer_norm(by(p), n, heads, d, by(a), by(c), stats, by(save), None)


def cache(codes=CODES, scale=SCALE, L=15, heads=1, d=64, dtype=hk.FP8_E4M3):
    return hk.Cache(codes, scale, L, heads, d, dtype, 0)


def kept(**kw):
    return cache(**{"L": 300, **kw})


def backward(lib, n=100, heads=3, d=64, dy=dict(), x=dict(), dx=dict(), saved=None, w=W, dtype=FP32, stats=STATS, dw=DW, db=None, ws=WS,
             ws_bytes=1 << 30, norm=True):
    """With dbias over dweight, which is looked for last."""
    a = None if dy is None else rows(**{"addr": DY, "heads": heads, "d": d, **dy})
    c = None if x is None else rows(**{"addr": X, "heads": heads, "d": d, **x})
    e = None if dx is None else rows(**{"addr": DX, "heads": heads, "d": d, **dx})
    p = hk.Norm(w, None, dtype, 0.0) if norm else None
    return lib.hytopk_layer_norm_backward(by(p), n, heads, d, by(a), by(c), by(saved), stats, by(e), dw, dw if db is None else db, ws,
                                          ws_bytes, None)


def test_the_last_checks(lib):
    for kw in (dict(), dict(n=1), dict(heads=1), dict(x=dict(hs=0)), dict(y=dict(addr=X)), dict(y=dict(dtype=FP32)), dict(save=cache()),
               dict(save=cache(dtype=hk.MXFP8_E4M3)), dict(save=cache(L=1 << 20)), dict(d=8192, heads=1), dict(eps=0.0), dict(d=1)):
        refused(lib, forward(lib, **kw), EINVAL, LAST_FWD)
    for kw in (dict(), dict(n=1), dict(dx=dict(addr=DY)), dict(dx=dict(addr=X)), dict(dx=None), dict(dy=dict(ts=0, hs=0)),
               dict(x=None, saved=kept()), dict(x=None, saved=kept(dtype=hk.MXFP8_E4M3)), dict(w=None), dict(d=8192, heads=1), dict(n=5)):
        refused(lib, backward(lib, **kw), EINVAL, LAST_BACK)


@pytest.mark.parametrize("kw,status,words", [
    (dict(n=-1), EINVAL, "n must be >= 0"), (dict(heads=0), EINVAL, "heads, d > 0"), (dict(d=0), EINVAL, "heads, d > 0"),
    (dict(n=1 << 31), EUNSUPPORTED, "n >= 2^31"), (dict(heads=1 << 20, d=1 << 12), EUNSUPPORTED, "heads * d"),
    (dict(d=8193, heads=1), EUNSUPPORTED, "d <= 8192"), (dict(n=1 << 30, heads=2, d=8), EUNSUPPORTED, "n * heads >= 2^31"),
    (dict(norm=False), EINVAL, "norm is NULL"), (dict(dtype=2), EINVAL, "norm's parameters"), (dict(dtype=-1), EINVAL, "norm's parameters"),
    (dict(w=W + 2, b=None), EINVAL, "weight and bias"), (dict(b=B + 2), EINVAL, "weight and bias"),
    (dict(w=W + 1, dtype=BF16), EINVAL, "weight and bias"),
    (dict(x=dict(addr=None)), EINVAL, "rows data is NULL"), (dict(x=dict(dtype=2)), EINVAL, "rows dtype"),
    (dict(x=dict(addr=X + 1)), EINVAL, "aligned to their element"), (dict(x=dict(ts=-1)), EINVAL, "strides"),
    (dict(x=dict(ts=1 << 60)), EINVAL, "more memory"),
])
def test_what_both_passes_refuse(lib, kw, status, words):
    refused(lib, forward(lib, **kw), status, words)
    if "b" not in kw or "w" in kw:  # the backward reads no bias
        refused(lib, backward(lib, **{k: v for k, v in kw.items() if k != "b"}), status, words)


@pytest.mark.parametrize("kw,status,words", [
    (dict(eps=-1e-9), EINVAL, "eps"), (dict(eps=float("nan")), EINVAL, "eps"), (dict(eps=float("inf")), EINVAL, "eps"),
    (dict(x=None), EINVAL, "rows are NULL"), (dict(y=None), EINVAL, "rows are NULL"), (dict(y=dict(hs=0)), EINVAL, "rows of y overlap"), (dict(y=dict(ts=191)), EINVAL, "rows of y overlap"),
    (dict(y=dict(addr=X + 64)), EINVAL, "x and y overlap"), (dict(y=dict(addr=X, dtype=FP32)), EINVAL, "x and y overlap"),
    (dict(y=dict(addr=X, ts=200)), EINVAL, "x and y overlap"), (dict(stats=at(4) + 4), EINVAL, "8-byte"),
    (dict(save=cache(), stats=None), EINVAL, "needs stats"), (dict(save=cache(L=14)), EINVAL, "outside the cache"),
    (dict(save=cache(heads=2, d=32)), EINVAL, "the norm's"), (dict(save=cache(d=96)), EINVAL, "the norm's"),
    (dict(save=cache(dtype=hk.BF16)), EUNSUPPORTED, "FP8 or MXFP8"), (dict(save=cache(dtype=hk.MXFP4_E2M1)), EUNSUPPORTED, "FP8 or MXFP8"),
    (dict(save=cache(codes=None)), EINVAL, "codes are NULL"), (dict(save=cache(scale=None)), EINVAL, "need scales"),
    (dict(save=cache(codes=CODES + 8)), EINVAL, "16-byte"), (dict(save=cache(d=40), d=40), EUNSUPPORTED, "multiples of 32"),
])
def test_forward_refusals(lib, kw, status, words):
    refused(lib, forward(lib, **kw), status, words)


STEP = 5 * 3 * 64  # elements of the rows


@pytest.mark.parametrize("kw", [
    dict(y=dict(addr=W)), dict(y=dict(addr=W - 2 * STEP + 2)), dict(y=dict(addr=W + 4 * 64 - 2)), dict(y=dict(addr=at(3))),
    dict(stats=X), dict(stats=X + 2 * STEP - 8), dict(stats=Y), dict(stats=Y - 8 * 15 + 8), dict(stats=at(3)),
    dict(save=cache(codes=X)), dict(save=cache(codes=Y + 16)), dict(save=cache(codes=at(3))), dict(save=cache(scale=CODES + 4)),
    dict(save=cache(scale=X)), dict(save=cache(scale=Y)), dict(save=cache(scale=at(4))), dict(save=cache(codes=at(4) - 960 + 16)),
])
def test_forward_overlaps(lib, kw):
    """Each of what is written over each of what lies elsewhere."""
    kw = dict(dict(b=at(3), stats=at(4)), **kw)
    refused(lib, forward(lib, **kw), EINVAL, LAST_FWD)


@pytest.mark.parametrize("kw,status,words", [
    (dict(dy=None), EINVAL, "rows are NULL"), (dict(x=None), EINVAL, "input or its checkpoint"),
    (dict(saved=kept()), EINVAL, "input or its checkpoint"), (dict(stats=None), EINVAL, "needs the forward's stats"),
    (dict(stats=STATS + 4), EINVAL, "8-byte"), (dict(dw=DW + 2), EINVAL, "4-byte"), (dict(db=DB + 1), EINVAL, "4-byte"),
    (dict(ws=None), EWORKSPACE, "NULL"), (dict(ws=WS + 128), EWORKSPACE, "256-byte"), (dict(ws_bytes=255), EWORKSPACE, "too small"),
    (dict(dx=dict(hs=0)), EINVAL, "rows of dx overlap"), (dict(dx=dict(dtype=3)), EINVAL, "rows dtype"),
    (dict(dx=dict(addr=DY + 2)), EINVAL, "dy and dx overlap"), (dict(dx=dict(addr=DY, dtype=FP32)), EINVAL, "dy and dx overlap"),
    (dict(dx=dict(addr=X - 2)), EINVAL, "x and dx overlap"), (dict(x=dict(hs=0), dx=dict(addr=X)), EINVAL, "x and dx overlap"),
    (dict(x=None, saved=kept(L=299)), EINVAL, "outside the cache"), (dict(x=None, saved=kept(dtype=hk.MXFP4_E2M1)), EUNSUPPORTED, "FP8 or MXFP8"),
])
def test_backward_refusals(lib, kw, status, words):
    refused(lib, backward(lib, **kw), status, words)


@pytest.mark.parametrize("kw", [
    dict(dx=dict(addr=W)), dict(dx=dict(addr=STATS - 2)), dict(dx=dict(addr=DW)), dict(dx=dict(addr=WS)), dict(dw=W), dict(dw=STATS),
    dict(dw=DY), dict(dw=X + 40 * STEP - 4), dict(db=X), dict(db=DX), dict(db=WS), dict(ws=DY), dict(ws=X), dict(ws=W), dict(ws=STATS),
    dict(ws=DX), dict(x=None, saved=kept(codes=DX)), dict(x=None, saved=kept(scale=DW)), dict(x=None, saved=kept(codes=WS)),
])
def test_backward_overlaps(lib, kw):
    kw = dict(dict(db=DB), **kw)
    refused(lib, backward(lib, **kw), EINVAL, LAST_BACK)


def test_nothing_to_do(lib):
    none = rows(None, 3, 64)
    p = hk.Norm(None, None, FP32, 1e-5)
    assert lib.hytopk_layer_norm(by(p), 0, 3, 64, by(none), by(none), None, None, None) == 0
    assert lib.hytopk_layer_norm(by(p), 0, 3, 64, by(none), by(none), None, by(cache(codes=None, L=0)), None) == 0
    assert lib.hytopk_layer_norm_backward(by(p), 0, 3, 64, by(none), by(none), None, None, by(none), None, None, None, 0, None) == 0
    # no sums wanted: no workspace
    refused(lib, backward(lib, dw=None, dx=dict(addr=W), ws=None), EINVAL, LAST_BACK)


def test_workspace(lib):
    need = lib.hytopk_layer_norm_backward_workspace
    assert need(0, 1, 64) == 0 and need(-1, 1, 64) == 0 and need(5, 0, 64) == 0 and need(5, 1, 8193) == 0 and need(1 << 30, 2, 64) == 0
    # few rows: none, and one that is given is not looked at
    for n, heads, d in ((0, 1, 64), (1, 1, 1), (1, 1, 8192), (1, 64, 128), (8, 1, 64), (1024, 1, 1)):
        assert need(n, heads, d) == 0
        for ws in (dict(ws=None), dict(ws=W), dict(ws=W + 4, ws_bytes=1)):
            refused(lib, backward(lib, n=n, heads=heads, d=d, **ws), EINVAL, LAST_BACK)
            refused(lib, backward(lib, n=n, heads=heads, d=d, db=W, **ws), EINVAL, LAST_BACK)
    for n, heads, d in ((77, 6, 201), (131072, 1, 128), (8192, 1, 5120), (2 ** 31 - 1, 1, 8192)):
        size = need(n, heads, d)
        assert size % 256 == 0 and 0 < size <= 512 * 2 * (d + 3) * 4 + 256
        # one byte less is refused
        refused(lib, backward(lib, n=n, heads=heads, d=d, ws_bytes=size - 1, dx=None), EWORKSPACE, "too small")


# ------------------------------------------------------ plans of several axes

def plan(freq=FREQ, gain=1.0, dim=64, first=0, layout=0, axes=3):
    return hk.RotaryPlan(freq, gain, dim, first, layout, axes)


def rotary(lib, p, n=4, pos=POS, y=Y):
    a, b = rows(X, 3, 64), rows(y, 3, 64)
    return lib.hytopk_rotary(by(p), n, 3, 64, by(a), by(b), pos, 0, 0, None)


def test_axes_refusals(lib):
    refused(lib, rotary(lib, plan(axes=-1)), EINVAL, "axes")
    refused(lib, rotary(lib, plan(axes=17)), EUNSUPPORTED, "axes > 16")
    # y over the positions and the plan, to their last byte: [n][axes] positions, the axes behind the frequencies
    for axes, pos, plan_bytes in ((0, 16, 256), (1, 16, 256), (2, 32, 384), (3, 48, 384), (16, 256, 384)):
        size = 2 * 4 * 3 * 64
        for kw in (dict(pos=Y - pos + 4), dict(pos=Y + size - 4), dict(pos=Y)):
            refused(lib, rotary(lib, plan(axes=axes), **kw), EINVAL, "the positions or the plan")
        refused(lib, rotary(lib, plan(freq=Y - plan_bytes + 8, axes=axes)), EINVAL, "the positions or the plan")
        if axes > 1:  # what lies apart with one axis
            refused(lib, rotary(lib, plan(axes=axes), pos=Y - 16 * 1 - 4), EINVAL, "the positions or the plan")
            refused(lib, rotary(lib, plan(freq=Y - 256, axes=axes)), EINVAL, "the positions or the plan")
    c = hk.Cache(CODES, CODES + 256, 100, 3, 64, hk.FP8_E4M3, 0)  # scales over the codes: looked for last
    x = rows(X, 3, 64)

    def write(p, pos):
        return lib.hytopk_cache_write(by(c), 4, by(x), None, 0, by(p), pos, 0, None, 0, None)
    refused(lib, write(plan(), POS), EINVAL, "codes and scales overlap")
    refused(lib, write(plan(), CODES - 44), EINVAL, "overlap the cache")
    refused(lib, write(plan(axes=1), CODES - 44), EINVAL, "codes and scales overlap")
    refused(lib, write(plan(freq=CODES - 376), POS), EINVAL, "overlap the cache")
    refused(lib, write(plan(axes=17), POS), EUNSUPPORTED, "axes > 16")


@pytest.mark.parametrize("kw", [
    dict(sections=(16, 15)), dict(sections=(16, 17)), dict(sections=(32, 0)), dict(sections=(33, -1)), dict(sections=()),
    dict(sections=(16,) + (1,) * 16), dict(cycle=True), dict(restart=True), dict(sections=(10, 11, 11), cycle=True),
    dict(sections=(1, 31), cycle=True), dict(sections=(16, 16), restart=True, freq=[0.1] * 32),
])
def test_plans_that_do_not_exist(kw):
    with pytest.raises(ValueError):
        hk.Rotary(64, device="cpu", **kw)


def test_axes_and_frequencies_of_the_pairs():
    def axes(dim=64, **kw):
        return hk.Rotary(dim, device="cpu", **kw).axis.tolist()
    assert axes(sections=(16, 8, 8)) == [0] * 16 + [1] * 8 + [2] * 8
    assert axes(dim=16, sections=(4, 2, 2), cycle=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert axes(dim=12, sections=[3, 3], cycle=True) == [0, 1, 0, 1, 0, 1]
    assert axes(dim=10, sections=(1, 1, 1, 1, 1), cycle=True) == [0, 1, 2, 3, 4]
    assert axes(sections=iter((12, 10, 10)), cycle=True)[:6] == [0, 1, 2, 0, 1, 2]
    one = hk.Rotary(64, device="cpu", sections=(32,))
    assert one.axes == 1 and one.axis is None and one._plan.axes == 0
    f = torch.from_numpy(op.rotary_frequencies(64))
    for kw in (dict(sections=(16, 8, 8)), dict(sections=(12, 10, 10), cycle=True)):
        p = hk.Rotary(64, device="cpu", **kw)
        assert torch.allclose(p.freq, f, rtol=1e-14, atol=0) and p._plan.axes == 3 and p.freq.shape == (32,)
        # behind the frequencies, as the library reads them
        tail = (ctypes.c_int32 * 32).from_address(p._plan.freq + 8 * 32)
        assert list(tail) == p.axis.tolist()
        r = hk.Rotary(64, device="cpu", restart=True, scaling="yarn", factor=4.0, original=4096, **kw)
        for a, s in enumerate(kw["sections"]):
            want, gain = op.rotary_plan(2 * s, scaling="yarn", factor=4.0, original=4096)
            assert torch.allclose(r.freq[p.axis == a], torch.from_numpy(want), rtol=1e-13, atol=0) and abs(r.gain - gain) < 1e-15
    # an odd number of pairs: the axes end in the middle of eight bytes
    odd = hk.Rotary(10, device="cpu", sections=(3, 2), freq=[1.0, 2.0, 3.0, 4.0, 5.0])
    assert odd.axis.tolist() == [0, 0, 0, 1, 1] and odd.freq.tolist() == [1.0, 2.0, 3.0, 4.0, 5.0]


# ------------------------------------------------------------------ the binding

def test_the_binding_s_refusals():
    x = torch.zeros((4, 2, 64))
    saved = hk.NormSaved(x, None, torch.zeros((4, 2, 2)), None)
    with pytest.raises(ValueError, match="GPU"):
        hk.layer_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        hk.layer_norm_backward(x, saved)


@pytest.mark.gpu
def test_the_binding_s_refusals_on_the_gpu():
    x = torch.randn((4, 2, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    y, saved = hk.layer_norm(x, w, save="x")
    _, coded = hk.layer_norm(x, w, save="fp8")
    for kw in (dict(weight=w[:63]), dict(weight=w.half()), dict(weight=w.cpu()), dict(bias=w.bfloat16(), weight=w), dict(weight=w[None]),
               dict(out=torch.empty((4, 2, 63), device="cuda")), dict(out=x.bfloat16(), out_dtype=torch.float32), dict(out_dtype=torch.float16),
               dict(save="bf16"), dict(save="mxfp4"), dict(save=saved._replace(stats=saved.stats[:3])), dict(save=saved._replace(rows=y)),
               dict(save=saved._replace(scale=w)), dict(save=coded._replace(fmt="mxfp8")), dict(save=coded._replace(scale=None)),
               dict(save=coded._replace(fmt="int8")), dict(out=x, save="x")):
        with pytest.raises((ValueError, TypeError)):
            hk.layer_norm(x, **kw)
    for bad in (x[0, 0], x[None], x.transpose(1, 2), x.half(), x.int()):
        with pytest.raises((ValueError, TypeError)):
            hk.layer_norm(bad)
    with pytest.raises(ValueError):  # d no multiple of 32
        hk.layer_norm(x[..., :48].contiguous(), save="fp8")
    for kw in (dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(hk.HytopkError):
            hk.layer_norm(x, **kw)
    with pytest.raises(hk.HytopkError):
        hk.layer_norm(torch.zeros((2, 8200), device="cuda"))
    for kw in (dict(weight=w[:63]), dict(want=("dx", "dbeta")), dict(out={"dbeta": w}), dict(out={"dweight": w[:63]}), dict(out={"dbias": w.bfloat16()}),
               dict(out={"dx": y.bfloat16()}, dx_dtype=torch.float32), dict(out={"dx": y[:3]}), dict(dx_dtype=torch.float16),
               dict(workspace=torch.empty(4096, device="cuda")), dict(workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            hk.layer_norm_backward(y, saved, **kw)
    z, kept_z = hk.layer_norm(torch.randn((400, 2, 64), device="cuda"), w, save="x")
    with pytest.raises(hk.HytopkError):
        hk.layer_norm_backward(z, kept_z, workspace=torch.empty(255, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        hk.layer_norm_backward(y[:, :1], saved)
    with pytest.raises(hk.HytopkError):  # a gradient over what is read
        hk.layer_norm_backward(y, saved, w, out={"dweight": w})
    plan = hk.Rotary(64, sections=(16, 16))
    pos = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for bad in (pos[:, 0].contiguous(), pos.t().contiguous(), pos.long(), pos[:3], torch.zeros((4, 3), dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            hk.rotary(x, plan, q_pos=bad)
        with pytest.raises(ValueError):
            hk.quantize(x, "fp8", rotary=plan, q_pos=bad)
    with pytest.raises(ValueError):
        hk.rotary(x, hk.Rotary(64), q_pos=pos)
