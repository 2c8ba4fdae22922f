"""Refusals of the operators around the selection, without a GPU: every bad
argument is rejected before any launch, in the C ABI and in the binding."""
import ctypes

import pytest
import torch

import exact_top_token_amd as hk

BF16, FP32 = 0, 1
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    return hk.load_library()


def rows(data=FAKE, ts=8192, hs=128, dtype=BF16):
    return hk.RowsArray(data, ts, hs, dtype, 0)


def plan(freq=FAKE, gain=1.0, dim=64, first=0, layout=0):
    return hk.RotaryPlan(freq, gain, dim, first, layout, 0)


def cache(codes=FAKE, scale=FAKE, L=1000, heads=1, d=128, dtype=hk.FP8_E4M3):
    return hk.Cache(codes, scale, L, heads, d, dtype, 0)


def rotary(lib, p=None, n=4, heads=64, d=128, x=None, y=None, pos=None, start=0):
    p, x, y = p or plan(), x or rows(), y or rows(data=FAKE + (1 << 30))
    return lib.hytopk_rotary(ctypes.byref(p), n, heads, d, ctypes.byref(x), ctypes.byref(y), pos,
                             start, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(p=plan(dim=63)), -1), (dict(p=plan(dim=0)), -1), (dict(p=plan(dim=130)), -1),
    (dict(p=plan(first=-2)), -1), (dict(p=plan(first=66)), -1), (dict(p=plan(layout=2)), -1),
    (dict(p=plan(freq=None)), -1), (dict(p=plan(freq=FAKE + 4)), -1),
    (dict(p=plan(gain=float("nan"))), -1), (dict(p=plan(gain=float("inf"))), -1),
    (dict(p=plan(dim=2048), d=4096, heads=1), -2),
    (dict(n=-1), -1), (dict(heads=0), -1), (dict(d=0), -1), (dict(n=1 << 31), -2),
    (dict(heads=1 << 20, d=1 << 12), -2),
    (dict(x=rows(data=None)), -1), (dict(x=rows(dtype=2)), -1), (dict(x=rows(data=FAKE + 1)), -1),
    (dict(x=rows(data=FAKE + 2, dtype=FP32)), -1), (dict(x=rows(ts=-1)), -1),
    (dict(y=rows(data=None)), -1), (dict(x=rows(ts=1 << 62)), -1),
    # rows of y that share elements: broadcast heads, overlapping tokens
    (dict(y=rows(data=FAKE + (1 << 30), hs=0)), -1), (dict(y=rows(data=FAKE + (1 << 30), hs=64)), -1),
    (dict(y=rows(data=FAKE + (1 << 30), ts=8191)), -1),
    # x and y overlap without being the same rows
    (dict(y=rows(data=FAKE + 64)), -1), (dict(y=rows(dtype=FP32)), -1), (dict(x=rows(hs=0)), 0),
    (dict(start=-1), -1), (dict(start=(1 << 31) - 3), -1),
])
def test_rotary_refusals(lib, kw, code):
    if code == 0:  # x broadcast over heads is allowed: refused only for its NULL y
        kw = dict(kw, y=rows(data=None))
        code = -1
    assert rotary(lib, **kw) == code
    assert lib.hytopk_last_error().decode()


def test_empty_calls_do_nothing(lib):
    assert rotary(lib, n=0, x=rows(data=None), y=rows(data=None)) == 0
    c = cache()
    x = rows(data=None)
    assert lib.hytopk_cache_write(ctypes.byref(c), 0, ctypes.byref(x), None, 0, None, None, 0, None, 0, None) == 0
    assert lib.hytopk_cache_read(ctypes.byref(c), 0, None, 0, None, 0, None) == 0
    a = hk.Attention(100, 0, 8, 1, 128, 64, 0.1, 0)
    assert lib.hytopk_attention_mass(ctypes.byref(a), *([None] * 6), 0, None) == 0
    assert lib.hytopk_index_loss(0, 5, *([None] * 6)) == 0


@pytest.mark.parametrize("args,code", [
    ((63, 1e4, 0, 1.0, 0), -1), ((0, 1e4, 0, 1.0, 0), -1), ((2048, 1e4, 0, 1.0, 0), -2),
    ((64, 1.0, 0, 1.0, 0), -1), ((64, float("inf"), 0, 1.0, 0), -1), ((64, 1e4, 4, 1.0, 0), -1),
    ((64, 1e4, 1, 0.5, 0), -1), ((64, 1e4, 2, float("nan"), 0), -1), ((64, 1e4, 3, 4.0, 0), -1),
])
def test_frequency_refusals(lib, args, code):
    f = (ctypes.c_double * 1024)()
    g = ctypes.c_double()
    assert lib.hytopk_rotary_frequencies(*args, ctypes.cast(f, ctypes.c_void_p), ctypes.byref(g)) == code


def test_frequencies_by_their_definitions():
    f = hk.Rotary(64, device="cpu").freq
    want = 10000.0 ** (-2 * torch.arange(32, dtype=torch.float64) / 64)
    assert torch.allclose(f, want, rtol=1e-14, atol=0)
    assert torch.allclose(hk.Rotary(64, scaling="linear", factor=8, device="cpu").freq, want / 8,
                          rtol=1e-14, atol=0)
    n = hk.Rotary(64, scaling="ntk", factor=8, device="cpu").freq
    assert abs(n[0] - 1) < 1e-15 and abs(n[-1] / (want[-1] / 8) - 1) < 1e-12
    y = hk.Rotary(64, scaling="yarn", factor=8, original=4096, device="cpu")
    turns = 4096 * want / (2 * torch.pi)
    # kept where a pair turns more than 32 times, divided where it turns less than once (one
    # pair beside each border rounds to the other side)
    keep, div = (turns > 32).nonzero().flatten()[:-1], (turns < 1).nonzero().flatten()[1:]
    assert torch.allclose(y.freq[keep], want[keep], rtol=1e-14, atol=0)
    assert torch.allclose(y.freq[div], want[div] / 8, rtol=1e-14, atol=0)
    assert (y.freq[1:] < y.freq[:-1]).all() and abs(y.gain - (0.1 * torch.log(torch.tensor(8.0)).item() + 1)) < 1e-7


def write(lib, c=None, n=4, x=None, slots=None, start=0, p=None, pos=None, ws=None, wb=0):
    c, x = c or cache(), x or rows(data=FAKE + (1 << 30), ts=128)
    return lib.hytopk_cache_write(ctypes.byref(c), n, ctypes.byref(x), slots, start,
                                  None if p is None else ctypes.byref(p), pos, 0, ws, wb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(c=cache(codes=None)), -1), (dict(c=cache(codes=FAKE + 8)), -1), (dict(c=cache(scale=None)), -1),
    (dict(c=cache(scale=FAKE + 2)), -1), (dict(c=cache(L=0)), -1), (dict(c=cache(dtype=4)), -1),
    (dict(c=cache(dtype=-1)), -1), (dict(c=cache(d=100)), -2), (dict(c=cache(d=16)), -2),
    (dict(c=cache(heads=65)), -2), (dict(c=cache(L=1 << 31)), -2), (dict(c=cache(heads=0)), -1),
    (dict(n=-1), -1), (dict(n=1 << 31), -2), (dict(start=-1), -1), (dict(start=997), -1), (dict(n=1001), -1),
    (dict(x=rows(data=None)), -1), (dict(x=rows(dtype=3)), -1), (dict(x=rows(data=FAKE)), -1),
    (dict(c=cache(scale=FAKE + (1 << 30) + 64)), -1), (dict(slots=FAKE + 1), -1), (dict(p=plan(dim=130)), -1), (dict(p=plan(), pos=FAKE + 2), -1),
    # more rows by slot than look for later ones by themselves take a workspace
    (dict(c=cache(L=1 << 20), n=2000, slots=FAKE), -3),
    (dict(c=cache(L=1 << 20), n=2000, slots=FAKE, ws=FAKE, wb=(4 << 20) - 1), -3),
    (dict(c=cache(L=1 << 20), n=2000, slots=FAKE, ws=FAKE + 128, wb=1 << 30), -3),
])
def test_cache_write_refusals(lib, kw, code):
    assert write(lib, **kw) == code
    assert lib.hytopk_last_error().decode()


def test_cache_workspace_and_read_refusals(lib):
    c = cache(L=1 << 20)
    ws = lib.hytopk_cache_write_workspace
    assert ws(ctypes.byref(c), 1024, 1) == 0 and ws(ctypes.byref(c), 1 << 20, 0) == 0
    assert ws(ctypes.byref(c), 1025, 1) == 4 << 20
    assert ws(ctypes.byref(cache(d=100)), 4096, 1) == 0
    out = FAKE + (1 << 30)
    rd = lib.hytopk_cache_read
    assert rd(ctypes.byref(c), 4, None, 0, None, 0, None) == -1
    assert rd(ctypes.byref(c), 4, None, 0, out + 8, 0, None) == -1
    assert rd(ctypes.byref(c), 4, None, 0, out, 2, None) == -1
    assert rd(ctypes.byref(c), 4, None, (1 << 20) - 3, out, 0, None) == -1
    assert rd(ctypes.byref(c), 4, None, 0, FAKE + 1024, 0, None) == -1  # inside the cache
    assert rd(ctypes.byref(c), 4, FAKE + 3, 0, out, 0, None) == -1
    assert rd(ctypes.byref(cache(scale=None)), 4, None, 0, out, 0, None) == -1


def attention(L=1000, n=4, heads=64, kh=1, d=128, k=100, scale=0.1):
    return hk.Attention(L, n, heads, kh, d, k, scale, 0)


@pytest.mark.parametrize("a,code", [
    (attention(L=0), -1), (attention(n=-1), -1), (attention(heads=0), -1), (attention(kh=0), -1),
    (attention(kh=3), -1), (attention(k=0), -1), (attention(k=2049), -2), (attention(d=100), -2),
    (attention(scale=float("nan")), -1), (attention(L=1 << 31), -2), (attention(n=1 << 24), -2),
    (attention(heads=1025), -2), (attention(heads=1 << 30), -2),
])
def test_attention_mass_refusals(lib, a, code):
    assert lib.hytopk_attention_mass_workspace(ctypes.byref(a)) == 0
    assert lib.hytopk_attention_mass(ctypes.byref(a), *([FAKE] * 6), 1 << 40, None) == code


def test_attention_mass_pointers_and_workspace(lib):
    a = attention()
    need = lib.hytopk_attention_mass_workspace(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    assert lib.hytopk_attention_mass_workspace(ctypes.byref(attention(heads=128, d=576))) > 0
    call = lambda *v: lib.hytopk_attention_mass(ctypes.byref(a), *v, None)  # noqa: E731
    for i in (0, 1, 2, 4):
        v = [FAKE] * 6 + [1 << 30]
        v[i] = None
        assert call(*v) == -1
        v[i] = FAKE + 1
        assert call(*v) == -1
    assert call(FAKE, FAKE, FAKE, FAKE + 2, FAKE, FAKE, 1 << 30) == -1
    assert call(FAKE, FAKE, FAKE, None, FAKE, None, 0) == -3
    assert call(FAKE, FAKE, FAKE, None, FAKE, FAKE, need - 1) == -3


@pytest.mark.parametrize("args,code", [
    ((-1, 5) + (FAKE,) * 5, -1), ((4, 0) + (FAKE,) * 5, -1), ((4, 2049) + (FAKE,) * 5, -2),
    ((1 << 31, 5) + (FAKE,) * 5, -2), ((4, 5, None) + (FAKE,) * 4, -1),
    ((4, 5, FAKE, None) + (FAKE,) * 3, -1), ((4, 5, FAKE, FAKE, FAKE, None, None), -1),
    ((4, 5, FAKE + 2) + (FAKE,) * 4, -1), ((4, 5, FAKE, FAKE, FAKE + 1, FAKE, FAKE), -1),
])
def test_index_loss_refusals(lib, args, code):
    assert lib.hytopk_index_loss(*args, None) == code


def test_binding_refusals_without_a_gpu():
    """CPU tensors, wrong shapes, types and layouts never reach the library."""
    r = hk.Rotary(64, device="cpu")
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hk.rotary(x, r)
    with pytest.raises(TypeError):
        hk.operators._rows_array(x.half(), "x")
    with pytest.raises(ValueError):
        hk.operators._rows_array(x.transpose(1, 2), "x")
    with pytest.raises(ValueError):
        hk.operators._rows_array(x[0, 0], "x")
    with pytest.raises(ValueError):
        hk.Rotary(64, layout="pairs", device="cpu")
    with pytest.raises(ValueError):
        hk.Rotary(64, scaling="cubic", device="cpu")
    with pytest.raises(hk.HytopkError):
        hk.Rotary(63, device="cpu")
    for bad in (dict(dim=(1 << 32) + 64), dict(dim=64, first=-1), dict(dim=64, first=1 << 32), dict(dim=-2)):
        with pytest.raises(ValueError):
            hk.Rotary(**bad, device="cpu")
    with pytest.raises(ValueError):
        hk.cache_write(x, torch.zeros(8, 2, 128, dtype=torch.uint8), torch.ones(8))
    with pytest.raises(ValueError):
        hk.quantize(x, "fp8")
    with pytest.raises(ValueError):
        hk.quantize(x, "int4")
    with pytest.raises(ValueError):
        hk.cache_read(torch.zeros(8, 128, dtype=torch.uint8), torch.ones(8))
    with pytest.raises(ValueError):
        hk.attention_mass(x, torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(4, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        hk.index_loss(torch.zeros(4, 3), torch.zeros(4, 3))


def test_written_memory_stays_apart_from_what_is_read(lib):
    """Every call refuses results that lie over its inputs, its plan or its workspace."""
    y = rows(data=FAKE + (1 << 30))
    assert rotary(lib, y=y, p=plan(freq=FAKE + (1 << 30) + 64)) == -1
    assert rotary(lib, y=y, pos=FAKE + (1 << 30) + 2 * 4 * 8192 - 4) == -1  # the last row's last bytes
    c = cache(L=1 << 20)  # 128 MiB of codes; its scales lie over their beginning
    assert write(lib, c=c, slots=FAKE + 256) == -1
    assert write(lib, c=c, p=plan(freq=FAKE + 256)) == -1
    assert write(lib, c=c, p=plan(freq=FAKE + (1 << 29)), pos=FAKE + 512) == -1
    assert write(lib, c=c, n=2000, slots=FAKE + (1 << 29), ws=FAKE + 256, wb=1 << 30) == -1
    out = FAKE + (1 << 30)
    assert lib.hytopk_cache_read(ctypes.byref(c), 4, out + 512, 0, out, 0, None) == -1

    a = attention()
    need = lib.hytopk_attention_mass_workspace(ctypes.byref(a))
    q, k, idx, lse, mass, ws = (FAKE + (i << 28) for i in range(6))
    call = lambda *v: lib.hytopk_attention_mass(ctypes.byref(a), *v, None)  # noqa: E731
    for m in (q + 16, k + 16, idx, lse + 16):
        assert call(q, k, idx, lse, m, None, 0) == -1
    for w in (q, k, idx, mass):
        assert call(q, k, idx, None, mass, w, need) == -1

    score, mass, w, loss, d = (FAKE + (i << 28) for i in range(5))
    call = lambda *v: lib.hytopk_index_loss(4, 100, *v, None)  # noqa: E731
    for bad in (score + 16, mass - 16, w):
        assert call(score, mass, w, loss, bad) == -1
    for bad in (score, mass + 16, w, d + 1596):
        assert call(score, mass, w, bad, d) == -1


def test_limits_of_queries_and_scales(lib):
    """A launch's threads bound the queries (wide heads take twice as many threads), and factors
    must be finite as the kernels hold them."""
    ws = lib.hytopk_attention_mass_workspace
    assert ws(ctypes.byref(attention(n=(1 << 24) - 1, heads=1, d=256))) > 0
    for d in (512, 576):
        assert ws(ctypes.byref(attention(n=(1 << 23) - 1, heads=1, d=d))) > 0
        a = attention(n=1 << 23, heads=1, d=d)
        assert ws(ctypes.byref(a)) == 0
        assert lib.hytopk_attention_mass(ctypes.byref(a), *([FAKE] * 6), 1 << 40, None) == -2
    a = attention(scale=3e38)
    assert lib.hytopk_attention_mass(ctypes.byref(a), *([FAKE] * 6), 1 << 40, None) == -1
    assert rotary(lib, p=plan(gain=1e39)) == -1


def test_yarn_of_a_context_shorter_than_a_turn():
    """Positions below 2 pi leave every pair with less than one turn: all are divided."""
    f = hk.Rotary(64, scaling="yarn", factor=8, original=6, device="cpu").freq
    want = 10000.0 ** (-2 * torch.arange(32, dtype=torch.float64) / 64) / 8
    assert torch.allclose(f, want, rtol=1e-14, atol=0)
