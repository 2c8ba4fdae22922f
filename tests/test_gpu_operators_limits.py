"""The operators around the selection at their limits: calls from two host threads at once,
workspaces that the binding takes while a graph is recorded, and more rows than one launch holds."""
import threading

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_amd as m
    m.load_library()
    return m


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


class _Work:
    """One chain of calls on inputs of its own."""

    def __init__(self, hk, seed, n, heads, d, k):
        g = torch.Generator().manual_seed(seed)
        self.hk, self.k = hk, k
        self.x, self.q = _rand((n, heads, 128), seed), _rand((n, heads, d), seed + 1)
        self.keys = _rand((500, 1, d), seed + 2)
        self.idx = torch.randint(-20, 520, (n, k), generator=g, dtype=torch.int32).cuda()
        self.score = _rand((n, k), seed + 3, torch.float32)
        self.slots = torch.randint(-5, 400, (n,), generator=g, dtype=torch.int32).cuda()
        self.plan = hk.Rotary(64, layout="half" if seed % 2 else "interleaved")

    def run(self):
        hk, n = self.hk, self.x.shape[0]
        y = hk.rotary(self.x, self.plan, q_start=100 * n)
        codes = torch.zeros((400, self.x.shape[1], 128), dtype=torch.uint8, device="cuda")
        scale = torch.ones(400, device="cuda")
        hk.cache_write(y, codes, scale, fmt="fp8", slots=self.slots, rotary=self.plan)
        back = hk.cache_read(codes, scale, fmt="fp8", slots=self.slots, dtype=torch.float32)
        mass = hk.attention_mass(self.q, self.keys, self.idx)
        loss, grad = hk.index_loss(self.score, mass)
        return y, codes, scale, back, mass, loss, grad


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_from_two_threads(hk):
    """Two host threads with a stream each: every result equals the call made alone."""
    work = [_Work(hk, 1, 30, 4, 128, 200), _Work(hk, 2, 1500, 2, 64, 77)]
    alone = [w.run() for w in work]
    torch.cuda.synchronize()
    wrong, gate = [], threading.Barrier(2)

    def go(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gate.wait(60)
                for rep in range(6):
                    got = work[i].run()
                    stream.synchronize()
                    if not _equal(got, alone[i]):
                        wrong.append((i, rep))
        except Exception as e:  # a thread's failure is the test's
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=go, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_graphs_with_workspaces_of_the_binding(hk):
    """Two recorded chains whose results and workspaces come from the graphs' own memory, replayed
    in turn with eager calls between."""
    work = [_Work(hk, 3, 24, 8, 128, 300), _Work(hk, 4, 1200, 4, 64, 50)]
    alone = [w.run() for w in work]
    torch.cuda.synchronize()
    graphs, out = [], []
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.append(w.run())
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1):
            graphs[i].replay()
        other = work[rep % 2].run()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert _equal(out[i], alone[i]), (rep, i)
        assert _equal(other, alone[rep % 2])
        for w in work:
            w.score.mul_(1.5)
        alone = [w.run() for w in work]
        torch.cuda.synchronize()


def test_rotary_of_more_tokens_than_a_launch_holds(hk):
    """Heads without 16-byte access, one row a workgroup's turn: 2^23 tokens fill the grid."""
    _room(20)
    n, d = (1 << 23) + 5, 258
    say(f"limits: rotary n={n} d={d}")
    plan = hk.Rotary(4, first=1)
    row = _rand((1, d), 5)
    y = hk.rotary(row.expand(n, d), plan)
    for at in (0, (1 << 22) + 1, (1 << 23) - 2, n - 9):
        assert torch.equal(y[at:at + 9], hk.rotary(row.expand(9, d).contiguous(), plan, q_start=at)[:n - at])
    assert int((y[:, 5:] != row[:, 5:]).sum()) == 0


def test_cache_of_more_rows_than_a_launch_holds(hk):
    """Rows written and read by slot in more workgroups than one grid has; nearly all are padding."""
    _room(60)
    n, d = (1 << 23) + 3, 2048
    say(f"limits: cache write n={n} d={d}")
    row = _rand((1, d), 6)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    for s, at in ((0, 5), (1, (1 << 23) - 1), (2, (1 << 23) + 1), (2, 77), (0, n - 1)):
        slots[at] = s
    codes = torch.full((4, d), 99, dtype=torch.uint8, device="cuda")
    scale = torch.full((4, d // 32), 99, dtype=torch.uint8, device="cuda")
    plan = hk.Rotary(64)
    hk.cache_write(row.expand(n, d), codes, scale, fmt="mxfp8", slots=slots, rotary=plan)
    for s, at in ((0, n - 1), (1, (1 << 23) - 1), (2, (1 << 23) + 1)):
        want, ws = hk.quantize(row, "mxfp8", rotary=plan, q_start=at)
        assert torch.equal(codes[s], want[0]) and torch.equal(scale[s], ws[0]), s
    assert (codes[3] == 99).all() and (scale[3] == 99).all()

    n = (1 << 21) + 13
    cache = _rand((3, 8192), 7)
    pick = torch.arange(n, dtype=torch.int32, device="cuda") % 4
    out = hk.cache_read(cache, slots=pick)  # every fourth row lies outside
    want = torch.cat([cache, torch.zeros_like(cache[:1])])
    for at in (0, (1 << 20) + 4, (1 << 21) - 8, n - 16):
        assert torch.equal(out[at:at + 16], want[pick[at:at + 16].long()][:n - at])
    del out


@pytest.mark.parametrize("d,most", [(64, 1 << 24), (256, 1 << 24), (512, 1 << 23)])
def test_mass_of_the_most_queries(hk, d, most):
    """One live entry a query holds all of its mass, padding none."""
    _room(40)
    n = most - 1
    say(f"limits: mass n={n} d={d}")
    q = _rand((1, 1, d), 8).expand(n, 1, d).contiguous()
    keys = _rand((10, 1, d), 9)
    idx = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1) % 11  # 10 is padding
    mass = hk.attention_mass(q, keys, idx)
    assert not mass[idx == 10].any()
    # |x| below 12 in base 2: its rounding 12 * 2^-24 ln 2, two powers of one ulp (2 * 2^-23), the
    # reciprocal and the product of half one each
    assert (mass[idx < 10] - 1).abs().max() <= (12 * 0.7 + 4 + 2) * 2.0 ** -24
