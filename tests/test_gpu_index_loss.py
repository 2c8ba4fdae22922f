"""The attention's mass at the selected entries and the indexer's loss with its
gradient, against the fp64 definitions (oracle.operators).

Mass: a logit's fp32 accumulation over d exact products is off by at most
2 d 2^-24 scale sum |q k| (twice the rounding, should partial sums be cut off), so with D the
largest such bound of a head's row and X its largest |logit|, an exponential is off by a
factor within 2 D + (8 X + 80 + k) 2^-24 (the reference exponent and its
argument's rounding, the function, the row's sum of k terms, the mean over
heads).  Loss: see _loss_tolerance."""
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


def _inputs(n, k, heads, groups, d, L, seed, pad=0.2, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    q = (sharp * torch.randn((n, heads, d), generator=g)).to(torch.bfloat16)
    keys = torch.randn((L, groups, d), generator=g).to(torch.bfloat16)
    idx = torch.randint(0, L, (n, k), generator=g, dtype=torch.int32)
    live = torch.randint(0, k + 1, (n,), generator=g)
    idx[(torch.arange(k) >= live[:, None]) & (torch.rand((n, 1), generator=g) < pad)] = -1
    return q, keys, idx


def _mass_check(out, q, keys, idx, scale, lse=None):
    q64, k64, ix = q.double().numpy(), keys.double().numpy(), idx.numpy()
    n, heads, d = q64.shape
    per = heads // k64.shape[1]
    out = out.double().cpu().numpy()
    lse64 = None if lse is None else lse.double().numpy()
    for i, (p, x) in enumerate(op.attention_probabilities(q64, k64, ix, scale, lse64)):
        live = np.isfinite(x[0])
        assert not out[i][~live].any(), i
        if not live.any():
            continue
        tol = np.zeros(ix.shape[1])
        for h in range(heads):
            ab = np.abs(k64[ix[i][live], h // per]) @ np.abs(q64[i, h]) * abs(scale)
            big = np.abs(x[h, live]).max() + (0 if lse is None else abs(lse64[i, h]))
            rel = 4 * d * U * ab.max() + (8 * big + 80 + ix.shape[1]) * U
            tol[live] += p[h, live] * rel
        err = np.abs(out[i] - p.mean(0))
        bad = err > tol / heads + 1e-37
        assert not bad.any(), (i, np.argwhere(bad)[0], err[bad][0], tol[bad][0] / heads)


CASES = [  # n, k, heads, key heads, d, L
    (1, 1, 1, 1, 64, 5), (3, 17, 5, 1, 128, 100), (2, 64, 64, 1, 128, 300), (1, 2048, 64, 1, 128, 3000),
    (4, 333, 32, 4, 64, 400), (2, 100, 40, 8, 128, 200), (3, 65, 16, 16, 96, 90), (2, 129, 128, 1, 576, 200),
    (2, 40, 20, 1, 512, 64), (5, 250, 24, 2, 256, 300), (2, 500, 144, 1, 192, 600), (1, 130, 256, 2, 64, 140),
    (70, 100, 8, 1, 64, 200), (1100, 20, 4, 2, 64, 64), (1030, 300, 33, 1, 64, 200), (1030, 90, 64, 1, 128, 100), (9, 16, 17, 1, 128, 40), (2, 15, 200, 200, 64, 33),
    (1, 70, 256, 1, 576, 90), (1, 33, 256, 2, 576, 50), (1, 2048, 128, 1, 576, 500), (2, 50, 1024, 2, 64, 60),
    (1, 40, 300, 3, 512, 60), (2, 300, 96, 1, 128, 200), (2, 90, 80, 1, 64, 70), (1, 200, 144, 1, 128, 150),
    (3, 33, 190, 2, 64, 40),
]


LONG = [  # enough queries for one workgroup each, k up to the longest: (k, heads, key heads, d)
    (2048, 64, 1, 128), (2047, 48, 1, 128), (1300, 16, 1, 64), (2000, 40, 2, 64), (777, 100, 1, 128),
    (2048, 8, 2, 64), (1025, 30, 1, 128), (640, 128, 2, 64), (129, 64, 1, 64), (700, 90, 1, 64), (300, 128, 1, 128), (200, 270, 2, 128),
]


@pytest.mark.parametrize("case", LONG)
def test_mass_of_long_rows_of_many_queries(hk, case):
    """One workgroup a query (over 512 queries): statistics and mass together, some of the logits and
    keys kept between them.  A few queries, padded ones among them, against the definition, every
    row's sum, and the same rows computed for few queries (several workgroups each)."""
    k, heads, groups, d = case
    n, L = 1030, 3000
    say(f"mass: {case} n={n}")
    q, keys, idx = _inputs(n, k, heads, groups, d, L, sum(case), pad=0.5)
    out = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda())
    some = torch.tensor([0, 1, 2, 500, 1029])
    _mass_check(out[some], q[some], keys, idx[some], d ** -0.5)
    few = hk.attention_mass(q[some].cuda(), keys.cuda(), idx[some].cuda())
    _mass_check(few, q[some], keys, idx[some], d ** -0.5)
    live = (idx >= 0).any(1)
    # a row's sum: k terms, each off by its bound above (below 2^-11 for these logits), and the sum itself
    total = out.double().sum(1).cpu()
    assert (total[live] - 1).abs().max() < 2.0 ** -11 and not total[~live].any()


@pytest.mark.parametrize("case", CASES)
def test_mass_matches_the_definition(hk, case):
    n, k, heads, groups, d, L = case
    say(f"mass: {case}")
    q, keys, idx = _inputs(n, k, heads, groups, d, L, sum(case))
    out = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda())
    _mass_check(out, q, keys, idx, d ** -0.5)
    # from the attention's own normaliser, over more keys than the selected ones
    lse = (torch.einsum("nhd,lhd->nhl", q.float(), keys.float().repeat_interleave(heads // groups, 1))
           * d ** -0.5).logsumexp(-1)
    out = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda(), lse=lse.cuda().contiguous())
    _mass_check(out, q, keys, idx, d ** -0.5, lse)


def test_mass_rows_of_padding_repeats_and_what_padding_points_at(hk):
    q, keys, idx = _inputs(6, 90, 8, 2, 64, 50, 3, pad=0.0)
    keys[7] = float("nan")               # a key that no row selects
    keys[0] = float("inf")
    idx[idx == 7] = 8
    idx[idx == 0] = 9
    idx[0] = -1                          # nothing selected
    idx[1, 1:] = torch.iinfo(torch.int32).min
    idx[2, ::2] = 50                     # outside the table
    idx[3] = 4                           # one key 90 times
    idx[4, 0:80] = -1                    # live entries at the end alone
    out = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda())
    _mass_check(out, q, keys, idx, 0.125)
    assert not out[0].any() and out[1, 0] == 1.0
    assert torch.allclose(out[3].cpu(), torch.full((90,), 1 / 90), rtol=1e-5)
    # a head whose attention saw nothing beside the entries: exp(x - (-inf)) shows, other rows do not change
    lse = torch.full((6, 8), 3.0)
    lse[5, 2] = float("inf")
    got = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda(), lse=lse.cuda())
    _mass_check(got[:5], q[:5], keys, idx[:5], 0.125, lse[:5])
    # a selected key of NaN shows in its own row alone
    idx[5, 3] = 7
    bad = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda())
    assert torch.isnan(bad[5]).any() and torch.equal(bad[:5], out[:5])


def test_mass_of_sharp_and_flat_rows(hk):
    """Logits over a range of thousands, rising along the row; a scale of 0."""
    n, k, d = 2, 400, 64
    q, keys, idx = _inputs(n, k, 16, 1, d, 400, 9, pad=0.0, sharp=40.0)
    keys = (keys.float() * torch.linspace(0.1, 30, 400)[:, None, None]).to(torch.bfloat16)
    idx[:] = torch.arange(400, dtype=torch.int32)
    out = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda(), softmax_scale=0.5)
    _mass_check(out, q, keys, idx, 0.5)
    flat = hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda(), softmax_scale=0.0)
    assert torch.allclose(flat.cpu(), torch.full((n, k), 1 / k), rtol=1e-5)


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_mass_of_padded_rows_at_any_scale(hk, scale):
    q, keys, idx = _inputs(5, 130, 24, 1, 128, 90, 15, pad=1.0)
    idx[:, 3::7] = -1
    _mass_check(hk.attention_mass(q.cuda(), keys.cuda(), idx.cuda(), softmax_scale=scale), q, keys, idx, scale)


def test_mass_is_the_same_bits_every_time_and_for_any_batch(hk):
    q, keys, idx = (t.cuda() for t in _inputs(40, 300, 64, 1, 128, 500, 11))
    a = hk.attention_mass(q, keys, idx)
    assert torch.equal(a, hk.attention_mass(q, keys, idx))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = hk.attention_mass(q, keys, idx)
    side.synchronize()
    assert torch.equal(a, b)
    nan_ws = torch.full((hk.attention_mass_workspace_bytes(q, keys, idx),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(a, hk.attention_mass(q, keys, idx, workspace=nan_ws))


def test_mass_behind_32_bit_offsets(hk):
    L = (1 << 25) + 50
    keys = torch.zeros((L, 1, 64), dtype=torch.bfloat16, device="cuda")
    q, few, _ = _inputs(3, 4, 8, 1, 64, 50, 13)
    keys[L - 50:] = few.cuda()
    idx = torch.randint(0, 50, (3, 40), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    far = hk.attention_mass(q.cuda(), keys, (idx + (L - 50)).cuda())
    assert torch.equal(far, hk.attention_mass(q.cuda(), few.cuda(), idx.cuda()))


def test_mass_of_a_table_beyond_64_gib(hk):
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB of GPU memory")
    L = (1 << 28) + 50
    keys = torch.empty((L, 1, 128), dtype=torch.bfloat16, device="cuda")
    q, few, _ = _inputs(3, 4, 20, 1, 128, 50, 14)
    keys[0] = 0
    keys[L - 50:] = few.cuda()
    idx = torch.randint(0, 50, (3, 70), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    idx[1, 30:] = -1
    far = hk.attention_mass(q.cuda(), keys, torch.where(idx < 0, idx, idx + (L - 50)).cuda())
    _mass_check(far, q, few, idx, 128 ** -0.5)
    del keys
    torch.cuda.empty_cache()


def _loss_tolerance(score, mass, weight):
    """fp32 error bound of loss and gradient, U = 2^-24.  With r = max - score of
    an entry and k terms: p is off by p (r + 80 + k/16) U (its argument's rounding, the
    exponential, the sum by 32 in a lane and 6 across), t by t (40 + k/16) U, ln t and ln p by that and 2 |ln| U
    more; the loss sums k terms t (ln t - ln p) - t + p whose parts are rounded once each."""
    n, k = score.shape
    tl, tg = np.zeros(n), np.zeros((n, k))
    for i in range(n):
        live = ~np.isneginf(score[i])
        total = mass[i][live].sum() if live.any() else 0
        if total == 0:
            continue
        t, s = mass[i][live] / total, score[i][live]
        m = s.max()
        z = np.log(np.exp(s - m).sum())
        p = np.exp(s - m - z)
        w = 1.0 if weight is None else abs(float(weight[i]))
        r = (m - s) + 80 + k / 16
        gerr = (p * r + t * (40 + k / 16)) * U
        tg[i][live] = w * (gerr + 4 * (p + t) * U)
        with np.errstate(divide="ignore"):
            ln = np.where(t > 0, np.abs(np.log(t)), 0) + np.abs(s - m) + z
        terms = t * ln * (8 + 40) * U + t * (120 + k / 8) * U + gerr + (p + t) * (8 + k / 16) * U
        tl[i] = w * (terms.sum() + 1e-37)
    return tl, tg + 1e-37


def _loss_check(hk, score, mass, weight=None):
    dev = [None if t is None else t.cuda() for t in (score, mass, weight)]
    loss, grad = hk.index_loss(dev[0], dev[1], weight=dev[2])
    s, m = score.double().numpy(), mass.double().numpy()
    w = None if weight is None else weight.double().numpy()
    rl, rg = op.index_loss(s, m, w)
    m = np.where(np.isneginf(s), 0.0, m)
    tl, tg = _loss_tolerance(s, m, w)
    el, eg = np.abs(loss.double().cpu().numpy() - rl), np.abs(grad.double().cpu().numpy() - rg)
    assert np.all(el <= tl), (np.argmax(el - tl), el.max())
    assert np.all(eg <= tg), (np.argwhere(eg > tg)[0],)
    assert not grad.cpu().numpy()[np.isneginf(s)].any()
    return loss, grad


@pytest.mark.parametrize("k", [1, 2, 4, 63, 64, 65, 255, 256, 257, 500, 513, 1000, 1024, 1025, 2047, 2048])
def test_loss_and_gradient_match_the_definition(hk, k):
    say(f"index loss: k {k}")
    g = torch.Generator().manual_seed(k)
    n = 13
    score = 3 * torch.randn((n, k), generator=g)
    mass = torch.exp(2 * torch.randn((n, k), generator=g))
    live = torch.randint(0, k + 1, (n,), generator=g)
    live[0], live[1], live[2] = k, 0, min(1, k)
    dead = torch.arange(k) >= live[:, None]
    score[dead] = -float("inf")
    mass[dead] = float("nan")             # padding may hold anything
    mass[4] = torch.where(dead[4], mass[4], torch.zeros(()))  # a live row without mass
    mass[5, : k // 2] = 0.0               # entries without mass
    weight = torch.rand(n, generator=g)
    loss, grad = _loss_check(hk, score, mass, weight)
    assert loss[1] == 0 and loss[4] == 0 and not grad[1].any() and not grad[4].any()
    _loss_check(hk, score, mass)


def test_loss_of_extreme_rows(hk):
    """Scores of the type's lowest value, far apart, equal; masses tiny and huge; a target that is the softmax."""
    low = torch.finfo(torch.float32).min
    score = torch.zeros(7, 40)
    mass = torch.ones(7, 40)
    score[0, 10:] = low                   # live, but with no probability
    mass[0, 10:] = 0.0
    score[1] = low                        # every entry at the lowest value: uniform
    score[2] = torch.linspace(-80, 0, 40)
    mass[3] = 1e-40                       # a subnormal sum
    mass[4] = 1e36
    score[5] = torch.randn(40, generator=torch.Generator().manual_seed(3))
    mass[5] = torch.exp(score[5])
    score[6] += 1e6
    loss, grad = _loss_check(hk, score, mass)
    assert abs(loss[5].item()) < 1e-5 and grad[5].abs().max() < 1e-6 and bool((loss > -1e-6).all())


def test_not_finite_rows_show_and_stay_alone(hk):
    score, mass = torch.zeros(4, 100), torch.ones(4, 100)
    score[1, 3] = float("nan")
    mass[2, 5] = float("nan")
    loss, grad = hk.index_loss(score.cuda(), mass.cuda())
    assert torch.isnan(loss[1:3]).all() and torch.isnan(grad[1:3]).all()
    assert torch.isfinite(loss[[0, 3]]).all() and torch.isfinite(grad[[0, 3]]).all()


def test_a_large_gradient_and_many_rows(hk):
    """Over 32 MiB of gradient (stored past the caches), rows of every live count."""
    g = torch.Generator().manual_seed(7)
    n, k = 4200, 2048
    score, mass = 2 * torch.randn((n, k), generator=g), torch.rand((n, k), generator=g)
    score[torch.arange(k) >= torch.arange(n)[:, None]] = -float("inf")
    loss, grad = hk.index_loss(score.cuda(), mass.cuda())
    some = torch.tensor([0, 1, 2, 63, 64, 1000, 2047, 2048, 4199])
    rl, rg = op.index_loss(score[some].double().numpy(), mass[some].double().numpy())
    tl, tg = _loss_tolerance(score[some].double().numpy(), mass[some].double().numpy(), None)
    assert np.all(np.abs(loss[some].double().cpu().numpy() - rl) <= tl)
    assert np.all(np.abs(grad[some].double().cpu().numpy() - rg) <= tg)
    # each row's gradient sums to 0: k terms within their bound
    assert grad.double().sum(1).abs().max() < 2.0 ** -14


def test_gradient_against_differences(hk):
    g = torch.Generator().manual_seed(5)
    score, mass = torch.randn((1, 30), generator=g), torch.rand((1, 30), generator=g)
    _, grad = hk.index_loss(score.cuda(), mass.cuda())
    # a difference over h = 2^-6 leaves h^2/6 of a third derivative below 1, and the
    # rounding of two losses (within 1e-5) over 2 h
    h = 2.0 ** -6
    for j in range(0, 30, 7):
        up, down = score.clone(), score.clone()
        up[0, j] += h
        down[0, j] -= h
        num = (hk.index_loss(up.cuda(), mass.cuda())[0] - hk.index_loss(down.cuda(), mass.cuda())[0]).item() / (2 * h)
        assert abs(num - grad[0, j].item()) < h * h / 6 + 1e-5 / h


def test_loss_outputs_aliases_and_unaligned_rows(hk):
    g = torch.Generator().manual_seed(6)
    score, mass = torch.randn((9, 64), generator=g).cuda(), torch.rand((9, 64), generator=g).cuda()
    loss, grad = hk.index_loss(score, mass)
    a, b = hk.index_loss(score, mass, want=("loss",))
    assert b is None and torch.equal(a, loss)
    a, b = hk.index_loss(score, mass, want=("d_score",))
    assert a is None and torch.equal(b, grad)
    for target in (score.clone(), mass.clone()):  # the gradient over its own input
        s = target if torch.equal(target, score) else score
        m = mass if s is target else target
        _, got = hk.index_loss(s, m, out=(None, target))
        assert got is target and torch.equal(got, grad)
    off = torch.empty(9 * 64 + 1, device="cuda")[1:].view(9, 64)
    off.copy_(score)
    l2, g2 = hk.index_loss(off, mass)
    assert torch.allclose(l2, loss, rtol=1e-5, atol=1e-6) and torch.allclose(g2, grad, rtol=1e-5, atol=1e-7)
    l0, g0 = hk.index_loss(score[:0], mass[:0])
    assert l0.shape == (0,) and g0.shape == (0, 64)


BY_KEY = [  # rows long enough, of many queries on many keys, that their entries are walked by key:
    # k, heads, key heads, d, L
    (1024, 64, 1, 128, 33000), (2047, 5, 1, 64, 66001), (1500, 40, 4, 64, 20000), (2048, 48, 1, 128, 131072),
    (1030, 100, 2, 128, 17000), (1777, 32, 1, 64, 70000), (1100, 17, 1, 128, 40000), (1200, 33, 3, 64, 30000),
]


@pytest.mark.parametrize("case", BY_KEY)
def test_mass_of_entries_in_any_order(hk, case):
    """Rows sorted by key, reversed, of one key, of one bucket, with padding of both signs anywhere, the last
    key among them: each entry's mass comes back at its own place, and the same bits every time."""
    k, heads, groups, d, L = case
    n = 600
    say(f"mass by key: {case}")
    q, keys, idx = _inputs(n, k, heads, groups, d, L, sum(case) + 1, pad=0.0)
    idx[0] = idx[0].sort().values
    idx[1] = idx[1].sort(descending=True).values
    idx[2] = L - 1
    idx[3] = torch.arange(k, dtype=torch.int32) % 200
    idx[4, ::3] = -7
    idx[4, 1::5] = L
    idx[5] = 2 ** 31 - 1
    idx[6, :-1] = -1
    idx[7, 1:] = -(2 ** 31)
    idx[8] = L - 1 - torch.arange(k, dtype=torch.int32)
    idx[9, 64:] = -1
    g = torch.Generator().manual_seed(3)
    lse = (torch.rand((n, heads), generator=g) * 3 + 8)
    dev = [t.cuda() for t in (q, keys, idx)]
    out = hk.attention_mass(*dev)
    given = hk.attention_mass(*dev, lse=lse.cuda())
    some = torch.cat([torch.arange(10), torch.tensor([300, n - 1])])
    _mass_check(out[some], q[some], keys, idx[some], d ** -0.5)
    _mass_check(given[some], q[some], keys, idx[some], d ** -0.5, lse[some])
    assert torch.equal(out, hk.attention_mass(*dev)) and torch.equal(given, hk.attention_mass(*dev, lse=lse.cuda()))
    dead = (idx < 0) | (idx >= L)
    assert not out.cpu()[dead].any() and not given.cpu()[dead].any()


@pytest.mark.parametrize("n,k,heads,groups,d", [(5, 700, 16, 1, 128), (600, 200, 32, 4, 64), (301, 500, 32, 4, 64), (3, 150, 200, 2, 64)])
def test_mass_of_rows_that_end_early(hk, n, k, heads, groups, d):
    """Blocks behind a row's last entry are left out: rows that end before, at and behind a block, and a
    split without an entry."""
    q, keys, idx = _inputs(n, k, heads, groups, d, 900, 77, pad=0.0)
    ends = [0, 1, 15, 16, 17, 63, 64, 65, k - 1, k]
    for i in range(n):
        idx[i, ends[i % len(ends)]:] = -1
    idx[min(n - 1, 2), k - 1] = 5  # one entry at the very end
    lse = torch.full((n, heads), 9.0)
    some = torch.arange(min(n, 12))
    dev = [t.cuda() for t in (q, keys, idx)]
    _mass_check(hk.attention_mass(*dev)[some], q[some], keys, idx[some], d ** -0.5)
    given = hk.attention_mass(*dev, lse=lse.cuda())
    _mass_check(given[some], q[some], keys, idx[some], d ** -0.5, lse[some])
    assert not given.cpu()[idx < 0].any()
