"""Pins of the fp64 definitions in oracle.operators: closed forms, invariants
and differences."""
import numpy as np
import pytest

from oracle import operators as op


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_relative_positions(layout):
    rng = np.random.default_rng(1)
    f = op.rotary_frequencies(8)
    x, y = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))

    def dot(p, q):
        return float((op.rotary(x, np.array([p]), f, layout=layout)
                      * op.rotary(y, np.array([q]), f, layout=layout)).sum())
    assert abs(dot(7, 3) - dot(1007, 1003)) < 1e-12
    r = op.rotary(x, np.array([12345]), f, layout=layout)
    assert abs((r ** 2).sum() - (x ** 2).sum()) < 1e-12
    # pair 0 turns by one radian a position
    a, b = (0, 4) if layout == "half" else (0, 1)
    one = np.zeros((1, 1, 8))
    one[..., a] = 1.0
    r = op.rotary(one, np.array([2]), f, layout=layout)
    assert np.allclose([r[0, 0, a], r[0, 0, b]], [np.cos(2.0), np.sin(2.0)], atol=1e-15)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_backward_is_the_gradient(layout):
    rng = np.random.default_rng(2)
    f = op.rotary_frequencies(6)
    x, g = rng.standard_normal((3, 2, 10)), rng.standard_normal((3, 2, 10))
    pos = np.array([0, 5, 100000])
    kw = dict(first=2, layout=layout, gain=1.25)
    dx = op.rotary(g, pos, f, backward=True, **kw)
    for at in [(0, 0, 0), (1, 1, 2), (2, 0, 5), (2, 1, 7), (1, 0, 9)]:
        e = np.zeros_like(x)
        e[at] = 1e-4
        num = ((op.rotary(x + e, pos, f, **kw) - op.rotary(x - e, pos, f, **kw)) * g).sum() / 2e-4
        assert abs(num - dx[at]) < 1e-9


def test_attention_mass_sums_to_one_and_skips_padding():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 4, 16)), rng.standard_normal((9, 2, 16))
    idx = np.array([[3, 8, -1, 0], [-1, -1, 9, 100]])
    m = op.attention_mass(q, k, idx, 0.25)
    assert abs(m[0].sum() - 1) < 1e-14 and m[0, 2] == 0 and not m[1].any()
    lse = np.stack([np.log(np.exp(x[:, np.isfinite(x[0])]).sum(1) + 1e-300)
                    for _, x in op.attention_probabilities(q, k, idx, 0.25)])
    assert np.allclose(op.attention_mass(q, k, idx, 0.25, lse)[0], m[0], atol=1e-14)


def test_index_loss_gradient_matches_differences():
    rng = np.random.default_rng(4)
    s, m = rng.standard_normal((3, 5)), rng.random((3, 5))
    s[1, 3:] = -np.inf
    m[1, 3:] = np.nan   # dead entries may hold anything
    s[2] = -np.inf
    w = np.array([1.0, 0.5, 2.0])
    loss, grad = op.index_loss(s, m, w)
    assert loss[2] == 0 and not grad[2].any() and (loss[:2] > 0).all()
    for i, j in [(0, 0), (0, 4), (1, 2)]:
        e = np.zeros_like(s)
        e[i, j] = 1e-5
        num = (op.index_loss(s + e, m, w)[0] - op.index_loss(s - e, m, w)[0]).sum() / 2e-5
        assert abs(num - grad[i, j]) < 1e-8
    # the loss is 0 where the softmax is the target, and only there
    z = rng.standard_normal((1, 6))
    l0, g0 = op.index_loss(z, np.exp(z) * 3.0)
    assert abs(l0[0]) < 1e-14 and np.abs(g0).max() < 1e-14
