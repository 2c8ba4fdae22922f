"""CPU fp64 definitions of the operators around the selection: layer norm, rotary
positions, the attention's mass at the selected entries, the indexer's loss.

TEST INFRASTRUCTURE ONLY (see ``oracle.oracle``).  The storage formats'
quantisers are ``datagen``'s and their decoders ``oracle.decode_*``.
"""
from __future__ import annotations

import numpy as np

__all__ = ["rotary_frequencies", "rotary_plan", "rotary", "layer_norm", "layer_norm_backward",
           "attention_probabilities", "attention_mass", "index_loss"]


def rotary_frequencies(dim: int, base: float = 10000.0) -> np.ndarray:
    """base^(-2i/dim) for i = 0 .. dim/2 - 1."""
    return float(base) ** (-2.0 * np.arange(dim // 2) / dim)


def rotary_plan(dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: int = 0):
    """(frequencies, factor on the rotated part).  NTK: the base at which the slowest pair comes out divided by
    the factor.  YaRN: per pair a share of f / factor that rises along the pairs' numbers, from the last whole
    number at which a pair still makes 32 turns in the original context to the first at which it makes one or less
    (within 0 .. dim - 1); where every pair makes one or less, all are divided."""
    if scaling == "none":
        return rotary_frequencies(dim, base), 1.0
    if scaling == "linear":
        return rotary_frequencies(dim, base) / factor, 1.0
    if scaling == "ntk":
        return rotary_frequencies(dim, base * factor ** (dim / max(dim - 2, 1))), 1.0
    f = rotary_frequencies(dim, base)
    # original base^(-2 x / dim) = 2 pi turns, solved for x
    many, one = (0.5 * dim * np.log(original / (2 * np.pi * turns)) / np.log(base) for turns in (32, 1))
    a, b = max(np.floor(many), 0.0), min(np.ceil(one), dim - 1.0)
    share = np.empty(dim // 2)
    for i in range(dim // 2):
        if one <= 0 or i >= max(b, a + 1e-3):
            share[i] = 1.0
        else:
            share[i] = 0.0 if i <= a else (i - a) / (b - a)
    return f * ((1 - share) + share / factor), 1 + np.log(factor) / 10


def rotary(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, *, first: int = 0,
           layout: str = "half", gain: float = 1.0, backward: bool = False, axis=None) -> np.ndarray:
    """x [n][heads][d]: pair i = (a, b) of elements first .. first + dim - 1
    becomes gain * (a cos - b sin, b cos + a sin) at angle pos * freq[i];
    backward applies the transpose.  With ``axis`` [dim/2] pos is [n][axes] and pair i turns by its own axis' position."""
    half = len(freq)
    pos = pos[:, axis] if axis is not None else pos[:, None]
    # the angle as turns in extended precision, so that far positions keep theirs
    turns = pos.astype(np.longdouble) * freq.astype(np.longdouble) / (2 * np.longdouble(np.pi)
                                                                               + np.longdouble(2.4492935982947064e-16))
    ang = ((turns - np.rint(turns)) * 2 * np.longdouble(np.pi)).astype(np.float64)
    c, s = gain * np.cos(ang)[:, None], gain * np.sin(ang)[:, None]
    if backward:
        s = -s
    i = np.arange(half)
    ia, ib = (first + i, first + half + i) if layout == "half" else (first + 2 * i, first + 2 * i + 1)
    y = np.array(x, dtype=np.float64)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def layer_norm(x, weight, bias, eps: float):
    """Rows x [..., d] in fp64: (y, mean [...], rstd [...])."""
    mean = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    return (x - mean) * rstd * weight + bias, mean[..., 0], rstd[..., 0]


def layer_norm_backward(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias) of rows in fp64 with the statistics given: the derivative of sum(dy * y) where mean and rstd are
    x's own."""
    h = (x - mean[..., None]) * rstd[..., None]
    g = dy * weight
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * h).sum(rows), dy.sum(rows)


def attention_probabilities(q, k, idx, scale: float, lse=None):
    """Per query, probabilities [heads][k] and logits [heads][k] of its entries (0 and
    -inf at padding).  q [n][heads][d], k [L][key_heads][d], idx [n][k]."""
    n, heads, _ = q.shape
    per = heads // k.shape[1]
    L = k.shape[0]
    for i in range(n):
        live = (idx[i] >= 0) & (idx[i] < L)
        x = np.full((heads, idx.shape[1]), -np.inf)
        for h in range(heads):
            x[h, live] = (k[idx[i][live], h // per] @ q[i, h]) * scale
        p = np.zeros_like(x)
        if live.any():
            if lse is None:
                e = np.exp(x - x.max(1, keepdims=True))
                p = e / e.sum(1, keepdims=True)
            else:
                with np.errstate(over="ignore"):
                    p = np.exp(x - lse[i][:, None])
        yield p, x


def attention_mass(q, k, idx, scale: float, lse=None) -> np.ndarray:
    """Mean over heads of the attention's probability at every entry."""
    return np.stack([p.mean(0) for p, _ in attention_probabilities(q, k, idx, scale, lse)])


def index_loss(score: np.ndarray, mass: np.ndarray, weight=None):
    """(loss [n], d_score [n][k]): divergence of softmax(score) from
    mass / sum(mass) over the live entries (score other than -inf)."""
    score, mass = np.asarray(score, np.float64), np.asarray(mass, np.float64)
    n, k = score.shape
    loss, grad = np.zeros(n), np.zeros((n, k))
    for i in range(n):
        live = ~np.isneginf(score[i])
        total = mass[i][live].sum() if live.any() else 0.0
        if total == 0.0:
            continue
        t = mass[i][live] / total
        s = score[i][live]
        m = s.max()
        logp = (s - m) - np.log(np.exp(s - m).sum())
        with np.errstate(divide="ignore", invalid="ignore"):
            terms = np.where(t > 0, t * (np.log(t) - logp), 0.0)
        w = 1.0 if weight is None else float(weight[i])
        loss[i] = w * terms.sum()
        grad[i][live] = w * (np.exp(logp) - t)
    return loss, grad
