"""Windowed attention under tables with large finite entries, against fp64.

A row's softmax does not change when the largest entry that the row sees, its
base, is taken out of all of its scores; lse gets it back.  The bounds are those
of the other attention tests (one rounding to bf16, 2^-8 relative, for each of P,
dS, o and the results; D from the rounded o), with the fp32 slack counted from
the scores without the base: an entry of -1e9 that a row sees alone costs it
nothing.  Pairs 2^-200 below their row's largest have P = 0 in fp32 whatever
their score is rounded to.
"""
import numpy as np
import pytest

from tests.gpu_util import sync
from tests.test_gpu_window_distill import HD, U, Case, b, buckets_by_distance, np64  # noqa: F401

pytestmark = pytest.mark.gpu


class Shifted:
    """One (sequence, head) in fp64, every row relative to its base."""

    def __init__(self, q, k, v, do, window, sinks, bias, of):
        n = q.shape[0]
        i, j = np.arange(n)[:, None], np.arange(n)[None, :]
        see = (j <= i) & ((i - j < window) | (j < sinks))
        hide = bias <= -1e30
        of = of[:n][np.clip(i - j, 0, None)]
        see = see & ~hide[of]
        t = np.where(hide, 0.0, bias)[of]
        base = np.max(np.where(see, t, -np.inf), axis=1, initial=-np.inf, keepdims=True)
        none = ~np.isfinite(base)
        base = np.where(none, 0.0, base)
        s = np.where(see, q @ k.T / 8.0 + (t - base), -np.inf)
        m = np.max(s, axis=1, initial=-np.inf, keepdims=True)
        m = np.where(none, 0.0, m)
        e = np.exp(s - m)
        l = e.sum(1, keepdims=True)
        with np.errstate(divide="ignore"):
            rest = m + np.log(l)
        self.lse = (base + rest)[:, 0]
        p = self.p = e / np.where(l > 0, l, 1.0)
        self.o = p @ v
        counts = see & (s > m - 200 * np.log(2.0))
        size = np.where(counts, np.abs(q) @ np.abs(k).T / 8.0 + np.abs(t - base), 0.0)
        # entries of up to 256 stay in the scores
        big = size.max(initial=0.0) + np.max(np.abs(rest[~none]), initial=0.0) + 256.0 * bool((np.abs(base) <= 256).any())
        eps = 8 * (big * 1.4427 * 2.0 ** -24 * 4 + size.max(initial=0.0) * 64 * 2.0 ** -24 + 2.0 ** -22)
        self.lse_tol = (eps + (n + 64) * 2.0 ** -24 + 2.0 ** -23 * np.abs(np.where(none, 0.0, base)))[:, 0][~none[:, 0]]
        pv = p @ np.abs(v)
        self.o_tol = U * (np.abs(self.o) + pv) * 1.01 + (eps + n * 2.0 ** -24) * pv
        dp = do @ v.T
        D = (do * self.o).sum(1, keepdims=True)
        ds = p * (dp - D)
        mag = p * (np.abs(do) @ np.abs(v).T + np.abs(do * self.o).sum(1, keepdims=True))
        dD = (self.o_tol * np.abs(do)).sum(1, keepdims=True)
        slack = eps * mag
        ds_tol = U * np.abs(ds) * 1.01 + p * dD * 1.01 + slack
        acc = (n + 64) * 2.0 ** -24
        self.dq = ds @ k / 8.0
        self.dq_tol = (ds_tol + acc * np.abs(ds)) @ np.abs(k) / 8.0
        self.dk = ds.T @ q / 8.0
        self.dk_tol = (ds_tol + acc * np.abs(ds)).T @ np.abs(q) / 8.0
        self.dv = p.T @ do
        self.dv_tol = (U * 1.01 + eps + acc) * p.T @ np.abs(do)
        nb = len(bias)
        flat = np.where(i >= j, of, nb).ravel()
        self.dt = np.bincount(flat, weights=ds.ravel(), minlength=nb + 1)[:nb]
        tol = slack * 2 + (np.abs(ds) + p * dD) * (n + 512) * 2.0 ** -24 + p * dD * eps * 2
        self.dt_tol = np.bincount(flat, weights=tol.ravel(), minlength=nb + 1)[:nb]


class LargeCase(Case):
    def refs(self):
        n, s, h, kv, w, si, nb, md = self.shape
        x, do, table = np64(self.qkv).reshape(n, s, -1, HD), np64(self.do).reshape(n, s, h, HD), np64(self.table)
        of = buckets_by_distance(s, nb, md)
        for i in range(n):
            ln = min(max(self.lens[i], 0), s)
            for j in range(h):
                g = j // (h // kv)
                yield i, j, ln, Shifted(x[i, :ln, j], x[i, :ln, h + g], x[i, :ln, h + kv + g], do[i, :ln, j], w, si,
                                        table[:, j], of)


def table_of(which, value, buckets, heads):
    """Small entries but for the first head's (the second keeps its own)."""
    t = np.random.default_rng(5).standard_normal((buckets, heads)).astype(np.float32)
    if which == "first":       # the first query sees this bucket alone
        t[0, 0] = value
    elif which == "last":
        t[-1, 0] = value
    elif which == "near":      # the first rows see nothing but these
        t[:buckets // 2, 0] = value
    elif which == "all":       # a common offset
        t[:, 0] += value
    else:                      # far apart from each other
        t[:, 0] = value * (1 + np.arange(buckets) % 3)
    return t


SHAPES = [
    # nseq, seq, heads, kv, window, sinks, buckets, max_distance, lens
    (1, 150, 2, 1, 1, 0, 8, 40, None),           # each query sees itself alone
    (2, 150, 2, 2, 70, 3, 8, 40, [150, 90]),
    (1, 400, 3, 1, 100, 20, 32, 300, None),      # sinks far from their queries, in buckets of their own
    (1, 700, 2, 1, 700, 0, 8, 600, None),        # wide buckets
]


@pytest.mark.parametrize("value", [-1e4, -1e6, -1e9, 1e4, 1e6, -300.0, 300.0, 200.0])
@pytest.mark.parametrize("which", ["first", "last", "near", "all", "apart"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(x) for x in s[:8]))
def test_large_entries(b, shape, which, value):  # noqa: F811
    c = LargeCase(b, *shape[:8], lens=shape[8], table=table_of(which, value, shape[6], shape[2]))
    c.fwd()
    c.bwd()
    c.check()


def test_large_entries_among_hidden_ones(b):  # noqa: F811
    t = table_of("near", -1e9, 8, 2)
    t[0, 0], t[2, 0], t[5, 1] = -np.inf, -np.finfo(np.float32).max, -1e30
    c = LargeCase(b, 2, 150, 2, 1, 70, 3, 8, 40, lens=[150, 90], table=t)
    c.fwd()
    c.bwd()
    c.check()


def test_largest_entries(b):  # noqa: F811
    t = table_of("first", 3e38, 8, 2)
    t[1, 0], t[0, 1] = -9e29, -9.9e29
    c = LargeCase(b, 1, 150, 2, 1, 70, 3, 8, 40, table=t)
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(x) for x in s[:8]))
def test_a_large_entry_leaves_the_other_heads_and_a_frozen_table_as_they_are(b, shape):  # noqa: F811
    """Gradients without the table's are the same bits; a head without large entries
    does not see that another has them."""
    import torch
    c = LargeCase(b, *shape[:8], lens=shape[8], table=table_of("near", -1e6, shape[6], shape[2]))
    c.fwd()
    c.bwd()
    sync()
    first, c.dtable = c.dqkv.clone(), None
    c.dqkv.fill_(7.0)
    c.bwd()
    sync()
    assert torch.equal(first, c.dqkv)
    rows = shape[0] * shape[1]
    o, lse, heads = c.o[:rows].clone(), c.lse[:rows].clone(), shape[2]
    c.table[:, 0] = 0.0
    c.fwd()
    c.bwd()
    sync()
    assert torch.equal(o.view(rows, heads, HD)[:, 1:], c.o[:rows].view(rows, heads, HD)[:, 1:])
    assert torch.equal(lse[:, 1:], c.lse[:rows, 1:])
    assert torch.equal(first[:rows, HD:heads * HD], c.dqkv[:rows, HD:heads * HD])


@pytest.mark.parametrize("value", [-300.0, -280.0, 1e4])
@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: "x".join(str(x) for x in s[:8]))
def test_large_scores_against_large_entries(b, shape, value):  # noqa: F811
    """Scores of some 290 on the diagonal: with entries of -300 a row's lse is small
    although its base is large, with larger ones it is not."""
    c = LargeCase(b, *shape[:8], lens=shape[8], table=table_of("all", value, shape[6], shape[2]))
    cols = shape[2] + shape[3]   # queries and keys, made alike so that each row's own key has the largest score
    x = c.qkv.view(shape[0] * shape[1], -1, HD)
    x[:, :shape[2]] = x[:, shape[2]:cols].repeat_interleave(shape[2] // shape[3], 1)
    x[:, :cols] *= 6
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("scale", [6.0, 30.0])
def test_large_scores(b, scale):  # noqa: F811
    """The bounds grow with the scores, as fp32 does."""
    c = Case(b, 2, 200, 2, 1, 90, 3, 8, 40, lens=[200, 77])
    c.qkv[:, :3 * HD] *= scale
    c.fwd()
    c.bwd()
    c.check()
