"""The table's gradient of buckets that weigh little in the softmax keeps fp32
accuracy relative to its own size: the error that the bf16 rounding of o puts into D
is taken out of them too.

Per pair, P is off by at most four roundings of its exponent (|t| <= 64 in the log2
domain: score, bias, lse), 4 2^-24 64 ln 2 < 2^-16 of P, and dP and D by the fp32
sums of their 64 products, 2^-20 of the products' size; sums over pairs add little."""
import numpy as np
import pytest

from tests.gpu_util import sync
from tests.test_gpu_window_distill import HD, Case, b, buckets_by_distance, np64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low", [0.0, -10.0, -14.0, -18.0])
@pytest.mark.parametrize("shape", [
    # nseq, seq, window, sinks, buckets, max_distance, lens
    (1, 300, 300, 0, 8, 60, None),          # every kind of tile
    (2, 700, 700, 0, 32, 128, [700, 333]),
    (1, 1500, 1500, 0, 8, 2000, None),      # two buckets a row
    (1, 700, 100, 20, 32, 600, None),       # the sinks' buckets
])
def test_faint_buckets(b, shape, low):  # noqa: F811
    nseq, seq, window, sinks, buckets, md, lens = shape
    t = np.random.default_rng(9).standard_normal((buckets, 1)).astype(np.float32)
    t[1::2] += low
    c = Case(b, nseq, seq, 1, 1, window, sinks, buckets, md, lens=lens, table=t)
    c.dtable.zero_()
    c.fwd()
    c.bwd()
    sync()
    want, tol = np.zeros(buckets + 1), np.zeros(buckets + 1)
    of = buckets_by_distance(seq, buckets, md)
    x, do = np64(c.qkv).reshape(nseq, seq, 3, HD), np64(c.do).reshape(nseq, seq, HD)
    for i, _, n, ref in c.refs():
        v, g = x[i, :n, 2], do[i, :n]
        dp, d = g @ v.T, (g * ref.o).sum(1, keepdims=True)
        size = np.abs(g) @ np.abs(v).T + (np.abs(g) * (ref.p @ np.abs(v))).sum(1, keepdims=True)
        dist = np.arange(n)[:, None] - np.arange(n)[None, :]
        flat = np.where(dist >= 0, of[:n][np.clip(dist, 0, None)], buckets).ravel()
        want += np.bincount(flat, weights=ref.ds.ravel(), minlength=buckets + 1)
        err = ref.p * (2.0 ** -16 * (np.abs(dp) + np.abs(d)) + 2.0 ** -20 * size)
        tol += np.bincount(flat, weights=err.ravel(), minlength=buckets + 1)
    err = np.abs(np64(c.dtable)[:, 0] - want[:buckets])
    assert np.all(err <= tol[:buckets]), np.max(err / np.maximum(tol[:buckets], 1e-30))
