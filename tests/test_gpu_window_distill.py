"""Windowed attention with position buckets and the distillation loss against
plain fp64 forms (numpy), element by element, with bounds counted from the
roundings the kernels make.

Attention.  u = 2^-8 is half a bf16 step, relative.  The kernel rounds P (for
P V), dS (for dQ, dK) and P (for dV) to bf16 before the products and the results
afterwards, and D = rowsum(dO o O) starts from the rounded O:
  |o  - ref| <= u (|o| + P |V|) + slack
  |dV - ref| <= u (|dV| + P^T |dO|) + slack
  dD_i       <= sum_c u (|o_ic| + (P |V|)_ic) |dO_ic| + slack
  |dS - ref| <= u |dS| + P dD + slack
  |dQ - ref| <= u |dQ| + (bound of dS) |K| / 8,   dK alike with |Q|.
slack: P itself is off by a relative e_P from fp32 arithmetic in the exponent,
|t| 2^-24 for each of a handful of roundings of a value of size |t| (scores, bias
and log-sum-exp in the log2 domain), plus 64 2^-24 of the summed products' size,
plus 2^-22 of the exponential; it is taken as 8 times the largest such size.
The table's gradient keeps dS in fp32 and corrects D, so it has the slack alone,
and a rounding per addition: 2^-24 (seq + 512) of the summed magnitudes.
"""
import numpy as np
import pytest

from tests.gpu_util import KEEP, dev, host, sync
from tests.gpu_util import stream as cur_stream

pytestmark = pytest.mark.gpu
HD = 64
U = 2.0 ** -8


@pytest.fixture(scope="module")
def b():
    import __graft_entry__ as ge
    ge.build()
    from micro_pipeline_re_gb300 import binding
    return binding


def T():
    import torch
    return torch


def np64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def buckets_by_distance(n, buckets, max_distance):
    """Bucket of every distance below n, in whole numbers."""
    e = buckets // 2
    m, out = buckets - e, []
    for d in range(n):
        k = 0
        while d >= e and k + 1 < m and d ** m >= max_distance ** (k + 1) * e ** (m - k - 1):
            k += 1
        out.append(d if d < e else e + k)
    return np.array(out, dtype=int)


class Ref:
    """One (sequence, head) of the attention in fp64, with the bounds."""

    def __init__(self, q, k, v, do, window, sinks, bias, of):
        n = q.shape[0]
        i, j = np.arange(n)[:, None], np.arange(n)[None, :]
        see = (j <= i) & ((i - j < window) | (j < sinks))
        s = q @ k.T / 8.0
        size = np.abs(q) @ np.abs(k).T / 8.0
        if bias is not None:
            hide = bias <= -1e30
            bb = np.where(hide, 0.0, bias)[of[:n]]
            see = see & ~hide[of[:n]][np.clip(i - j, 0, None)]
            s = s + bb[np.clip(i - j, 0, None)]
            size = size + np.abs(bb)[np.clip(i - j, 0, None)]
        s = np.where(see, s, -np.inf)
        m = np.max(s, axis=1, initial=-np.inf, keepdims=True)
        ms = np.where(np.isfinite(m), m, 0.0)
        e = np.exp(s - ms)
        l = e.sum(1, keepdims=True)
        with np.errstate(divide="ignore"):
            self.lse = (ms + np.log(l))[:, 0]
        p = self.p = e / np.where(l > 0, l, 1.0)
        self.o = p @ v
        big = np.max(np.where(see, size, 0.0), initial=0.0) + np.max(np.abs(self.lse[np.isfinite(self.lse)]), initial=0.0)
        self.eps = eps = 8 * (big * 1.4427 * 2.0 ** -24 * 4 + size.max(initial=0.0) * 64 * 2.0 ** -24 + 2.0 ** -22)
        self.lse_tol = eps + (n + 64) * 2.0 ** -24
        pv = p @ np.abs(v)
        self.o_tol = U * (np.abs(self.o) + pv) * 1.01 + (eps + n * 2.0 ** -24) * pv
        if do is None:
            return
        dp = do @ v.T
        D = (do * self.o).sum(1, keepdims=True)
        ds = self.ds = p * (dp - D)
        mag = p * (np.abs(do) @ np.abs(v).T + np.abs(do * self.o).sum(1, keepdims=True))
        dD = (self.o_tol * np.abs(do)).sum(1, keepdims=True)
        self.ds_slack = ds_slack = eps * mag
        ds_tol = U * np.abs(ds) * 1.01 + p * dD * 1.01 + ds_slack
        acc = (n + 64) * 2.0 ** -24
        self.dq = ds @ k / 8.0
        self.dq_tol = (ds_tol + acc * np.abs(ds)) @ np.abs(k) / 8.0
        self.dk = ds.T @ q / 8.0
        self.dk_tol = (ds_tol + acc * np.abs(ds)).T @ np.abs(q) / 8.0
        self.dv = p.T @ do
        self.dv_tol = (U * 1.01 + eps + acc) * p.T @ np.abs(do)
        if bias is not None:
            nb = len(bias)
            flat = np.where(i >= j, of[:n][np.clip(i - j, 0, None)], nb).ravel()
            self.dt = np.bincount(flat, weights=ds.ravel(), minlength=nb + 1)[:nb]
            # the correction's own error: the error of D times that of P, and the rounding of its sums
            tol = ds_slack * 2 + (np.abs(ds) + p * dD) * (n + 512) * 2.0 ** -24 + p * dD * eps * 2
            self.dt_tol = np.bincount(flat, weights=tol.ravel(), minlength=nb + 1)[:nb]


class Case:
    """Device inputs of one call and its outputs; padded rows hold NaN."""

    def __init__(self, b, nseq, seq, heads, kv, window, sinks, buckets=0, md=0, lens=None, table=None, seed=0):
        t = T()
        self.b, self.shape = b, (nseq, seq, heads, kv, window, sinks, buckets, md)
        self.lens = [seq] * nseq if lens is None else lens
        rng = np.random.default_rng(seed + nseq * 7 + seq * 13 + heads)
        self.cols = cols = (heads + 2 * kv) * HD
        self.qkv = t.from_numpy(rng.standard_normal((nseq * seq, cols)).astype(np.float32)).cuda().bfloat16()
        self.do = t.from_numpy(rng.standard_normal((nseq * seq, heads * HD)).astype(np.float32)).cuda().bfloat16()
        for s, n in enumerate(self.lens):
            n = min(max(n, 0), seq)
            self.qkv[s * seq + n:(s + 1) * seq] = float("nan")
            self.do[s * seq + n:(s + 1) * seq] = float("nan")
        self.dlens = None if lens is None else dev(np.array(lens, dtype=np.int32))
        if buckets and table is None:
            table = rng.standard_normal((buckets, heads)) - 2.0 * np.arange(buckets)[:, None] / buckets
        self.table = None if table is None else dev(np.asarray(table, dtype=np.float32))
        # outputs with rows behind the last sequence, which stay as they were
        self.o = t.full((nseq * seq + 3, heads * HD), 7.0, device="cuda", dtype=t.bfloat16)
        self.lse = t.full((nseq * seq + 3, heads), 7.0, device="cuda")
        self.dqkv = t.full((nseq * seq + 3, cols), 7.0, device="cuda", dtype=t.bfloat16)
        self.dtable0 = rng.standard_normal((buckets, heads)).astype(np.float32) if buckets else None
        self.dtable = dev(self.dtable0) if buckets else None
        size = b.lib().gpipe_op_attention_window_scratch_bytes(nseq, seq, heads, window, sinks, buckets)
        self.size = size
        self.scratch = t.full((size + 256,), 0xFF, device="cuda", dtype=t.uint8)   # NaN wherever it is read unwritten
        KEEP.append(self)

    def fwd(self, stream=None):
        n, s, h, kv, w, si, nb, md = self.shape
        rc = self.b.lib().gpipe_op_attention_window_fwd(
            n, s, h, kv, w, si, self.b._ptr(self.dlens), self.b._ptr(self.table), nb, md, self.qkv.data_ptr(),
            self.o.data_ptr(), self.lse.data_ptr(), cur_stream() if stream is None else stream)
        assert rc == 0, self.b.lib().gpipe_last_error(None)

    def bwd(self, stream=None):
        n, s, h, kv, w, si, nb, md = self.shape
        rc = self.b.lib().gpipe_op_attention_window_bwd(
            n, s, h, kv, w, si, self.b._ptr(self.dlens), self.b._ptr(self.table), nb, md, self.qkv.data_ptr(),
            self.o.data_ptr(), self.do.data_ptr(), self.lse.data_ptr(), self.dqkv.data_ptr(),
            self.b._ptr(self.dtable), self.scratch.data_ptr(), cur_stream() if stream is None else stream)
        assert rc == 0, self.b.lib().gpipe_last_error(None)

    def refs(self):
        n, s, h, kv, w, si, nb, md = self.shape
        x, do = np64(self.qkv).reshape(n, s, -1, HD), np64(self.do).reshape(n, s, h, HD)
        table = None if self.table is None else np64(self.table)
        of = buckets_by_distance(s, nb, md) if nb else None
        for i in range(n):
            ln = min(max(self.lens[i], 0), s)
            for j in range(h):
                g = j // (h // kv)
                yield i, j, ln, Ref(x[i, :ln, j], x[i, :ln, h + g], x[i, :ln, h + kv + g], do[i, :ln, j], w, si,
                                    None if table is None else table[:, j], of)

    def check(self):
        n, s, h, kv, w, si, nb, md = self.shape
        sync()
        flag = __import__("ctypes").c_int()
        assert self.b.lib().gpipe_op_device_error(__import__("ctypes").byref(flag), 1, cur_stream()) == 0
        assert flag.value == 0
        for x in (self.o, self.lse, self.dqkv):
            assert bool((x[n * s:] == 7.0).all())
        o, lse = np64(self.o[:n * s]).reshape(n, s, h, HD), np64(self.lse[:n * s]).reshape(n, s, h)
        d = np64(self.dqkv[:n * s]).reshape(n, s, -1, HD)
        dk, dkt = np.zeros((n, s, kv, HD)), np.zeros((n, s, kv, HD))
        dv, dvt = np.zeros((n, s, kv, HD)), np.zeros((n, s, kv, HD))
        dt, dtt = (np.zeros((nb, h)), np.zeros((nb, h))) if nb else (None, None)

        def near(got, want, tol, what):
            bad = ~(np.abs(got - want) <= tol + 1e-30)
            assert not bad.any(), (what, int(bad.sum()), bad.size, [int(z) for z in np.argwhere(bad)[0]],
                                   float(got[bad][0]), float(want[bad][0]), float(np.broadcast_to(tol, bad.shape)[bad][0]))

        for i, j, ln, ref in self.refs():
            g = j // (h // kv)
            near(o[i, :ln, j], ref.o, ref.o_tol, ("o", i, j))
            some = np.isfinite(ref.lse)
            near(lse[i, :ln, j][some], ref.lse[some], ref.lse_tol, ("lse", i, j))
            assert np.all(np.isneginf(lse[i, :ln, j][~some])) and np.all(o[i, :ln, j][~some] == 0)
            assert np.all(np.isneginf(lse[i, ln:, j])) and np.all(o[i, ln:, j] == 0) and np.all(d[i, ln:] == 0)
            near(d[i, :ln, j], ref.dq, ref.dq_tol + U * np.abs(ref.dq) * 1.01, ("dq", i, j))
            dk[i, :ln, g] += ref.dk
            dkt[i, :ln, g] += ref.dk_tol
            dv[i, :ln, g] += ref.dv
            dvt[i, :ln, g] += ref.dv_tol
            if nb and ln:
                dt[:, j] += ref.dt
                dtt[:, j] += ref.dt_tol
        near(d[:, :, h:h + kv], dk, dkt + U * np.abs(dk) * 1.01, "dk")
        near(d[:, :, h + kv:], dv, dvt + U * np.abs(dv) * 1.01, "dv")
        if nb:
            got = np64(self.dtable) - self.dtable0.astype(np.float64)
            near(got, dt, dtt + 2.0 ** -23 * (np.abs(self.dtable0) + np.abs(dt)), "dtable")


SHAPES = [
    # nseq, seq, heads, kv, window, sinks, buckets, max_distance, lens
    (1, 1, 1, 1, 1, 0, 0, 0, None),
    (2, 1, 2, 1, 5, 3, 2, 2, None),
    (3, 19, 4, 2, 8, 2, 8, 16, None),
    (1, 64, 1, 1, 64, 0, 0, 0, None),
    (1, 65, 2, 2, 1, 1, 32, 128, None),
    (2, 127, 1, 1, 40, 64, 0, 0, None),
    (1, 128, 3, 3, 128, 0, 17, 100, None),
    (1, 129, 2, 1, 1, 0, 0, 0, None),            # each query sees itself alone
    (2, 200, 2, 2, 64, 4, 32, 128, None),
    (1, 700, 2, 1, 100, 64, 32, 128, None),      # most query blocks far from 64 sinks
    (1, 515, 3, 3, 130, 1, 0, 0, None),
    (1, 640, 2, 2, 129, 33, 64, 4096, None),     # the sinks in several buckets, far and near
    (1, 640, 1, 1, 257, 5, 2, 3, None),
    (1, 385, 4, 4, 10 ** 6, 0, 64, 4096, None),  # full causal
    (1, 1000, 8, 2, 200, 16, 32, 900, None),
    (2, 384, 3, 1, 384, 7, 32, 128, None),
    (4, 300, 2, 1, 37, 33, 17, 300, [300, 0, 1, 129]),
    (3, 257, 2, 2, 300, 0, 32, 128, [128, 64, 257]),
    (3, 600, 1, 1, 90, 20, 0, 0, [7, 599, 500]),  # a sequence shorter than the sinks
    (2, 130, 2, 2, 4, 2, 8, 9, [-5, 1000]),       # lengths outside [0, seq] are clamped
    (1, 2100, 2, 1, 513, 7, 32, 128, None),
    (1, 1500, 1, 1, 1500, 0, 24, 700, None),      # wide buckets, many of them across a tile
    (70, 40, 1, 1, 12, 3, 5, 20, None),           # many short sequences
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(x) for x in s[:8]))
def test_attention_window(b, shape):
    c = Case(b, *shape[:8], lens=shape[8])
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("shape", [
    (1, 1500, 2, 1, 1500, 0, 8, 2000, None),    # buckets of 4, 13, 57, 251, 1119 .. distances
    (1, 1300, 2, 2, 700, 40, 8, 1000, [1290]),  # the sinks' distances in wide buckets, some of them across a tile
    (1, 1700, 3, 1, 900, 3, 48, 4096, None),    # sums of 48 buckets: one backward CTA on an SM
    (2, 1200, 4, 2, 1200, 0, 2, 600, None),     # two buckets, the boundary far from the diagonal
])
def test_attention_window_wide_buckets(b, shape):
    """Distances from which on every bucket is wider than a tile."""
    c = Case(b, *shape[:8], lens=shape[8])
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("hide", ["-inf", "lowest", "all", "nearest"])
def test_attention_window_hidden_buckets(b, hide):
    """Table entries that hide a bucket; with the nearest bucket hidden the first
    query sees nothing, with all of them hidden no query does."""
    rng = np.random.default_rng(3)
    table = rng.standard_normal((8, 2))
    if hide == "all":
        table[:, 1] = -np.inf
    elif hide == "nearest":
        table[0, 0] = -np.inf
    else:
        table[3], table[6, 0] = (-np.inf, -np.inf) if hide == "-inf" else (np.finfo(np.float32).min, -1e30)
    c = Case(b, 2, 150, 2, 1, 70, 3, 8, 40, lens=[150, 90], table=table)
    c.fwd()
    c.bwd()
    c.check()


def test_attention_window_frozen_table(b):
    """Without a table gradient the other results are the same bits."""
    c = Case(b, 2, 300, 2, 1, 80, 3, 16, 64)
    c.fwd()
    c.bwd()
    sync()
    first, c.dtable = c.dqkv.clone(), None
    c.dqkv.fill_(7.0)
    c.bwd()
    sync()
    assert T().equal(first, c.dqkv)


def test_attention_window_wide_buckets_frozen_table(b):
    c = Case(b, 1, 900, 2, 1, 600, 5, 8, 1000)
    c.fwd()
    c.bwd()
    c.check()
    first, c.dtable = c.dqkv.clone(), None
    c.dqkv.fill_(7.0)
    c.bwd()
    sync()
    assert T().equal(first, c.dqkv)


def test_attention_window_equals_plain_attention(b):
    """A window over everything is gpipe_op_attention_fwd, up to roundings."""
    t = T()
    c = Case(b, 2, 256, 3, 3, 256, 0)
    c.fwd()
    o, lse = t.empty_like(c.o), t.empty_like(c.lse)
    assert b.lib().gpipe_op_attention_fwd(2, 256, 3, c.qkv.data_ptr(), o.data_ptr(), lse.data_ptr(), cur_stream()) == 0
    sync()
    assert float((o[:512].float() - c.o[:512].float()).abs().max()) <= 2 * U * float(o[:512].float().abs().max())
    assert float((lse[:512] - c.lse[:512]).abs().max()) <= 1e-5


def test_attention_window_same_bits_and_streams(b):
    """Two calls, one of them on another stream, give the same bits."""
    t = T()
    c = Case(b, 3, 500, 4, 2, 150, 9, 32, 128, lens=[500, 3, 400])
    c.fwd()
    c.bwd()
    sync()
    first = [x.clone() for x in (c.o, c.lse, c.dqkv, c.dtable)]
    for x in (c.o, c.lse, c.dqkv):
        x.fill_(7.0)
    c.dtable.copy_(t.from_numpy(c.dtable0))
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    c.fwd(s.cuda_stream)
    c.bwd(s.cuda_stream)
    sync()
    for x, y in zip(first, (c.o, c.lse, c.dqkv, c.dtable)):
        assert t.equal(x, y)


def test_attention_window_two_calls_at_once(b):
    """Two problems on two streams, each with its own scratch, running side by side."""
    t = T()
    cs = [Case(b, 2, 700, 4, 2, 200, 5, 32, 128, seed=s) for s in (1, 2)]
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for s in streams:
        s.wait_stream(t.cuda.current_stream())
    for _ in range(3):
        for c, s in zip(cs, streams):
            c.fwd(s.cuda_stream)
    for c, s in zip(cs, streams):
        c.bwd(s.cuda_stream)
    for c in cs:
        c.check()


def test_attention_window_captured(b):
    """Both passes captured into a graph, replayed on new inputs."""
    t = T()
    c = Case(b, 2, 300, 2, 1, 90, 4, 16, 64)
    c.fwd()
    c.bwd()
    sync()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        c.fwd(t.cuda.current_stream().cuda_stream)
        c.bwd(t.cuda.current_stream().cuda_stream)
    d = Case(b, 2, 300, 2, 1, 90, 4, 16, 64, seed=99)
    for name in ("qkv", "do", "table"):
        getattr(c, name).copy_(getattr(d, name))
    c.dtable0 = d.dtable0
    c.dtable.copy_(t.from_numpy(c.dtable0))
    g.replay()
    c.check()


def test_attention_window_gradients_against_differences(b):
    """Gradients of sum(o dO) against central differences of the fp64 form."""
    c = Case(b, 1, 150, 2, 1, 50, 3, 8, 30)
    c.fwd()
    c.bwd()
    sync()
    x0, do, tab = np64(c.qkv), np64(c.do).reshape(150, 2, HD), np64(c.table)
    of = buckets_by_distance(150, 8, 30)

    def value(x, tab):
        y, total = x.reshape(150, 4, HD), 0.0
        for j in range(2):
            total += (Ref(y[:, j], y[:, 2], y[:, 3], None, 50, 3, tab[:, j], of).o * do[:, j]).sum()
        return total

    grads, dtab = np64(c.dqkv[:150]), np64(c.dtable) - c.dtable0
    rng, h = np.random.default_rng(1), 1e-5
    scale = np.sqrt((grads ** 2).mean())
    for _ in range(24):
        r, k = int(rng.integers(150)), int(rng.integers(4 * HD))
        x = x0.copy()
        x[r, k] += h
        up = value(x, tab)
        x[r, k] -= 2 * h
        want = (up - value(x, tab)) / (2 * h)
        # bf16 roundings of O, P, dS and of the result: a few 2^-8 of the gradients' size
        assert abs(grads[r, k] - want) <= 8 * U * (abs(want) + scale), (r, k)
    for e in range(8):
        t2 = tab.copy()
        t2[e, 1] += h
        up = value(x0, t2)
        t2[e, 1] -= 2 * h
        want = (up - value(x0, t2)) / (2 * h)
        assert abs(dtab[e, 1] - want) <= 1e-4 * (abs(want) + np.abs(dtab).max()), e


# ---------------------------------------------------------------------------
# Distillation
# ---------------------------------------------------------------------------
def distill_ref(z, idx, tl, temp, kd, ce, seq, tokens, row0):
    rows, vocab = z.shape
    loss, dz = np.zeros(rows), np.zeros((rows, vocab))
    mag = np.zeros((rows, vocab))   # sizes of the terms of dz
    size = np.zeros(rows)           # and of the loss
    for r in range(rows):
        keep = (idx[r] >= 0) & (idx[r] < vocab)
        t = np.where(keep, tl[r].astype(np.float64) / temp, -np.inf)
        m = z[r].max()
        if np.isfinite(t.max()):
            p = np.exp(t - t.max())
            p /= p.sum()
            x = (z[r] - m) / temp
            ls = np.log(np.exp(x).sum())
            q = np.exp(x - ls)
            for k in range(len(p)):
                if p[k] > 0:
                    loss[r] += kd * temp ** 2 * p[k] * (np.log(p[k]) - (x[idx[r, k]] - ls))
                    size[r] += kd * temp ** 2 * p[k] * (abs(np.log(p[k])) + abs(x[idx[r, k]]) + abs(ls) +
                                                        abs(t[k]) + abs(t.max()) + abs(z[r, idx[r, k]] / temp) + 1)
                    dz[r, idx[r, k]] -= kd * temp * p[k]
                    mag[r, idx[r, k]] += kd * temp * p[k] * (1 + abs(t[k]) + abs(t.max()))
            dz[r] += kd * temp * q
            mag[r] += kd * temp * q * (1 + np.abs(np.where(q > 0, x, 0.0)))
        if ce > 0 and (row0 + r) % seq != seq - 1 and 0 <= tokens[row0 + r + 1] < vocab:
            g = tokens[row0 + r + 1]
            x = z[r] - m
            ls = np.log(np.exp(x).sum())
            loss[r] += ce * (ls - x[g])
            size[r] += ce * (abs(ls) + abs(x[g]) + 1)
            dz[r] += ce * np.exp(x - ls)
            mag[r] += ce * np.exp(x - ls) * (1 + np.abs(np.where(np.isfinite(x), x, 0.0)))
            dz[r, g] -= ce
            mag[r, g] += ce
    return loss, dz, size, mag


class Distill:
    def __init__(self, b, rows, vocab, topk, dtype="f32", temp=2.0, kd=0.7, ce=0.3, ld=None, lddz=None, seq=None,
                 row0=0, in_place=False, seed=0):
        t = T()
        rng = np.random.default_rng(seed + rows + vocab * 3 + topk)
        self.b, self.a = b, (rows, vocab, topk, temp, kd, ce, seq or rows, row0)
        self.ld = ld or vocab
        self.bf16 = dtype == "bf16"
        full = np.full((rows, self.ld), np.nan, dtype=np.float32)   # columns behind the vocabulary: never read
        full[:, :vocab] = rng.standard_normal((rows, vocab)) * 3
        self.z = t.from_numpy(full).cuda()
        if self.bf16:
            self.z = self.z.bfloat16()
        self.idx = np.stack([rng.permutation(vocab)[:topk] if vocab >= topk else rng.integers(0, vocab, topk)
                             for _ in range(rows)]).astype(np.int32)
        self.tl = (rng.standard_normal((rows, topk)) * 3).astype(np.float32)
        self.tokens = rng.integers(0, vocab, row0 + rows + 1).astype(np.int32)
        self.in_place = in_place
        self.lddz = lddz or ((self.ld * (1 if self.bf16 else 2)) if in_place else vocab)

    def run(self, want=True, stream=None):
        t = T()
        rows, vocab, topk, temp, kd, ce, seq, row0 = self.a
        self.z0 = np64(self.z)[:, :vocab]
        self.dz = None
        if want:
            if self.in_place:
                self.dz = self.z.view(t.bfloat16).reshape(rows, -1)
            else:
                self.dz = t.full((rows + 1, self.lddz), 7.0, device="cuda", dtype=t.bfloat16)
        self.loss = t.full((rows + 1,), 7.0, device="cuda")
        self.d = [dev(self.idx), dev(self.tl), dev(self.tokens)]
        rc = self.b.lib().gpipe_op_distill(1 if self.bf16 else 0, rows, vocab, self.z.data_ptr(), self.ld, topk,
                                           self.d[0].data_ptr(), self.d[1].data_ptr(), temp, kd, seq,
                                           self.d[2].data_ptr(), row0, ce, self.loss.data_ptr(),
                                           self.dz.data_ptr() if want else None, self.lddz,
                                           cur_stream() if stream is None else stream)
        assert rc == 0, self.b.lib().gpipe_last_error(None)
        KEEP.append(self)
        return self

    def check(self, flagged=0):
        import ctypes
        sync()
        flag = ctypes.c_int()
        assert self.b.lib().gpipe_op_device_error(ctypes.byref(flag), 1, cur_stream()) == 0
        assert flag.value == flagged
        rows, vocab, topk, temp, kd, ce, seq, row0 = self.a
        temp, kd, ce = (float(np.float32(x)) for x in (temp, kd, ce))
        loss, dz, size, mag = distill_ref(self.z0, self.idx, self.tl, temp, kd, ce, seq, self.tokens, row0)
        assert float(self.loss[rows]) == 7.0
        got = np64(self.loss[:rows])
        # fp32: a handful of roundings of each term, and the sums of the exponentials
        eps = 2.0 ** -24 * (32 + vocab / 512 + topk / 32)
        assert np.all(np.abs(got - loss) <= eps * size + 1e-30), np.max(np.abs(got - loss) / (size + 1e-30))
        if self.dz is None:
            return
        g = np64(self.dz)
        if not self.in_place:
            assert np.all(g[rows] == 7.0) and np.all(g[:, vocab:] == 7.0)
        # one rounding to bf16 (values below its normal range: to 2^-134), on top of the fp32 ones
        tol = U * np.abs(dz) + (1 + U) * eps * mag + 2.0 ** -134
        bad = ~(np.abs(g[:rows, :vocab] - dz) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], g[:rows, :vocab][bad][0], dz[bad][0], tol[bad][0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,topk,kw", [
    (1, 1, 1, {}),
    (3, 5, 2, {}),
    (5, 517, 8, dict(ld=520, seq=5)),
    (4, 512, 256, dict(seq=2)),
    (7, 4096, 33, dict(temp=0.5, row0=3, seq=4)),
    (3, 32000, 64, dict(lddz=32008)),
    (2, 50001, 100, dict(ld=50008, lddz=50008)),
    (2, 50001, 100, {}),                       # odd rows: single loads
    (2, 131072, 16, dict(ce=0.0)),
    (3, 70000, 7, dict(kd=0.0)),
    (2, 300000, 9, {}),
    (200, 2048, 5, dict(seq=64)),
    (5, 1000, 10, dict(in_place=True)),
    (4, 33000, 20, dict(in_place=True, ld=33024)),
    (3, 1001, 12, dict(in_place=True)),
    (2, 131080, 12, dict(in_place=True)),
])
def test_distill(b, dtype, rows, vocab, topk, kw):
    Distill(b, rows, vocab, topk, dtype, **kw).run().check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,topk,kw", [
    (400, 9000, 200, dict(seq=100)),          # several rows a CTA, one after the other
    (330, 9000, 5, dict(ce=0.0, in_place=True)),
    (170, 9001, 70, dict(seq=10)),            # unaligned rows, more than SMs
    (160, 9001, 70, dict(in_place=True)),
    (3, 100001, 9, dict(seq=3)),              # unaligned, across a cluster
    (30, 5001, 20, dict(seq=10)),
    (30, 5001, 20, dict(in_place=True)),
    (5, 20001, 30, dict(lddz=20002)),         # logits and dz of different alignments
    (200, 9001, 40, dict(ld=9003)),
    (9, 100003, 256, dict(ld=100005, lddz=100013, seq=3)),
    (2, 270001, 33, {}),                      # unaligned, more than a cluster holds
])
def test_distill_many_and_long_rows(b, dtype, rows, vocab, topk, kw):
    Distill(b, rows, vocab, topk, dtype, **kw).run().check()


@pytest.mark.parametrize("dtype,rows,vocab,kw", [
    ("f32", 160, 70004, dict(seq=16)),        # a row is more than the ring of chunks holds
    ("bf16", 200, 150000, dict(ce=0.0)),
    ("f32", 1, 300003, dict(ld=300004)),
    ("f32", 500, 6000, dict(seq=5)),
])
def test_distill_loss_alone_of_long_rows(b, dtype, rows, vocab, kw):
    Distill(b, rows, vocab, 12, dtype, **kw).run(want=False).check()


@pytest.mark.parametrize("vocab", [5, 4000, 131072])
def test_distill_loss_alone(b, vocab):
    Distill(b, 9, vocab, 3).run(want=False).check()


def test_distill_empty_and_repeated_slots(b):
    d = Distill(b, 6, 3000, 40, seq=6)
    d.idx[0, :] = -1                     # no teacher
    d.tl[0] = np.nan                     # whose logits are not looked at
    d.idx[1, 5:] = -7
    d.idx[2, :] = 11                     # one token in every slot
    d.idx[3, ::2] = d.tokens[4]          # the target itself, twenty times
    d.tl[4, 3:] = -np.inf                # filled slots of no weight
    d.tl[5, :] = -np.inf                 # nothing but those: no teacher term
    d.run().check()


def test_distill_extreme_logits(b):
    """Logits far from 0 and -inf ones; a finite loss where no weight falls on them."""
    d = Distill(b, 4, 1000, 10, seq=4)
    d.z[0] += 3e4
    d.z[1, 500:] = -float("inf")
    d.idx[1] = np.arange(10)
    d.tokens[2] = 3
    d.z[2] = -1e30
    d.z[2, 7] = 0.0
    d.idx[2] = 7
    d.tokens[3] = 7
    d.z[3] *= 1e-3
    d.run().check()


def test_distill_bad_ids_are_flagged(b):
    d = Distill(b, 3, 100, 4)
    d.idx[1, 2] = 100
    d.run().check(flagged=5)
    d = Distill(b, 3, 100, 4)
    d.tokens[2] = -1
    d.run().check(flagged=5)


def test_distill_nan_propagates(b):
    d = Distill(b, 3, 1000, 4, ce=0.0)
    d.z[1, 77] = float("nan")
    d.run()
    sync()
    assert bool(d.loss[1].isnan()) and bool(d.dz[1].isnan().all())
    assert not bool(d.loss[[0, 2]].isnan().any()) and not bool(d.dz[[0, 2]].isnan().any())


def test_distill_same_bits_streams_and_capture(b):
    t = T()
    d = Distill(b, 50, 5000, 30).run()
    sync()
    loss, dz = d.loss.clone(), d.dz.clone()
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    d.run(stream=s.cuda_stream)
    sync()
    assert t.equal(loss, d.loss) and t.equal(dz, d.dz)
    g = t.cuda.CUDAGraph()
    rows, vocab, topk, temp, kd, ce, seq, row0 = d.a
    with t.cuda.graph(g):
        rc = b.lib().gpipe_op_distill(0, rows, vocab, d.z.data_ptr(), d.ld, topk, d.d[0].data_ptr(),
                                      d.d[1].data_ptr(), temp, kd, seq, d.d[2].data_ptr(), row0, ce,
                                      d.loss.data_ptr(), d.dz.data_ptr(), d.lddz,
                                      t.cuda.current_stream().cuda_stream)
    assert rc == 0
    d.z.mul_(0.5)
    d.z0 = np64(d.z)
    g.replay()
    d.check()


def test_distill_gradient_against_differences(b):
    d = Distill(b, 4, 600, 12, seq=4).run()
    sync()
    rows, vocab, topk, temp, kd, ce, seq, row0 = d.a
    g, z = np64(d.dz[:rows]), d.z0
    rng, h = np.random.default_rng(5), 1e-5
    for r in range(rows):
        for v in [int(x) for x in rng.integers(0, vocab, 6)] + [int(d.idx[r, 0]), int(d.tokens[r + 1])]:
            up, dn = z.copy(), z.copy()
            up[r, v] += h
            dn[r, v] -= h
            want = (distill_ref(up, d.idx, d.tl, temp, kd, ce, seq, d.tokens, 0)[0][r] -
                    distill_ref(dn, d.idx, d.tl, temp, kd, ce, seq, d.tokens, 0)[0][r]) / (2 * h)
            assert abs(g[r, v] - want) <= U * abs(want) + 1e-6


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def test_student_step(b):
    """A student's step through the library: windowed attention with positions on a
    projection of the input, logits over a vocabulary, the distillation loss in
    place over them, and the gradients back to every weight, against fp64.

    Roundings to bf16 on the way to a weight's gradient: qkv, P, o, y, dz, dy, do,
    dS (with P and D) and dqkv.  Each is off by at most 2^-8 of a value, and by
    less of a norm; nothing on the way is ill-conditioned (rows of unit size,
    softmaxes, projections of variance 1/d), so the gradients are within 9 times
    that of their norm."""
    t = T()
    lib = b.lib()
    n, s, d, heads, kv, vocab, k = 2, 96, 128, 2, 1, 512, 16
    window, sinks, nb, md, temp, kd, ce = 40, 3, 8, 64, 2.0, 0.6, 0.4
    rows, cols = n * s, (heads + 2 * kv) * HD
    rng = np.random.default_rng(8)

    def bf(*shape, scale=1.0):
        x = dev((rng.standard_normal(shape) * scale).astype(np.float32), "bf16")
        return x, np64(x)

    x, x64 = bf(rows, d)
    wq, wq64 = bf(cols, d, scale=d ** -0.5)
    wo, wo64 = bf(d, heads * HD, scale=(heads * HD) ** -0.5)
    emb, emb64 = bf(vocab, d, scale=2 * d ** -0.5)
    table64 = rng.standard_normal((nb, heads)).astype(np.float32)
    table = dev(table64)
    lens = np.array([s, 70], dtype=np.int32)
    dlens = dev(lens)
    idx = np.stack([rng.permutation(vocab)[:k] for _ in range(rows)]).astype(np.int32)
    tl = rng.standard_normal((rows, k)).astype(np.float32)
    idx[s + 70:] = -1                              # padded rows have no teacher
    tokens = rng.integers(0, vocab, rows + 1).astype(np.int32)
    kd1, ce1 = kd / rows, ce / rows
    didx, dtl, dtok = dev(idx), dev(tl), dev(tokens)

    def empty(r, c, dt=None):
        y = t.empty((r, c), device="cuda", dtype=dt or t.bfloat16)
        KEEP.append(y)
        return y

    def zeros(*shape):
        y = t.zeros(shape, device="cuda")
        KEEP.append(y)
        return y

    def gemm(m, nn, kk, A, lda, ak, B, ldb, bk, epi, C, ldc):
        rc = lib.gpipe_op_gemm(1, m, nn, kk, A.data_ptr(), lda, ak, B.data_ptr(), ldb, bk, epi, C.data_ptr(), ldc, None,
                               None, 0, None, None, 0, cur_stream())
        assert rc == 0, lib.gpipe_last_error(None)

    qkv, o, lse, y = empty(rows, cols), empty(rows, heads * HD), zeros(rows, heads), empty(rows, d)
    logits, loss = empty(rows, vocab, t.float32), zeros(rows)
    gemm(rows, cols, d, x, d, 1, wq, d, 1, 0, qkv, cols)
    form = (n, s, heads, kv, window, sinks, dlens.data_ptr(), table.data_ptr(), nb, md, qkv.data_ptr(), o.data_ptr())
    assert lib.gpipe_op_attention_window_fwd(*form, lse.data_ptr(), cur_stream()) == 0
    gemm(rows, d, heads * HD, o, heads * HD, 1, wo, heads * HD, 1, 0, y, d)
    gemm(rows, vocab, d, y, d, 1, emb, d, 1, 4, logits, vocab)
    # the labels of padded rows would count; this step's loss takes the teacher and the labels of all rows
    assert lib.gpipe_op_distill(0, rows, vocab, logits.data_ptr(), vocab, k, didx.data_ptr(), dtl.data_ptr(), temp, kd1,
                                s, dtok.data_ptr(), 0, ce1, loss.data_ptr(), logits.data_ptr(), 2 * vocab,
                                cur_stream()) == 0
    dz = logits.view(t.bfloat16)                   # leading dimension 2 vocab
    demb, dwo, dwq = zeros(vocab, d), zeros(d, heads * HD), zeros(cols, d)
    dy, do, dqkv, dtable, dx = empty(rows, d), empty(rows, heads * HD), empty(rows, cols), zeros(nb, heads), empty(rows, d)
    gemm(vocab, d, rows, dz, 2 * vocab, 0, y, d, 0, 3, demb, d)
    gemm(rows, d, vocab, dz, 2 * vocab, 1, emb, d, 0, 0, dy, d)
    gemm(d, heads * HD, rows, dy, d, 0, o, heads * HD, 0, 3, dwo, heads * HD)
    gemm(rows, heads * HD, d, dy, d, 1, wo, heads * HD, 0, 0, do, heads * HD)
    scratch = t.empty(lib.gpipe_op_attention_window_scratch_bytes(n, s, heads, window, sinks, nb), device="cuda",
                      dtype=t.uint8)
    assert lib.gpipe_op_attention_window_bwd(*form, do.data_ptr(), lse.data_ptr(), dqkv.data_ptr(), dtable.data_ptr(),
                                             scratch.data_ptr(), cur_stream()) == 0
    gemm(cols, d, rows, dqkv, cols, 0, x, d, 0, 3, dwq, d)
    gemm(rows, d, cols, dqkv, cols, 1, wq, d, 0, 0, dx, d)
    sync()

    # the same in fp64
    q64 = x64 @ wq64.T
    of = buckets_by_distance(s, nb, md)
    o64, refs = np.zeros((rows, heads * HD)), {}
    def attend(i, j, dout):
        r0, r1 = i * s, i * s + int(lens[i])
        z = q64[r0:r1].reshape(-1, heads + 2 * kv, HD)
        return Ref(z[:, j], z[:, heads], z[:, heads + kv], dout, window, sinks, table64[:, j].astype(np.float64), of)
    for i in range(n):
        for j in range(heads):
            o64[i * s:i * s + int(lens[i]), j * HD:(j + 1) * HD] = attend(i, j, None).o
    y64 = o64 @ wo64.T
    l64, dz64, _, _ = distill_ref(y64 @ emb64.T, idx, tl, temp, np.float32(kd1), np.float32(ce1), s, tokens, 0)
    dy64 = dz64 @ emb64
    do64 = dy64 @ wo64
    dq64, dt64 = np.zeros((rows, heads + 2 * kv, HD)), np.zeros((nb, heads))
    for i in range(n):
        r0, r1 = i * s, i * s + int(lens[i])
        for j in range(heads):
            ref = attend(i, j, do64[r0:r1, j * HD:(j + 1) * HD])
            dq64[r0:r1, j] += ref.dq
            dq64[r0:r1, heads] += ref.dk
            dq64[r0:r1, heads + kv] += ref.dv
            dt64[:, j] += ref.dt
    dq64 = dq64.reshape(rows, cols)
    for got, want, what in [(loss, l64, "loss"), (demb, dz64.T @ y64, "demb"), (dwo, dy64.T @ o64, "dwo"),
                            (dtable, dt64, "dtable"), (dwq, dq64.T @ x64, "dwq"), (dx, dq64 @ wq64, "dx")]:
        err = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
        assert err <= 9 * U, (what, err)
