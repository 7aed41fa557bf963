"""Host side of the windowed attention and the distillation loss: bucket
boundaries, workspace sizes and every refusal.  No CUDA call is made here (a
pointer is only looked at for NULL and alignment before the arguments pass)."""
import ctypes
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import _build
    _build.build()
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


def bucket_of(d, buckets, max_distance):
    """The documented bucket of distance d in whole numbers: the largest k with
    (d / e)^m >= (max_distance / e)^k."""
    e = buckets // 2
    if d < e:
        return d
    m, k = buckets - e, 0
    while k + 1 < m and Fraction(d, e) ** m >= Fraction(max_distance, e) ** (k + 1):
        k += 1
    return e + k


@pytest.mark.parametrize("buckets,max_distance", [
    (2, 2), (2, 16), (2, 4096), (3, 7), (8, 16), (8, 5), (16, 128), (17, 100), (32, 128), (32, 17), (32, 256),
    (32, 1024), (64, 33), (64, 512), (63, 4095), (64, 4096)])
def test_bucket_starts_are_exact(b, buckets, max_distance):
    starts = (ctypes.c_int32 * buckets)()
    assert b.lib().gpipe_op_position_bucket_starts(buckets, max_distance, starts) == 0
    starts = list(starts)
    assert starts[0] == 0 and starts == sorted(starts)
    # next to every boundary, and over a sample of all distances
    at = sorted({d for s in starts for d in (s - 1, s, s + 1) if d >= 0} |
                set(range(0, max_distance + 50, max(1, max_distance // 97))))
    for d in at:
        got = max(k for k, s in enumerate(starts) if s <= d)
        assert got == bucket_of(d, buckets, max_distance), d


@pytest.mark.parametrize("buckets,max_distance", [(1, 8), (0, 8), (65, 128), (32, 16), (32, 4097), (-2, 4), (8, 0)])
def test_bucket_starts_refusals(b, buckets, max_distance):
    starts = (ctypes.c_int32 * 64)()
    assert b.lib().gpipe_op_position_bucket_starts(buckets, max_distance, starts) == -1
    assert b"position buckets" in b.lib().gpipe_last_error(None)
    assert b.lib().gpipe_op_position_bucket_starts(8, 16, None) == -1


def test_scratch_bytes(b):
    f = b.lib().gpipe_op_attention_window_scratch_bytes
    rows = (8 + 64) * 2 * 3 * 128  # (-lse, -D) of 2 sequences x 3 heads x one block of 128 queries, twice
    assert f(2, 100, 3, 100, 0, 0) == rows
    assert f(2, 100, 3, 100, 64, 0) == rows          # no query block is far from the sinks
    assert f(2, 100, 3, 100, 64, 32) == rows + 2 * 3 * 32 * 4
    # 4 blocks of queries, window 1: blocks 1..3 are far from the sinks
    assert f(1, 512, 1, 1, 2, 0) == (8 + 64) * 512 + 4 * 2 * 128 * 4 + 2 * 128 * 4
    for bad in [(0, 64, 1, 1, 0, 0), (1, 0, 1, 1, 0, 0), (1, 64, 0, 1, 0, 0), (1, 64, 1, 0, 0, 0), (1, 64, 1, 1, -1, 0),
                (1, 64, 1, 1, 65, 0), (1, 64, 1, 1, 0, 1), (1, 64, 1, 1, 0, 65), (1 << 20, 1 << 20, 1, 1, 0, 0)]:
        assert f(*bad) == 0, bad


OK = dict(nseq=2, seq=64, heads=4, kv_heads=2, window=16, sinks=4, lens=0, table=256, num_buckets=8, max_distance=16,
          qkv=256, o=256, dout=256, lse=256, dqkv=256, dtable=256, scratch=256)


def _fwd(b, **kw):
    a = dict(OK, **kw)
    return b.lib().gpipe_op_attention_window_fwd(
        a["nseq"], a["seq"], a["heads"], a["kv_heads"], a["window"], a["sinks"], a["lens"] or None, a["table"] or None,
        a["num_buckets"], a["max_distance"], a["qkv"], a["o"], a["lse"], None)


def _bwd(b, **kw):
    a = dict(OK, **kw)
    return b.lib().gpipe_op_attention_window_bwd(
        a["nseq"], a["seq"], a["heads"], a["kv_heads"], a["window"], a["sinks"], a["lens"] or None, a["table"] or None,
        a["num_buckets"], a["max_distance"], a["qkv"], a["o"], a["dout"], a["lse"], a["dqkv"], a["dtable"] or None,
        a["scratch"], None)


@pytest.mark.parametrize("bad", [
    dict(nseq=0), dict(seq=0), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(heads=4098, kv_heads=1),
    dict(window=0), dict(window=-5), dict(sinks=-1), dict(sinks=65), dict(nseq=1 << 16, seq=1 << 16),
    dict(num_buckets=0), dict(table=0), dict(num_buckets=1), dict(num_buckets=65), dict(max_distance=4),
    dict(max_distance=4097), dict(qkv=0), dict(o=0), dict(lse=0), dict(qkv=264), dict(o=8),
    dict(nseq=1 << 18, seq=1 << 12, heads=4096, kv_heads=4096)])
def test_attention_window_refusals(b, bad):
    assert _fwd(b, **bad) == -1
    assert b"attention_window" in b.lib().gpipe_last_error(None) or b"position" in b.lib().gpipe_last_error(None)
    assert _bwd(b, **bad) == -1


@pytest.mark.parametrize("bad", [dict(dout=0), dict(dout=8), dict(dqkv=0), dict(dqkv=24), dict(scratch=0),
                                 dict(scratch=128), dict(table=0, num_buckets=0)])
def test_attention_window_bwd_refusals(b, bad):
    assert _bwd(b, **bad) == -1


# tensors that do not touch each other: 2 x 64 rows of 512 (qkv, dqkv) or 256 (o, dout) columns, bf16
APART = dict(qkv=1 << 20, o=2 << 20, dout=3 << 20, lse=4 << 20, dqkv=5 << 20, scratch=6 << 20)


@pytest.mark.parametrize("bad", [dict(o=1 << 20), dict(o=(1 << 20) + 128 * 1024 - 16), dict(o=(1 << 20) - 128 * 512 + 16),
                                 dict(lse=1 << 20), dict(lse=(2 << 20) + 128 * 512 - 4), dict(lse=(2 << 20) - 16)])
def test_attention_window_refuses_overlapping_outputs(b, bad):
    assert _fwd(b, **dict(APART, **bad)) == -1
    assert b"overlap" in b.lib().gpipe_last_error(None)


@pytest.mark.parametrize("bad", [dict(dqkv=1 << 20), dict(dqkv=(2 << 20) - 128 * 1024 + 16), dict(dqkv=3 << 20),
                                 dict(dqkv=4 << 20), dict(dqkv=6 << 20), dict(scratch=1 << 20), dict(scratch=2 << 20),
                                 dict(scratch=3 << 20), dict(scratch=4 << 20), dict(scratch=5 << 20)])
def test_attention_window_bwd_refuses_overlaps(b, bad):
    assert _bwd(b, **dict(APART, **bad)) == -1
    assert b"overlap" in b.lib().gpipe_last_error(None)


GOOD = dict(dtype=0, rows=4, vocab=32, logits=1 << 20, ld=32, topk=4, idx=256, val=256, t=2.0, kd=1.0, seq=4,
            tokens=256, row0=0, ce=1.0, loss=256, dz=1 << 30, lddz=32)


def _distill(b, **kw):
    a = dict(GOOD, **kw)
    return b.lib().gpipe_op_distill(a["dtype"], a["rows"], a["vocab"], a["logits"] or None, a["ld"], a["topk"],
                                    a["idx"] or None, a["val"] or None, a["t"], a["kd"], a["seq"],
                                    a["tokens"] or None, a["row0"], a["ce"], a["loss"] or None, a["dz"] or None,
                                    a["lddz"], None)


@pytest.mark.parametrize("bad", [
    dict(rows=0), dict(vocab=0), dict(ld=31), dict(topk=0), dict(topk=257), dict(t=0.0), dict(t=-1.0),
    dict(t=float("nan")), dict(t=float("inf")), dict(kd=-1.0), dict(kd=float("nan")), dict(ce=-1.0),
    dict(ce=float("inf")), dict(logits=0), dict(idx=0), dict(val=0), dict(loss=0), dict(tokens=0), dict(seq=0),
    dict(row0=-1), dict(lddz=31), dict(logits=(1 << 20) + 2), dict(dz=(1 << 30) + 1),
    dict(dz=1 << 20, lddz=32),                     # in place, but with another row stride in bytes
    dict(dz=(1 << 20) + 64, lddz=64),              # overlapping the logits, not the same address
    dict(dz=(1 << 20) - 64, lddz=64)])
def test_distill_refusals(b, bad):
    assert _distill(b, **bad) == -1
    assert b"distill" in b.lib().gpipe_last_error(None)


@pytest.mark.parametrize("bad", [dict(t=1e-40), dict(t=3e20), dict(t=1e10, kd=1e30)])
def test_distill_refuses_temperatures_out_of_range(b, bad):
    """Finite ones whose reciprocal, or whose square times the scale, is not."""
    assert _distill(b, **bad) == -1
    assert b"temperature" in b.lib().gpipe_last_error(None)


def test_distill_refuses_other_types(b):
    assert _distill(b, dtype=2) == -6
