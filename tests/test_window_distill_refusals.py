"""Each refusal of the windowed attention and of the distillation by its own
message.  The calls' pointers overlap on purpose, which is refused last: a check
that has gone missing shows as the overlap's message, and nothing is launched on
addresses that do not exist.  No CUDA call is made here."""
import pytest


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import _build
    _build.build()
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


A = 1 << 20   # every pointer: aligned for everything
ATTENTION = dict(nseq=2, seq=64, heads=4, kv_heads=2, window=16, sinks=4, lens=A, table=A, num_buckets=8,
                 max_distance=16, qkv=A, o=A, dout=A, lse=A, dqkv=A, dtable=A, scratch=A)


def attention(b, backward, **kw):
    a = dict(ATTENTION, **kw)
    form = [a["nseq"], a["seq"], a["heads"], a["kv_heads"], a["window"], a["sinks"], a["lens"] or None,
            a["table"] or None, a["num_buckets"], a["max_distance"], a["qkv"] or None, a["o"] or None]
    lib = b.lib()
    if backward:
        rc = lib.gpipe_op_attention_window_bwd(*form, a["dout"] or None, a["lse"] or None, a["dqkv"] or None,
                                               a["dtable"] or None, a["scratch"] or None, None)
    else:
        rc = lib.gpipe_op_attention_window_fwd(*form, a["lse"] or None, None)
    return rc, lib.gpipe_last_error(None).decode()


@pytest.mark.parametrize("backward", [False, True])
def test_attention_calls_that_only_overlap(b, backward):
    """The calls below are refused for nothing else."""
    rc, said = attention(b, backward)
    assert rc == -1 and "overlap" in said


HEADS, SINKS, BUCKETS = "multiple of kv_heads", "window >= 1 and 0 <= sinks", "2 <= num_buckets"


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad,words", [
    (dict(nseq=0), HEADS), (dict(nseq=-1), HEADS), (dict(seq=0), HEADS), (dict(heads=0), HEADS),
    (dict(kv_heads=0), HEADS), (dict(kv_heads=3), HEADS), (dict(kv_heads=8), HEADS),
    (dict(heads=4097, kv_heads=1), HEADS),
    (dict(nseq=1 << 16, seq=1 << 16), "at most 2^30"),
    (dict(nseq=1 << 18, seq=1 << 12, heads=4096, kv_heads=4096), "2^28 blocks"),
    (dict(window=0), SINKS), (dict(window=-5), SINKS), (dict(sinks=-1), SINKS), (dict(sinks=65), SINKS),
    (dict(num_buckets=0), "goes with num_buckets"), (dict(table=0), "goes with num_buckets"),
    (dict(num_buckets=1), BUCKETS), (dict(num_buckets=65), BUCKETS), (dict(num_buckets=-2), BUCKETS),
    (dict(max_distance=4), BUCKETS), (dict(max_distance=4097), BUCKETS),
    (dict(qkv=0), "16-B aligned"), (dict(qkv=A + 8), "16-B aligned"), (dict(o=0), "16-B aligned"),
    (dict(o=A + 8), "16-B aligned"), (dict(lse=0), "lse not NULL")])
def test_attention_refusals(b, backward, bad, words):
    rc, said = attention(b, backward, **bad)
    assert rc == -1 and words in said and "overlap" not in said


@pytest.mark.parametrize("bad,words", [
    (dict(dout=0), "16-B aligned"), (dict(dout=A + 8), "16-B aligned"), (dict(dqkv=0), "16-B aligned"),
    (dict(dqkv=A + 24), "16-B aligned"), (dict(scratch=0), "256-B aligned"), (dict(scratch=A + 128), "256-B aligned"),
    (dict(table=0, num_buckets=0), "needs the table")])
def test_attention_backward_refusals(b, bad, words):
    rc, said = attention(b, True, **bad)
    assert rc == -1 and words in said and "overlap" not in said


DISTILL = dict(dtype=0, rows=4, vocab=32, logits=A, ld=32, topk=4, idx=A, val=A, t=2.0, kd=1.0, seq=4, tokens=A, row0=0,
               ce=1.0, loss=A, dz=A, lddz=32)


def distill(b, **kw):
    a = dict(DISTILL, **kw)
    lib = b.lib()
    rc = lib.gpipe_op_distill(a["dtype"], a["rows"], a["vocab"], a["logits"] or None, a["ld"], a["topk"],
                              a["idx"] or None, a["val"] or None, a["t"], a["kd"], a["seq"], a["tokens"] or None,
                              a["row0"], a["ce"], a["loss"] or None, a["dz"] or None, a["lddz"], None)
    return rc, lib.gpipe_last_error(None).decode()


def test_distill_call_that_only_overlaps(b):
    rc, said = distill(b)
    assert rc == -1 and "overlap" in said


SIZES, SCALES, NULLS, LABELS = "1 <= rows <= 2^27", "finite temperature > 0 and finite scales", "NULL", "seq >= 1 and row0"


@pytest.mark.parametrize("bad,words", [
    (dict(rows=0), SIZES), (dict(rows=(1 << 27) + 1), SIZES), (dict(vocab=0), SIZES),
    (dict(vocab=(1 << 30) + 1, ld=1 << 31, lddz=1 << 31), SIZES), (dict(ld=31), SIZES), (dict(topk=0), SIZES),
    (dict(topk=257), SIZES),
    (dict(t=0.0), SCALES), (dict(t=-1.0), SCALES), (dict(t=float("nan")), SCALES), (dict(t=float("inf")), SCALES),
    (dict(kd=-1.0), SCALES), (dict(kd=float("nan")), SCALES), (dict(kd=float("inf")), SCALES), (dict(ce=-1.0), SCALES),
    (dict(ce=float("nan")), SCALES), (dict(ce=float("inf")), SCALES),
    (dict(logits=0), NULLS), (dict(idx=0), NULLS), (dict(val=0), NULLS), (dict(loss=0), NULLS),
    (dict(tokens=0), LABELS), (dict(seq=0), LABELS), (dict(row0=-1), LABELS),
    (dict(logits=A + 2), "aligned to their elements"), (dict(dtype=1, logits=A + 1), "aligned to their elements"),
    (dict(dz=A + 1), "aligned to their elements"), (dict(lddz=31), "lddz must be at least vocab")])
def test_distill_refusals(b, bad, words):
    rc, said = distill(b, **bad)
    assert rc == -1 and words in said and "overlap" not in said


def test_distill_refuses_other_types(b):
    rc, said = distill(b, dtype=2)
    assert rc == -6 and "dtype must be 0 or 1" in said


@pytest.mark.parametrize("t", [1e-40, 2.0 ** -128, 3.5e-39, 4.2e-39, 1e-38])
def test_distill_refuses_temperatures_below_the_normal_range(b, t):
    """1 / T is finite from 2^-128 on, log2(e) / T only from 4.24e-39, and a number
    below 2^-126 has fewer bits than the others."""
    rc, said = distill(b, t=t)
    assert rc == -1 and "temperature" in said and "overlap" not in said


def test_distill_takes_the_smallest_normal_temperature(b):
    rc, said = distill(b, t=2.0 ** -126)
    assert rc == -1 and "overlap" in said


# tensors that do not touch each other: 2 x 64 rows of 512 (qkv, dqkv) or 256 (o, dout) columns, bf16; 8 buckets x 4 heads
M = 1 << 20
APART = dict(qkv=M, o=2 * M, dout=3 * M, lse=4 * M, dqkv=5 * M, scratch=6 * M, table=8 * M, lens=9 * M, dtable=10 * M)
BYTES = dict(qkv=128 * 1024, o=128 * 512, dout=128 * 512, lse=128 * 16, dqkv=128 * 1024, table=128, lens=8, dtable=128)


def onto(what, other, apart, sizes):
    """`what` onto the first bytes of `other`, and onto its last 16 (or as many as it has)."""
    yield {what: apart[other]}
    yield {what: apart[other] + max(0, sizes[other] - 256) // 256 * 256}


@pytest.mark.parametrize("out", ["o", "lse"])
@pytest.mark.parametrize("other", ["qkv", "table", "lens", "o", "lse"])
def test_attention_forward_outputs_overlap_nothing(b, out, other):
    if out == other:
        return
    for bad in onto(out, other, APART, BYTES):
        rc, said = attention(b, False, **dict(APART, **bad))
        assert rc == -1 and "overlap" in said, bad


@pytest.mark.parametrize("out", ["dqkv", "dtable", "scratch"])
@pytest.mark.parametrize("other", ["qkv", "o", "dout", "lse", "table", "lens", "dqkv", "dtable", "scratch"])
def test_attention_backward_outputs_overlap_nothing(b, out, other):
    if out == other or (out, other) == ("dtable", "table"):  # the table may take its own gradient
        return
    sizes = dict(BYTES, scratch=b.lib().gpipe_op_attention_window_scratch_bytes(2, 64, 4, 16, 4, 8))
    for bad in onto(out, other, APART, sizes):
        rc, said = attention(b, True, **dict(APART, **bad))
        assert rc == -1 and "overlap" in said, bad


# 4 rows of 32 fp32 logits, 4 slots, bf16 dz
DAPART = dict(logits=M, idx=2 * M, val=3 * M, tokens=4 * M, loss=5 * M, dz=6 * M)
DBYTES = dict(logits=512, idx=64, val=64, tokens=16, loss=16, dz=256)  # (the last row has no target)


@pytest.mark.parametrize("out", ["loss", "dz"])
@pytest.mark.parametrize("other", ["logits", "idx", "val", "tokens", "loss", "dz"])
def test_distill_outputs_overlap_nothing(b, out, other):
    if out == other:
        return
    for at in (DAPART[other] + (4 if other == "tokens" else 0), DAPART[other] + DBYTES[other] - 4):
        rc, said = distill(b, **dict(DAPART, **{out: at}))
        assert rc == -1 and "overlap" in said, at


@pytest.mark.parametrize("dz,lddz", [(M, 32), (M + 64, 64), (M - 64, 64)])
def test_distill_in_place_takes_the_same_rows(b, dz, lddz):
    rc, said = distill(b, **dict(DAPART, dz=dz, lddz=lddz))
    assert rc == -1 and "same address and the same row stride" in said


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("name", ["lse", "lens", "table"])
def test_attention_words_are_aligned(b, backward, name):
    rc, said = attention(b, backward, **{name: A + 2})
    assert rc == -1 and "aligned to their elements" in said


def test_attention_table_gradient_is_aligned(b):
    rc, said = attention(b, True, dtable=A + 2)
    assert rc == -1 and "aligned to their elements" in said


@pytest.mark.parametrize("name", ["idx", "val", "tokens", "loss"])
def test_distill_words_are_aligned(b, name):
    rc, said = distill(b, **{name: A + 2})
    assert rc == -1 and "aligned to their elements" in said
