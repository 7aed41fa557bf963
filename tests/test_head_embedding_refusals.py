"""Each refusal of the head's loss and of the scaled embedding by its own message,
and the sizes of their scratch.  The calls' pointers overlap on purpose, which is
refused last: a check that has gone missing shows as the overlap's message, and
nothing is launched on addresses that do not exist.  No CUDA call is made here."""
import pytest


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import _build
    _build.build()
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


A = 1 << 20   # every pointer: aligned for everything
NAN, INF = float("nan"), float("inf")
HEAD = dict(rows=4, d=64, vocab=300, h=A, ldh=64, emb=A, seq=4, tokens=A, row0=0, weight=A, inv=0.25, clip=0.0, piece=0,
            loss=A, dh=A, lddh=64, dtype=1, demb=A, scratch=A)


def head(b, **kw):
    a = dict(HEAD, **kw)
    lib = b.lib()
    rc = lib.gpipe_op_head_loss(a["rows"], a["d"], a["vocab"], a["h"] or None, a["ldh"], a["emb"] or None, a["seq"],
                                a["tokens"] or None, a["row0"], a["weight"] or None, a["inv"], a["clip"], a["piece"],
                                a["loss"] or None, a["dh"] or None, a["lddh"], a["dtype"], a["demb"] or None,
                                a["scratch"] or None, None)
    return rc, lib.gpipe_last_error(None).decode()


@pytest.mark.parametrize("kw", [{}, dict(dh=0), dict(demb=0), dict(dh=0, demb=0), dict(weight=0), dict(dtype=0),
                                dict(demb=0, dtype=7), dict(dh=0, lddh=0)])
def test_head_calls_that_only_overlap(b, kw):
    rc, said = head(b, **kw)
    assert rc == -1 and "overlap" in said


SIZES, H, SEQ, NUMBERS = "1 <= rows <= 2^24", "16-B aligned h and emb", "seq >= 1", "finite inv_count"


@pytest.mark.parametrize("bad,words", [
    (dict(rows=0), SIZES), (dict(rows=-3), SIZES), (dict(rows=(1 << 24) + 1), SIZES), (dict(d=0), SIZES),
    (dict(d=4), SIZES), (dict(d=60), SIZES), (dict(d=(1 << 16) + 8), SIZES), (dict(vocab=0), SIZES),
    (dict(vocab=(1 << 27) + 1), SIZES), (dict(piece=-1), SIZES),
    (dict(rows=1 << 24, vocab=1 << 27), SIZES),   # 2^16 x 2^19 tiles
    (dict(seq=0), SEQ), (dict(seq=-1), SEQ), (dict(row0=-1), SEQ), (dict(row0=2 ** 31 - 5), SEQ),
    (dict(inv=NAN), NUMBERS), (dict(inv=INF), NUMBERS), (dict(inv=-INF), NUMBERS), (dict(clip=-1.0), NUMBERS),
    (dict(clip=NAN), NUMBERS), (dict(clip=INF), NUMBERS),
    (dict(h=0), H), (dict(h=A + 8), H), (dict(emb=0), H), (dict(emb=A + 4), H), (dict(ldh=56), H), (dict(ldh=68), H),
    (dict(tokens=0), "aligned to their elements"), (dict(tokens=A + 2), "aligned to their elements"),
    (dict(weight=A + 1), "aligned to their elements"), (dict(loss=0), "aligned to their elements"),
    (dict(loss=A + 2), "aligned to their elements"), (dict(dh=A + 8), "16-B aligned dh"),
    (dict(lddh=56), "16-B aligned dh"), (dict(lddh=65), "16-B aligned dh"), (dict(demb=A + 8), "demb must be"),
    (dict(scratch=0), "256-B aligned"), (dict(scratch=A + 128), "256-B aligned")])
def test_head_refusals(b, bad, words):
    rc, said = head(b, **bad)
    assert rc == -1 and words in said and "overlap" not in said


def test_head_refuses_other_types(b):
    for dtype in (-1, 2):
        rc, said = head(b, dtype=dtype)
        assert rc == -6 and "demb_dtype" in said


# tensors that do not touch each other: 4 rows of 64, 300 x 64 table
M = 1 << 21
APART = dict(h=M, emb=2 * M, tokens=3 * M, weight=4 * M, loss=5 * M, dh=6 * M, demb=7 * M, scratch=8 * M)
BYTES = dict(h=512, emb=300 * 128, tokens=16, weight=16, loss=16, dh=512, demb=300 * 128)


@pytest.mark.parametrize("out", ["loss", "dh", "demb", "scratch"])
@pytest.mark.parametrize("other", ["h", "emb", "tokens", "weight", "loss", "dh", "demb", "scratch"])
def test_head_outputs_overlap_nothing(b, out, other):
    if out == other:
        return
    sizes = dict(BYTES, scratch=b.lib().gpipe_op_head_loss_scratch_bytes(4, 64, 300, 0, 3))
    step = 256 if out == "scratch" else 16
    # (of the tokens, the first is not read, and the last row has no target)
    first = APART[other] + (4 if other == "tokens" and step == 16 else 0)
    first += -first % 16 if out in ("dh", "demb") and other == "tokens" else 0
    ends = {first if other != "tokens" or out == "loss" else APART[other], APART[other] + (sizes[other] - 16) // step * step}
    for at in ends:
        rc, said = head(b, **dict(APART, **{out: at}))
        assert rc == -1 and "overlap" in said, at


def test_head_scratch_bytes(b):
    f = b.lib().gpipe_op_head_loss_scratch_bytes
    # sums of a row: 16 bytes a tile of 256 columns; up to 64 rows without gradients 64 (a sum each 32 columns)
    assert f(100, 64, 1000, 0, 0) == 100 * 4 * 16 and f(64, 64, 1000, 0, 0) == 64 * 4 * 64
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    rows, d, vocab = 1000, 712, 50001
    tiles = 196
    info, copy, g = up(rows * 16), up(rows * 768 * 2), 2 * up(rows * 8192 * 2)  # (several pieces: g of two)
    assert f(rows, d, vocab, 8192, 2) == up(rows * tiles * 16) + info + copy + g
    assert f(rows, d, vocab, 8000, 2) == f(rows, d, vocab, 8192, 2)
    # (a copy of h: for dE, and for any large call, whose h may not lie on 32-byte rows)
    with_dh = f(rows, d, vocab, 8192, 1) - (up(rows * tiles * 16) + info + copy + g)
    assert with_dh > 0 and with_dh % (1024 * d * 4) == 0          # parts of 1024 rows
    # all of the vocabulary in one piece, however wide it is asked for
    assert f(64, 64, 1000, 1 << 20, 3) == f(64, 64, 1000, 1024, 3) == f(64, 64, 1000, 0, 3)
    # 256 MB of g at most, unless that is under 2048 columns
    assert 2 ** 28 < f(8192, 64, 131072, 0, 2) < 2 ** 28 + 8192 * (512 * 16 + 16 + 128 + 64)
    assert f(8192, 64, 131072, 0, 2) == f(8192, 64, 131072, 8192, 2)
    for bad in ((0, 64, 10, 0, 0), (1, 4, 10, 0, 0), (1, 64, 0, 0, 0), (1, 64, 10, -1, 0), (1, 64, 10, 0, 4),
                (1, 64, 10, 0, -1), (1 << 24, 64, 1 << 27, 0, 0)):
        assert f(*bad) == 0


EMBED = dict(dtype=0, rows=4, d=64, vocab=300, tokens=A, emb=A, scale=1.0, x=A, ld=64, demb=A, scratch=A)


def embed(b, backward, **kw):
    a = dict(EMBED, **kw)
    lib = b.lib()
    if backward:
        rc = lib.gpipe_op_embedding_sorted_bwd(a["dtype"], a["rows"], a["d"], a["vocab"], a["tokens"] or None,
                                               a["x"] or None, a["ld"], a["scale"], a["demb"] or None,
                                               a["scratch"] or None, None)
    else:
        rc = lib.gpipe_op_embedding_scaled_fwd(a["dtype"], a["rows"], a["d"], a["vocab"], a["tokens"] or None,
                                               a["emb"] or None, a["scale"], a["x"] or None, a["ld"], None)
    return rc, lib.gpipe_last_error(None).decode()


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [0, 1])
def test_embedding_calls_that_only_overlap(b, backward, dtype):
    rc, said = embed(b, backward, dtype=dtype)
    assert rc == -1 and "overlap" in said


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad,words", [
    (dict(rows=0), "1 <= rows <= 2^27"), (dict(rows=(1 << 27) + 1), "1 <= rows <= 2^27"),
    (dict(d=0), "d % 8 == 0"), (dict(d=12), "d % 8 == 0"), (dict(d=(1 << 16) + 8), "d % 8 == 0"),
    (dict(vocab=0), "vocab <= 2^30"), (dict(vocab=(1 << 30) + 1), "vocab <= 2^30"),
    (dict(scale=NAN), "finite"), (dict(scale=INF), "finite"), (dict(scale=-INF), "finite"),
    (dict(tokens=0), "need tokens"), (dict(tokens=A + 2), "need tokens"), (dict(x=0), "16-B aligned"),
    (dict(x=A + 8), "16-B aligned"), (dict(ld=56), "a multiple of 8"), (dict(ld=68), "a multiple of 8")])
def test_embedding_refusals(b, backward, bad, words):
    rc, said = embed(b, backward, **bad)
    assert rc == -1 and words in said and "overlap" not in said


@pytest.mark.parametrize("bad,words", [(dict(emb=0), "16-B aligned"), (dict(emb=A + 8), "16-B aligned")])
def test_lookup_refusals(b, bad, words):
    rc, said = embed(b, False, **bad)
    assert rc == -1 and words in said and "overlap" not in said


@pytest.mark.parametrize("bad,words", [
    (dict(demb=0), "16-B aligned"), (dict(demb=A + 8), "16-B aligned"), (dict(scratch=0), "256-B aligned"),
    (dict(scratch=A + 64), "256-B aligned")])
def test_embedding_gradient_refusals(b, bad, words):
    rc, said = embed(b, True, **bad)
    assert rc == -1 and words in said and "overlap" not in said


@pytest.mark.parametrize("backward", [False, True])
def test_embedding_refuses_other_types(b, backward):
    for dtype in (-1, 2):
        rc, said = embed(b, backward, dtype=dtype)
        assert rc == -6 and "dtype must be 0 or 1" in said


EAPART = dict(tokens=M, emb=2 * M, x=3 * M, demb=4 * M, scratch=5 * M)


@pytest.mark.parametrize("other,size", [("tokens", 16), ("emb", 300 * 128)])
def test_lookup_overlaps_nothing(b, other, size):
    for at in (EAPART[other], EAPART[other] + size - 16):
        rc, said = embed(b, False, **dict(EAPART, x=at))
        assert rc == -1 and "overlap" in said


@pytest.mark.parametrize("out", ["demb", "scratch"])
@pytest.mark.parametrize("other,size", [("tokens", 16), ("x", 4 * 256), ("demb", 300 * 256), ("scratch", 0)])
def test_embedding_gradient_overlaps_nothing(b, out, other, size):
    if out == other:
        return
    size = size or b.lib().gpipe_op_embedding_sorted_bwd_scratch_bytes(4, 64, 300)
    step = 256 if out == "scratch" else 16
    for at in (EAPART[other], EAPART[other] + (size - 16) // step * step):
        rc, said = embed(b, True, **dict(EAPART, **{out: at}))
        assert rc == -1 and "overlap" in said


def test_embedding_scratch_bytes(b):
    f = b.lib().gpipe_op_embedding_sorted_bwd_scratch_bytes
    up = lambda n: -(-n // 256) * 256  # noqa: E731

    def want(rows, d):
        run = 8 if rows <= 24576 else 64
        runs = -(-rows // run)
        return 4 * up((rows + 64) * 4) + 4 * 128 * 512 * 4 + up((runs + 2) * 4) + up(runs * 2 * d * 4)
    for rows, d in ((1, 8), (19, 64), (24576, 1024), (24577, 1024), (131072, 512)):
        assert f(rows, d, 1000) == want(rows, d) == f(rows, d, 1)
    for bad in ((0, 64, 10), (1, 12, 10), (1, 64, 0), (1, 64, (1 << 30) + 1)):
        assert f(*bad) == 0
