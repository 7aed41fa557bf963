"""Embedding lookup with scaling (bit for bit) and its gradient by sorted tokens
against 64 bits: n additions of fp32 are n 2^-24 sum |dx| off at most, the scaled
addition to the accumulator 2^-24 of the result and of the product."""
import pytest

gpu = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


def error(b):
    import ctypes
    flag = ctypes.c_int()
    b._check(b.lib().gpipe_op_device_error(ctypes.byref(flag), 1, b.current_stream()))
    return flag.value


def lookup(b, tokens, emb, scale, f32, ldx=None):
    import torch
    rows, (vocab, d) = tokens.numel(), emb.shape
    x = torch.full((rows, ldx or d), float("nan"), device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    b._check(b.lib().gpipe_op_embedding_scaled_fwd(0 if f32 else 1, rows, d, vocab, tokens.data_ptr(), emb.data_ptr(),
                                                   scale, x.data_ptr(), ldx or d, b.current_stream()))
    return x


def gradient(b, tokens, dx, d, demb, scale, scratch=None):
    import torch
    rows, vocab, f32 = tokens.numel(), demb.shape[0], dx.dtype == torch.float32
    size = b.lib().gpipe_op_embedding_sorted_bwd_scratch_bytes(rows, d, vocab)
    assert size > 0
    if scratch is None:
        scratch = torch.full((size,), 0xFF, device="cuda", dtype=torch.uint8)
    b._check(b.lib().gpipe_op_embedding_sorted_bwd(0 if f32 else 1, rows, d, vocab, tokens.data_ptr(), dx.data_ptr(),
                                                   dx.stride(0), scale, demb.data_ptr(), scratch.data_ptr(),
                                                   b.current_stream()))
    return scratch


def check_gradient(tokens, dx, d, before, after, scale):
    import numpy as np
    import torch
    scale = float(np.float32(scale))
    vocab = before.shape[0]
    live = (tokens >= 0) & (tokens < vocab)
    t, x = tokens[live].long(), dx[live][:, :d].double()
    total = torch.zeros(vocab, d, device="cuda", dtype=torch.float64).index_add_(0, t, x)
    size = torch.zeros(vocab, d, device="cuda", dtype=torch.float64).index_add_(0, t, x.abs())
    n = torch.zeros(vocab, 1, device="cuda", dtype=torch.float64).index_add_(
        0, t, torch.ones(t.numel(), 1, device="cuda", dtype=torch.float64))
    want = before.double() + scale * total
    tol = U * (1.01 * n * abs(scale) * size + 2 * want.abs() + 2 * abs(scale) * total.abs())
    assert float(((after.double() - want).abs() - tol).max()) <= 0
    untouched = (n == 0)[:, 0]
    assert torch.equal(after[untouched], before[untouched])


def tokens_of(kind, rows, vocab, g):
    import torch
    if kind == "one":
        return torch.full((rows,), vocab - 1, device="cuda", dtype=torch.int32)
    if kind == "sorted":
        return (torch.arange(rows, device="cuda") * vocab // rows).to(torch.int32)
    if kind == "backwards":
        return (vocab - 1 - torch.arange(rows, device="cuda") % vocab).to(torch.int32)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "text":  # a few tokens make up most rows
        u = torch.rand(rows, generator=g, device="cuda")
        t = (vocab ** u - 1).to(torch.int32).clamp(0, vocab - 1)
    if kind == "padded":
        t[rows // 3:rows // 2] = -1
        t[rows - rows // 4:] = -2 ** 31
    return t


@gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,d,vocab,ldx", [(1, 8, 1, 8), (19, 64, 517, 64), (33, 264, 70, 272), (1000, 1024, 3000, 1024),
                                              (513, 2048, 5, 2056), (7, 1000, 100000, 1000)])
def test_lookup_is_the_rounded_product(b, rows, d, vocab, ldx, f32):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    emb = torch.randn(vocab, d, generator=g, device="cuda").bfloat16()
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    if rows > 4:
        tokens[rows // 2], tokens[-1] = -1, -5
    scale = 22.627417
    x = lookup(b, tokens, emb, scale, f32, ldx)
    want = emb[tokens.long().clamp(min=0)].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")
    want[tokens < 0] = 0.0
    assert torch.equal(x[:, :d], want if f32 else want.bfloat16())
    assert bool(torch.isnan(x[:, d:]).all())
    assert error(b) == 0


GRADS = [(1, 8, 1, "uniform"), (2, 8, 1, "one"), (19, 64, 517, "uniform"), (31, 64, 3, "uniform"), (32, 72, 1, "one"),
         (33, 72, 1, "one"), (64, 128, 2, "sorted"), (65, 2048, 2, "uniform"), (100, 264, 40, "padded"),
         (255, 1024, 9, "text"), (256, 2056, 1, "one"), (257, 2056, 1, "one"), (264, 72, 33, "sorted"),
         (1000, 712, 50, "text"), (2048, 1024, 32000, "uniform"), (4097, 512, 300, "text"), (8192, 64, 1000, "text"),
         (8193, 64, 1000, "text"), (9001, 136, 511, "uniform"), (9001, 136, 512, "padded"), (10000, 64, 7, "one"),
         (20000, 256, 131072, "text"), (40000, 64, 262143, "backwards"), (70001, 72, 900, "sorted"),
         (24576, 264, 40, "padded"), (24577, 1096, 40, "padded"), (300000, 16, 50000, "text"), (9000, 24, 400000, "uniform")]


@gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,d,vocab,kind", GRADS)
def test_gradient_against_64_bits(b, rows, d, vocab, kind, f32):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    tokens = tokens_of(kind, rows, vocab, g)
    dx = torch.randn(rows, d + 8, generator=g, device="cuda")
    dx[:, d:] = float("nan")
    dx[tokens < 0] = float("nan")  # padding may hold anything
    dx = dx if f32 else dx.bfloat16()
    before = torch.randn(vocab, d, generator=g, device="cuda")
    after = before.clone()
    gradient(b, tokens, dx, d, after, 0.7)
    check_gradient(tokens, dx, d, before, after, 0.7)
    again = before.clone()
    gradient(b, tokens, dx, d, again, 0.7)
    assert torch.equal(after, again) and error(b) == 0


@gpu
@pytest.mark.parametrize("rows", [50, 9000])
def test_ids_out_of_range_are_flagged_and_left_out(b, rows):
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, 30, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tokens[7], tokens[20], tokens[30] = 30, 2 ** 31 - 1, 512
    emb = torch.randn(30, 64, generator=g, device="cuda").bfloat16()
    x = lookup(b, tokens, emb, 1.0, True)
    assert error(b) == 5 and float(x[[7, 20, 30]].abs().max()) == 0
    dx = torch.randn(rows, 64, generator=g, device="cuda")
    dx[[7, 20, 30]] = float("nan")
    before = torch.randn(30, 64, generator=g, device="cuda")
    after = before.clone()
    gradient(b, tokens, dx, 64, after, 1.0)
    assert error(b) == 5
    check_gradient(tokens, dx, 64, before, after, 1.0)


@gpu
def test_rows_of_a_token_are_added_in_order(b):
    """2^24 + 1 - 2^24 in fp32 is 0 from the left, 1 from the right."""
    import torch
    for rows in (3, 700, 9000):
        tokens = torch.full((rows,), -1, device="cuda", dtype=torch.int32)
        at = [0, rows // 2, rows - 1]
        tokens[at] = 2
        dx = torch.zeros(rows, 8, device="cuda")
        dx[at] = torch.tensor([2.0 ** 24, 1.0, -2.0 ** 24], device="cuda")[:, None]
        demb = torch.zeros(4, 8, device="cuda")
        gradient(b, tokens, dx, 8, demb, 1.0)
        assert float(demb.abs().max()) == 0
        dx[at] = torch.tensor([2.0 ** 24, -2.0 ** 24, 1.0], device="cuda")[:, None]
        gradient(b, tokens, dx, 8, demb, 1.0)
        assert torch.equal(demb[2], torch.ones(8, device="cuda"))


@gpu
@pytest.mark.parametrize("rows", [700, 12000])
def test_the_same_bits_on_any_stream_and_replayed(b, rows):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    tokens = tokens_of("text", rows, 400, g)
    dx = torch.randn(rows, 128, generator=g, device="cuda")
    one, two, three = (torch.zeros(400, 128, device="cuda") for _ in range(3))
    scratch = gradient(b, tokens, dx, 128, one, 1.5)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        gradient(b, tokens, dx, 128, two, 1.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gradient(b, tokens, dx, 128, three, 1.5, scratch)
    three.zero_()
    scratch.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(one, three)
    # new tokens in the captured call
    tokens.copy_(tokens_of("padded", rows, 400, g))
    three.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check_gradient(tokens, dx, 128, torch.zeros_like(three), three, 1.5)


@gpu
def test_both_ends_of_a_tied_model_together(b):
    """Lookup, the head's loss on top of it and both gradients into one accumulator, then the update: each against 64
    bits of what it was given."""
    import torch
    from tests import test_gpu_head_loss as head
    g = torch.Generator(device="cuda").manual_seed(1)
    nseq, seq, d, vocab, scale = 4, 96, 128, 900, 128 ** 0.5
    rows = nseq * seq
    w = torch.randn(vocab, d, generator=g, device="cuda") / d ** 0.5
    emb = w.bfloat16()
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tokens.view(nseq, seq)[1, 60:] = -1  # a shorter sequence
    x = lookup(b, tokens, emb, scale, False)
    p = dict(rows=rows, d=d, vocab=vocab, seq=seq, emb=emb, tokens=tokens, h=x, weight=None)
    grad = torch.zeros(vocab, d, device="cuda")
    o = head.call(b, p, piece=256, f32=True, demb=grad)
    want = head.exact(p)
    head.compare(o, want, d, f32=True)
    mid = grad.clone()
    gradient(b, tokens, o["dh"], d, grad, scale)
    check_gradient(tokens, o["dh"], d, mid, grad, scale)
    v = torch.zeros(vocab, d, device="cuda")
    w0, g0 = w.double(), grad.double()
    b._check(b.lib().gpipe_op_rmsprop(w.numel(), w.data_ptr(), grad.data_ptr(), v.data_ptr(), emb.data_ptr(), 1e-3, 0.9,
                                      1e-8, 1, b.current_stream()))
    ref = w0 - 1e-3 * g0 / ((0.1 * g0 * g0).sqrt() + 1e-8)
    assert float((w.double() - ref).abs().max()) <= 1e-6 and float(grad.abs().max()) == 0
    assert torch.equal(emb, w.bfloat16()) and error(b) == 0


@gpu
@pytest.mark.parametrize("f32", [False, True])
def test_more_than_2_to_the_31_elements(b, f32):
    """Table, rows and accumulator beyond 32-bit offsets, with the tokens and rows that count at their ends."""
    import torch
    vocab, d, rows = 530000, 4096, 530000
    g = torch.Generator(device="cuda").manual_seed(2)
    emb = torch.zeros(vocab, d, device="cuda", dtype=torch.bfloat16)
    tokens = torch.full((rows,), -1, device="cuda", dtype=torch.int32)
    at = torch.tensor([0, 1, 262143, 262144, 524287, 524288, rows - 2, rows - 1], device="cuda")
    ids = torch.tensor([vocab - 1, 3, vocab - 1, vocab - 2, 524288, 3, vocab - 1, 524287], device="cuda", dtype=torch.int32)
    tokens[at] = ids
    emb[ids.long()] = torch.randn(8, d, generator=g, device="cuda").bfloat16()
    x = lookup(b, tokens, emb, 1.5, f32)
    want = emb[ids.long()].float() * 1.5
    assert torch.equal(x[at], want if f32 else want.bfloat16())
    assert float(x[2:262143].abs().max()) == 0 and float(x[524289:rows - 2].abs().max()) == 0
    del emb
    before = torch.zeros(vocab, d, device="cuda")
    before[-1] = 1.0
    x[tokens < 0] = float("nan")
    gradient(b, tokens, x, d, before, 0.5)
    total = torch.zeros(vocab, dtype=torch.float64, device="cuda")
    for i in ids.unique().long().tolist():
        rows_of = x[at[ids == i]].double()
        want = (1.0 if i == vocab - 1 else 0.0) + 0.5 * rows_of.sum(0)
        tol = U * (3 * rows_of.abs().sum(0) + 2 * want.abs() + 1)
        assert float(((before[i].double() - want).abs() - tol).max()) <= 0
        total[i] = 1
    assert float(before[total == 0].abs().max()) == 0
