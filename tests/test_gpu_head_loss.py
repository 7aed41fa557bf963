"""The head's loss without logits against its definition in 64 bits.

Tolerances are worst-case bounds, counted in roundings (u = 2^-24 for fp32):
  z      a product of d terms in fp32: dz = 2 d u max_v sum_k |h_k E_vk| (2 u an
         addition, for tensor cores that truncate)
  loss   w a (2 dz + 8 u (|m| + |z_t| + 1) + e_s), e_s = 2^-20 + 2 u (vocab / 128 + 140):
         z_t and the largest z are dz off each, the exponentials 2^-22 and the argument's
         rounding (d <= 128 in size where it matters: 2^-24 * 128 * 1.5 < 2^-16, weighted by
         e^-128; 2^-20 covers the maximum of x e^-x), the sums an addition each
  g      2^-8 of its value for bf16 (half a step: finfo.eps / 2 = 2^-7 / 2), and e_p = (2 (2 dz + e_s) + 2^-11) p +
         2^-38 for p, which passes through fp16 (2^-11; below 2^-28 of the largest of its 32
         neighbours, at most 1, steps of 2^-38); all of g where |z| is within dz of clip, as it may
         count as beyond it or not
  dh     sum_v |g_v| |E_v| (2^-8 + 2^-10) + e_p sum_v w p_v |E_v|, and 2^-8 of the result
  demb   the same over the rows; 2^-8 of the result as bf16
(2^-10 covers the products' own additions: 2 u times up to 2^13 terms.)"""
import math

import pytest

gpu = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


def make(rows, d, vocab, seq, weights=False, seed=0, ldh=None, know=8.0, size=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    emb = (size * torch.randn(vocab, d, generator=g, device="cuda") / math.sqrt(d)).bfloat16()
    tokens = torch.randint(0, vocab, (rows + 1,), generator=g, device="cuda", dtype=torch.int32)
    h = torch.zeros(rows, ldh or d, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(rows, d, generator=g, device="cuda") + know * torch.rand(rows, 1, generator=g, device="cuda") * \
        emb[tokens[1:].long()].float()
    h[:, :d] = x.bfloat16()
    weight = None
    if weights:
        u = torch.rand(rows, generator=g, device="cuda")
        weight = torch.where(u < 0.3, torch.zeros_like(u), 0.5 + u)
    return dict(rows=rows, d=d, vocab=vocab, seq=seq, emb=emb, tokens=tokens, h=h, weight=weight)


def call(b, p, piece=0, clip=0.0, grads="both", f32=False, inv=None, row0=0, demb=None, lddh=None, buf=None):
    """Outputs of one call: loss, dh, demb (None where not wanted)."""
    import torch
    rows, d, vocab = p["rows"], p["d"], p["vocab"]
    want = {"none": 0, "h": 1, "e": 2, "both": 3}[grads]
    inv = inv if inv is not None else 1.0 / rows
    o = buf if buf is not None else {}
    if not o:
        o["loss"] = torch.full((rows,), float("nan"), device="cuda")
        o["dh"] = torch.full((rows, lddh or d), float("nan"), device="cuda", dtype=torch.bfloat16) if want & 1 else None
        if want & 2:
            o["demb"] = demb if demb is not None else (
                torch.zeros(vocab, d, device="cuda") if f32 else
                torch.full((vocab, d), float("nan"), device="cuda", dtype=torch.bfloat16))
        else:
            o["demb"] = None
        size = b.lib().gpipe_op_head_loss_scratch_bytes(rows, d, vocab, piece, want)
        assert size > 0
        o["scratch"] = torch.full((size,), 0xFF, device="cuda", dtype=torch.uint8)  # NaN wherever it is not written
    ptr = b._ptr
    b._check(b.lib().gpipe_op_head_loss(rows, d, vocab, ptr(p["h"]), p["h"].stride(0), ptr(p["emb"]), p["seq"],
                                        ptr(p["tokens"]), row0, ptr(p["weight"]), inv, clip, piece, ptr(o["loss"]),
                                        ptr(o["dh"]), lddh or d, 0 if f32 else 1, ptr(o["demb"]), ptr(o["scratch"]),
                                        b.current_stream()))
    return o


def exact(p, clip=0.0, inv=None, row0=0):
    """Definition in 64 bits, with the bounds of the docstring."""
    import torch
    rows, d, vocab, seq = p["rows"], p["d"], p["vocab"], p["seq"]
    inv = inv if inv is not None else 1.0 / rows
    r = torch.arange(rows, device="cuda") + row0
    has = r % seq != seq - 1
    t = torch.zeros(rows, device="cuda", dtype=torch.long)
    t[has] = p["tokens"].long()[r[has] + 1]
    has &= (t >= 0) & (t < vocab)
    w = torch.ones(rows, device="cuda", dtype=torch.float64) if p["weight"] is None else p["weight"].double()
    w = torch.where(has, w, torch.zeros_like(w))
    t = t.clamp(0, vocab - 1)
    live = w != 0
    h = torch.where(live[:, None], p["h"][:, :d].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    e = p["emb"].double()
    z = h @ e.T
    dz = (2 * d * U * (h.abs() @ e.abs().T).amax(1))[:, None]
    inside, either = torch.ones_like(z), torch.zeros_like(z)
    if clip > 0:
        either = ((z.abs() - clip).abs() <= dz).double()  # too near the limit to say on which side it is
        inside = (z.abs() < clip).double()
        z = z.clamp(-clip, clip)
    m = z.amax(1, keepdim=True)
    s = (z - m).exp().sum(1, keepdim=True)
    zt = z.gather(1, t[:, None])
    e_s = 2.0 ** -20 + 2 * U * (vocab / 128 + 140)
    loss = (w[:, None] * inv * (m - zt + s.log()))[:, 0]
    loss_tol = (w[:, None].abs() * abs(inv) * (2 * dz + 8 * U * (m.abs() + zt.abs() + 1) + e_s))[:, 0]
    pr = (z - m).exp() / s
    gr = pr.clone()
    gr.scatter_add_(1, t[:, None], -torch.ones_like(zt))
    slack = either * gr.abs() * w[:, None].abs()
    gr *= w[:, None] * inside
    e_p = ((2 * (2 * dz + e_s) + 2.0 ** -11) * pr + 2.0 ** -38) * w[:, None].abs() * inside
    slack += gr.abs() * (2.0 ** -8 + 2.0 ** -10) + e_p
    a = abs(inv)
    dh, demb = inv * (gr @ e), inv * (gr.T @ h)
    return dict(loss=loss, loss_tol=loss_tol, dh=dh, dh_tol=a * (slack @ e.abs()) * 1.01 + 2.0 ** -8 * dh.abs(), demb=demb,
                demb_tol=a * (slack.T @ h.abs()) * 1.01)


def compare(o, x, d, f32=False, before=None):
    def near(got, want, tol, name):
        over = ((got.double() - want).abs() - tol).max()
        assert float(over) <= 0, (name, float(over), float(tol.mean()))
    near(o["loss"], x["loss"], x["loss_tol"] + 1e-30, "loss")
    if o["dh"] is not None:
        near(o["dh"][:, :d], x["dh"], x["dh_tol"] + 1e-30, "dh")
    if o["demb"] is not None:
        want = x["demb"] if before is None else x["demb"] + before.double()
        tol = x["demb_tol"] + 1e-30 + (8 * U if f32 else 2.0 ** -8) * want.abs()
        near(o["demb"], want, tol, "demb")


# rows, d, vocab, seq, piece, clip, weights, grads, f32 accumulator
FORMS = [
    (1, 8, 1, 2, 0, 0.0, False, "both", False),
    (1, 64, 1000, 5, 0, 0.0, False, "none", False),
    (1, 1024, 5000, 2, 0, 0.0, False, "both", True),
    (2, 8, 2, 3, 0, 0.0, False, "both", True),
    (1, 8, 1, 2, 0, 0.0, False, "none", False),
    (31, 136, 517, 4, 0, 4.0, True, "none", False),
    (64, 1024, 9001, 64, 0, 0.0, False, "none", False),
    (65, 200, 9001, 64, 0, 4.0, False, "none", False),
    (3, 248, 40000, 5, 0, 0.0, False, "both", False),
    (2000, 64, 20011, 90, 0, 5.0, True, "none", False),
    (1300, 784, 2900, 90, 1024, 4.0, True, "both", False),
    (5, 64, 517, 5, 0, 0.0, False, "both", False),
    (7, 72, 255, 3, 256, 0.0, False, "both", True),
    (33, 200, 257, 11, 256, 0.0, True, "both", False),
    (64, 64, 256, 64, 0, 6.0, False, "both", False),
    (127, 128, 1025, 16, 512, 0.0, True, "both", True),
    (128, 256, 4096, 32, 1024, 0.0, False, "h", False),
    (129, 264, 4097, 43, 0, 0.0, False, "e", False),
    (255, 512, 3001, 255, 1024, 0.0, True, "both", False),
    (257, 1000, 2050, 100, 768, 5.0, True, "both", True),
    (300, 8, 33, 7, 0, 0.0, False, "both", False),
    (512, 512, 8000, 128, 0, 0.0, False, "both", False),
    (512, 512, 8000, 128, 2048, 0.0, False, "both", True),
    (1000, 712, 5003, 59, 1024, 0.0, True, "both", False),
    (2048, 1024, 4000, 512, 0, 0.0, False, "both", False),
    (3000, 96, 700, 1000, 0, 0.0, False, "both", False),
    (4100, 320, 513, 64, 256, 0.0, True, "both", True),
    (2048, 712, 6001, 90, 0, 0.0, True, "both", False),
    (2048, 712, 6001, 90, 2048, 5.0, True, "both", True),
    (3000, 136, 22000, 1000, 0, 0.0, True, "none", False),
    (64, 1032, 131073, 50, 0, 0.0, False, "none", False),
    (65, 1032, 131073, 50, 0, 0.0, True, "none", False),
    (3000, 264, 11000, 1000, 0, 0.0, False, "h", False),
]


@gpu
@pytest.mark.parametrize("form", FORMS, ids=["-".join(map(str, f)) for f in FORMS])
def test_against_64_bits(b, form):
    rows, d, vocab, seq, piece, clip, weights, grads, f32 = form
    p = make(rows, d, vocab, seq, weights, seed=rows + d)
    import torch
    before = torch.randn(vocab, d, device="cuda") / rows if f32 else None
    o = call(b, p, piece, clip, grads, f32, demb=before.clone() if f32 and grads in ("e", "both") else None)
    compare(o, exact(p, clip), d, f32, before)


@gpu
def test_padded_leading_dimensions_and_a_later_part_of_the_batch(b):
    """h and dh inside wider rows, whose other columns stay as they were; rows from token row0 on."""
    import torch
    p = make(96, 72, 700, 10, ldh=88)
    p["h"][:, 72:] = float("nan")
    p["tokens"] = torch.cat([torch.randint(0, 700, (37,), device="cuda", dtype=torch.int32), p["tokens"]])
    o = call(b, p, row0=37, lddh=80)
    compare(o, exact(p, row0=37), 72)
    assert bool(torch.isnan(o["dh"][:, 72:]).all())


@gpu
def test_rows_that_count_for_nothing_may_hold_anything(b):
    """No target (a negative id, the end of a sequence) or weight 0: zeros, and no trace of the NaN and inf in h."""
    import torch
    p = make(40, 64, 300, 8, seed=3)
    p["weight"] = torch.ones(40, device="cuda")
    p["weight"][5] = 0.0
    p["tokens"][11] = -1   # row 10
    p["tokens"][31] = -7   # row 30
    dead = [5, 10, 30] + list(range(7, 40, 8))
    p["h"][dead] = float("nan")
    p["h"][10] = float("inf")
    o = call(b, p, piece=256)
    x = exact(p)
    compare(o, x, 64)
    assert float(o["loss"][dead].abs().max()) == 0 and float(o["dh"][dead].float().abs().max()) == 0
    assert b_error(b) == 0


def b_error(b):
    import ctypes
    flag = ctypes.c_int()
    b._check(b.lib().gpipe_op_device_error(ctypes.byref(flag), 1, b.current_stream()))
    return flag.value


@gpu
def test_nothing_to_learn(b):
    """Every row without a target: zeros, and an accumulator that keeps its bits."""
    import torch
    p = make(20, 64, 300, 1)
    before = torch.randn(300, 64, device="cuda")
    o = call(b, p, f32=True, demb=before.clone())
    assert float(o["loss"].abs().max()) == 0 and float(o["dh"].float().abs().max()) == 0
    assert torch.equal(o["demb"], before)


@gpu
def test_ids_out_of_range_are_flagged(b):
    import torch
    p = make(20, 64, 300, 20)
    p["tokens"][4] = 300
    p["tokens"][9] = 2 ** 31 - 1
    assert b_error(b) == 0
    o = call(b, p)
    assert b_error(b) == 5
    assert float(o["loss"][[3, 8]].abs().max()) == 0
    compare(o, exact(p), 64)
    del torch


@gpu
def test_large_logits(b):
    """Logits of several hundreds, far apart: p is 0 or 1 for most rows, and the loss keeps its digits."""
    p = make(130, 256, 1500, 13, seed=8, know=30.0, size=20.0)
    compare(call(b, p), exact(p), 256)


@gpu
@pytest.mark.parametrize("rows", [20, 64, 65, 300])
@pytest.mark.parametrize("grads", ["none", "both"])
def test_huge_logits_with_ties(b, rows, grads):
    """Logits that are whole multiples of 2^18 up to 2^24, exact in fp32: p is 1 / k for the k largest and 0 otherwise, and
    the loss a multiple of 2^18 plus ln k, to 8 roundings of its size.  (20 rows: the powers kept; 300: z made again.)"""
    import torch
    d, vocab = 64, 1000
    g = torch.Generator(device="cuda").manual_seed(rows)
    h = (torch.randint(-1, 2, (rows, d), generator=g, device="cuda").float() * 2.0 ** 10)
    emb = (torch.randint(-1, 2, (vocab, d), generator=g, device="cuda").float() * 2.0 ** 8)
    emb[1::2] = emb[::2]                      # every logit twice
    h[0], emb[10], emb[11] = 2.0 ** 10, 2.0 ** 8, 2.0 ** 8   # 2^24 itself
    tokens = torch.randint(0, vocab, (rows + 1,), generator=g, device="cuda", dtype=torch.int32)
    z = h.double() @ emb.double().T
    tokens[2::3] = z.argmax(1)[1::3].to(torch.int32)  # some targets among the largest
    p = dict(rows=rows, d=d, vocab=vocab, seq=rows + 1, emb=emb.bfloat16(), tokens=tokens, h=h.bfloat16(), weight=None)
    o = call(b, p, grads=grads, inv=1.0)
    t, n = tokens[1:].long(), torch.arange(rows, device="cuda")
    logp = torch.log_softmax(z, 1)
    loss = -logp[n, t]
    assert float(((o["loss"].double() - loss).abs() - 8 * U * (loss.abs() + z.abs().amax(1)) - 2.0 ** -18).max()) <= 0
    small = loss < 100
    assert bool(small.any()) and float((o["loss"].double() - loss)[small].abs().max()) <= 2.0 ** -18
    if grads == "none":
        return
    grad = logp.exp()
    grad[n, t] -= 1
    e, hd = emb.double(), h.double()
    slack = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18
    dh, demb = grad @ e, grad.T @ hd
    assert float(((o["dh"].double() - dh).abs() - slack * (grad.abs() @ e.abs()) - 2.0 ** -8 * dh.abs()).max()) <= 0
    tol = slack * (grad.abs().T @ hd.abs()) + 2.0 ** -8 * demb.abs()
    assert float(((o["demb"].double() - demb).abs() - tol).max()) <= 0


@gpu
def test_nan_and_inf_in_rows_that_count(b):
    """They show in their own row's loss and dh, and in no other row's."""
    import torch
    p = make(30, 64, 300, 30, seed=2)
    good = call(b, p)
    p["h"][4, 3] = float("nan")
    o = call(b, p)
    assert bool(torch.isnan(o["loss"][4])) and bool(torch.isnan(o["dh"][4]).all())
    rest = [r for r in range(30) if r != 4]
    assert torch.equal(o["loss"][rest], good["loss"][rest]) and torch.equal(o["dh"][rest], good["dh"][rest])


@gpu
def test_the_same_bits_on_any_stream_and_replayed(b):
    import torch
    p = make(300, 200, 3001, 60, True)
    first = call(b, p, piece=1024)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = call(b, p, piece=1024)
    torch.cuda.current_stream().wait_stream(other)
    graph = torch.cuda.CUDAGraph()
    buf = call(b, p, piece=1024)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(b, p, piece=1024, buf=buf)
    for k in ("loss", "dh", "demb"):
        buf[k].fill_(7.0)
    buf["scratch"].fill_(0xFF)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in ("loss", "dh", "demb"):
        assert torch.equal(first[k], second[k]) and torch.equal(first[k], buf[k])


@gpu
def test_two_calls_at_once(b):
    import torch
    p, q = make(700, 256, 3001, 60, seed=1), make(650, 256, 2999, 50, seed=2)
    one, two = call(b, p, piece=512), call(b, q, piece=512)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, x in enumerate((p, q)):
            with torch.cuda.stream(s[i]):
                got[i].append(call(b, x, piece=512))
    torch.cuda.synchronize()
    for want, have in ((one, got[0]), (two, got[1])):
        for o in have:
            assert all(torch.equal(want[k], o[k]) for k in ("loss", "dh", "demb"))


@gpu
def test_pieces_of_any_size(b):
    p = make(200, 136, 5000, 40)
    x = exact(p)
    for piece in (0, 1, 256, 1000, 4096, 5000, 100000):
        compare(call(b, p, piece=piece), x, 136)


@gpu
def test_gradients_against_differences(b):
    """loss(x + step) - loss(x - step) over 2 step, for a direction in h and one in E.  bf16 inputs leave room only for
    steps of their spacing, so the step is what the inputs really moved by.  The loss is smooth on that scale: third
    derivatives are below 1 (p in [0, 1]) times the cube of a logit's move, which is under 0.05."""
    import torch
    p = make(64, 64, 400, 64, know=3.0)
    o = call(b, p, f32=True, inv=1.0)
    g = torch.Generator(device="cuda").manual_seed(9)
    for name, grad in (("h", o["dh"]), ("emb", o["demb"])):
        base = p[name].clone()
        step = (torch.randn(base.shape, generator=g, device="cuda") * (2.0 ** -7 if name == "h" else 2.0 ** -10))
        up, down = (base.float() + step).bfloat16(), (base.float() - step).bfloat16()
        p[name] = up
        hi = call(b, p, grads="none", inv=1.0)["loss"].double().sum()
        p[name] = down
        lo = call(b, p, grads="none", inv=1.0)["loss"].double().sum()
        p[name] = base
        move = (up.double() - down.double()) / 2
        off = ((up.double() + down.double()) / 2 - base.double())
        want = (grad.double() * move).sum()
        # the midpoint is off by the roundings: second derivatives below 1/4 times the logits' moves
        scale = float((grad.double().abs() * move.abs()).sum())
        assert abs(float((hi - lo) / 2 - want)) <= 0.02 * scale + 1e-3, (name, float((hi - lo) / 2), float(want), scale,
                                                                         float(off.abs().max()))


@gpu
@pytest.mark.parametrize("grads", ["none", "h", "both"])
@pytest.mark.parametrize("rows,d,vocab,piece", [(40, 64, 3000, 1024), (300, 800, 2000, 0), (700, 128, 9000, 2048)])
def test_calls_in_a_row_that_write_each_others_inputs(b, grads, rows, d, vocab, piece):
    """Launches overlap their predecessors: hidden states, table and tokens that a kernel of the library writes right
    before a call and right after it, against the same calls one at a time."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    tables = [(torch.randn(vocab, d, generator=g, device="cuda") / d ** 0.5) for _ in range(3)]
    p = make(rows, d, vocab, 37)
    source = [torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32) for _ in range(3)]

    def chain(wait):
        got, emb, h = [], torch.empty_like(p["emb"]), torch.empty_like(p["h"])
        q = dict(p, emb=emb, h=h)
        buf = call(b, dict(p), piece, grads=grads)  # (its scratch and outputs are used again)
        lib, stream = b.lib(), b.current_stream()
        for i in range(6):
            b._check(lib.gpipe_op_cast_bf16(emb.numel(), tables[i % 3].data_ptr(), emb.data_ptr(), stream))
            b._check(lib.gpipe_op_embedding_scaled_fwd(1, rows, d, vocab, source[(i + 1) % 3].data_ptr(), emb.data_ptr(),
                                                       3.0, h.data_ptr(), d, stream))
            if wait:
                torch.cuda.synchronize()
            call(b, q, piece, grads=grads, buf=buf)
            if wait:
                torch.cuda.synchronize()
            keep = {}
            for k in ("loss", "dh", "demb"):
                if buf[k] is not None:  # copied by a kernel of torch's, which waits for the call to end
                    keep[k] = buf[k].clone()
            got.append(keep)
        torch.cuda.synchronize()
        return got
    for one, other in zip(chain(True), chain(False)):
        for k in one:
            assert torch.equal(one[k], other[k]), k
    # and without a foreign kernel between the calls
    alone, emb, h = [], torch.empty_like(p["emb"]), torch.empty_like(p["h"])
    lib, stream = b.lib(), b.current_stream()
    bufs = [call(b, dict(p), piece, grads=grads) for _ in range(6)]
    torch.cuda.synchronize()
    for i in range(6):
        b._check(lib.gpipe_op_cast_bf16(emb.numel(), tables[i % 3].data_ptr(), emb.data_ptr(), stream))
        b._check(lib.gpipe_op_embedding_scaled_fwd(1, rows, d, vocab, source[(i + 1) % 3].data_ptr(), emb.data_ptr(), 3.0,
                                                   h.data_ptr(), d, stream))
        alone.append(call(b, dict(p, emb=emb, h=h), piece, grads=grads, buf=bufs[i]))
    torch.cuda.synchronize()
    for one, other in zip(chain(True), alone):
        for k in one:
            assert torch.equal(one[k], other[k]), k


@gpu
@pytest.mark.parametrize("f32", [False, True])
def test_a_table_of_more_than_2_to_the_31_elements(b, f32):
    """Targets at both ends; h near 0, so that p is about 1 / vocab everywhere but at the target, and the rows of dE can be
    checked where they matter without the whole of it in 64 bits."""
    import torch
    rows, d, vocab = 24, 8192, 270001
    g = torch.Generator(device="cuda").manual_seed(7)
    emb = torch.empty(vocab, d, device="cuda", dtype=torch.bfloat16)
    for r0 in range(0, vocab, 20000):
        emb[r0:r0 + 20000] = (torch.randn(emb[r0:r0 + 20000].shape, generator=g, device="cuda") / d ** 0.5).bfloat16()
    tokens = torch.randint(0, vocab, (rows + 1,), generator=g, device="cuda", dtype=torch.int32)
    tokens[1], tokens[2], tokens[3] = vocab - 1, vocab - 2, 0
    h = torch.randn(rows, d, generator=g, device="cuda").bfloat16()
    p = dict(rows=rows, d=d, vocab=vocab, seq=rows + 1, emb=emb, tokens=tokens, h=h, weight=None)
    demb = torch.ones(vocab, d, device="cuda") if f32 else None
    o = call(b, p, piece=65536, f32=f32, demb=demb, inv=1.0)
    z = torch.cat([h.double() @ emb[r0:r0 + 20000].double().T for r0 in range(0, vocab, 20000)], 1)
    t = tokens[1:].long()
    logp = torch.log_softmax(z, 1)
    n = torch.arange(rows, device="cuda")
    dz = 2 * d * U * float((h.double().abs() @ emb[t].double().abs().T).max()) * 2
    assert float((o["loss"].double() + logp[n, t]).abs().max()) <= 2 * dz + 2.0 ** -18
    grad = logp.exp()
    grad[n, t] -= 1
    dh = torch.zeros(rows, d, device="cuda", dtype=torch.float64)
    size = torch.zeros_like(dh)
    for r0 in range(0, vocab, 20000):
        e = emb[r0:r0 + 20000].double()
        dh += grad[:, r0:r0 + 20000] @ e
        size += grad[:, r0:r0 + 20000].abs() @ e.abs()
    slack = 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11 + 4 * dz + 2.0 ** -18
    assert float(((o["dh"].double() - dh).abs() - (slack * size + 2.0 ** -8 * dh.abs())).max()) <= 0
    at = torch.cat([t, torch.tensor([1, 65535, 65536, 262143, 262144, vocab - 3], device="cuda")])
    want = grad[:, at].T @ h.double()
    tol = slack * (grad[:, at].abs().T @ h.double().abs()) + 2.0 ** -36
    if f32:
        want, tol = want + 1, tol + 8 * U * (want.abs() + 1)
    else:
        tol = tol + 2.0 ** -8 * want.abs()
    assert float(((o["demb"][at].double() - want).abs() - tol).max()) <= 0
