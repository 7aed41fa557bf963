"""Windowed attention and distillation in forms that the other tests leave out: many
query heads over one key/value head, many blocks far from the sinks, tensors of more
than 2^31 elements, rows that no cluster holds, outputs beside or over other tensors."""
import numpy as np
import pytest

from tests.gpu_util import KEEP, dev, sync
from tests.gpu_util import stream as cur_stream
from tests.test_gpu_window_distill import HD, U, Case, Distill, b, distill_ref, np64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    # nseq, seq, heads, kv, window, sinks, buckets, max_distance, lens
    (1, 300, 8, 1, 100, 5, 8, 60, None),
    (2, 200, 16, 1, 64, 0, 0, 0, [200, 77]),
    (1, 260, 32, 2, 260, 0, 32, 128, None),
    (1, 400, 16, 1, 30, 33, 17, 300, None),
    (1, 129, 64, 1, 20, 2, 64, 100, None),
])
def test_many_heads_over_one_key_value_head(b, shape):  # noqa: F811
    import torch
    c = Case(b, *shape[:8], lens=shape[8])
    c.fwd()
    c.bwd()
    c.check()
    first = c.dqkv.clone()
    c.dqkv.fill_(7.0)
    c.bwd()
    sync()
    assert torch.equal(first, c.dqkv)


@pytest.mark.parametrize("shape", [
    (1, 5003, 2, 1, 300, 64, 32, 128, None),      # 36 query blocks far from 64 sinks
    (1, 4100, 1, 1, 1, 3, 0, 0, None),
    (1, 4097, 2, 2, 2000, 16, 32, 1024, [4090]),
])
def test_long_sequences(b, shape):  # noqa: F811
    c = Case(b, *shape[:8], lens=shape[8])
    c.fwd()
    c.bwd()
    c.check()


def test_the_table_takes_its_own_gradient(b):  # noqa: F811
    c = Case(b, 2, 300, 2, 1, 90, 4, 16, 64)
    c.fwd()
    c.bwd()
    sync()
    grad = np64(c.dtable) - c.dtable0
    before = np64(c.table)
    c.dtable = c.table
    c.bwd()
    sync()
    # two roundings to fp32: of the first sum, and of this one
    tol = 2.0 ** -24 * (np.abs(before + grad) + np.abs(grad + c.dtable0)) * 1.01
    assert np.all(np.abs(np64(c.table) - (before + grad)) <= tol)


def test_tensors_beyond_2_31_elements(b):  # noqa: F811
    """The first and the last sequence of a batch have the bits of a call with those two alone."""
    import torch as t
    lib = b.lib()
    n, s, h, kv, window, sinks, nb, md = 1100, 1000, 24, 4, 50, 2, 8, 40
    cols = (h + 2 * kv) * HD
    assert n * s * cols > 2 ** 31
    t.manual_seed(3)
    qkv = t.randn(n * s, cols, device="cuda", dtype=t.bfloat16)
    do = t.randn(n * s, h * HD, device="cuda", dtype=t.bfloat16)
    table = t.randn(nb, h, device="cuda")

    def run(m, x, g):
        o, lse = t.empty(m * s, h * HD, device="cuda", dtype=t.bfloat16), t.empty(m * s, h, device="cuda")
        dx, dt = t.empty_like(x), t.zeros_like(table)
        scratch = t.empty(lib.gpipe_op_attention_window_scratch_bytes(m, s, h, window, sinks, nb), device="cuda",
                          dtype=t.uint8)
        form = (m, s, h, kv, window, sinks, None, table.data_ptr(), nb, md, x.data_ptr(), o.data_ptr())
        assert lib.gpipe_op_attention_window_fwd(*form, lse.data_ptr(), cur_stream()) == 0
        assert lib.gpipe_op_attention_window_bwd(*form, g.data_ptr(), lse.data_ptr(), dx.data_ptr(), dt.data_ptr(),
                                                 scratch.data_ptr(), cur_stream()) == 0
        sync()
        return o, lse, dx

    ends = [slice(0, s), slice((n - 1) * s, n * s)]
    whole = [t.cat([x[e] for e in ends]) for x in run(n, qkv, do)]
    two = run(2, t.cat([qkv[e] for e in ends]), t.cat([do[e] for e in ends]))
    for x, y in zip(whole, two):
        assert t.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [{}, dict(in_place=True), dict(ce=0.0), dict(lddz=600008)])
def test_rows_that_no_cluster_holds(b, dtype, kw):  # noqa: F811
    Distill(b, 3, 600000, 30, dtype, seq=3, **kw).run().check()
    Distill(b, 2, 600001, 30, dtype, seq=3, **{k: v for k, v in kw.items() if k != "lddz"}).run().check()


@pytest.mark.parametrize("rows,vocab,ld", [
    ((1 << 22) + 5000, 500, 512),       # rows in registers
    (66000, 32000, 32768),              # through the ring
    (430000, 5001, 5001),               # read twice
])
def test_logits_beyond_2_31_elements(b, rows, vocab, ld):  # noqa: F811
    """Rows at both ends and in the middle against fp64."""
    import torch as t
    assert rows * ld > 2 ** 31
    topk, seq, temp, kd, ce = 2, 7, 2.0, 0.5, 0.25
    t.manual_seed(4)
    z = t.randn(rows, ld, device="cuda", dtype=t.bfloat16)
    idx = t.randint(0, vocab, (rows, topk), device="cuda", dtype=t.int32)
    tl = t.randn(rows, topk, device="cuda")
    tokens = t.randint(0, vocab, (rows + 1,), device="cuda", dtype=t.int32)
    loss, dz = t.empty(rows, device="cuda"), t.empty(rows, ld, device="cuda", dtype=t.bfloat16)
    rc = b.lib().gpipe_op_distill(1, rows, vocab, z.data_ptr(), ld, topk, idx.data_ptr(), tl.data_ptr(), temp, kd, seq,
                                  tokens.data_ptr(), 0, ce, loss.data_ptr(), dz.data_ptr(), ld, cur_stream())
    assert rc == 0
    sync()
    for r0 in (0, rows // 2, rows - 5):
        e = slice(r0, r0 + 5)
        want, dwant, size, mag = distill_ref(np64(z[e, :vocab]), idx[e].cpu().numpy(), tl[e].cpu().numpy(), temp, kd, ce,
                                             seq, tokens.cpu().numpy(), r0)
        eps = 2.0 ** -24 * (32 + vocab / 512 + topk / 32)   # as in the other tests
        assert np.all(np.abs(np64(loss[e]) - want) <= eps * size)
        assert np.all(np.abs(np64(dz[e, :vocab]) - dwant) <= U * np.abs(dwant) + (1 + U) * eps * mag + 2.0 ** -134)


def test_loss_right_behind_the_tokens(b):  # noqa: F811
    """Whole sequences read no token behind their last, so what lies there may be an output."""
    rows, vocab, topk = 8, 100, 4
    d = Distill(b, rows, vocab, topk, seq=4).run()
    sync()
    both = dev(np.zeros(2 * rows, dtype=np.int32))
    both[:rows] = d.d[2][:rows]
    dz = dev(np.zeros((rows, vocab), dtype=np.float32), "bf16")
    rc = b.lib().gpipe_op_distill(0, rows, vocab, d.z.data_ptr(), d.ld, topk, d.d[0].data_ptr(), d.d[1].data_ptr(), 2.0,
                                  0.7, 4, both.data_ptr(), 0, 0.3, both.data_ptr() + 4 * rows, dz.data_ptr(), vocab,
                                  cur_stream())
    assert rc == 0, b.lib().gpipe_last_error(None)
    KEEP.append((both, dz))
    sync()
    import torch
    assert torch.equal(both[rows:].view(torch.float32), d.loss[:rows]) and torch.equal(dz, d.dz[:rows])
