"""Rows that count for nothing have a zero row of dh whatever the table holds, not 0 times it."""
import pytest

from tests.test_gpu_head_loss import call, make

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


# dh straight out of the products, summed over parts of the vocabulary, over pieces of it, and both
@gpu
@pytest.mark.parametrize("grads", ["h", "both"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows,d,vocab,piece", [(40, 64, 300, 0), (300, 800, 300, 0), (40, 64, 9000, 0),
                                                (300, 136, 9000, 0), (300, 136, 900, 256), (700, 72, 20000, 4096)])
def test_a_zero_row_of_dh(b, rows, d, vocab, piece, bad, grads):
    import torch
    p = make(rows, d, vocab, 8, seed=rows + d)
    p["weight"] = torch.ones(rows, device="cuda")
    p["weight"][5] = 0.0
    p["tokens"][11] = -1  # row 10
    dead = torch.zeros(rows, dtype=torch.bool, device="cuda")
    dead[[5, 10]] = True
    dead[7::8] = True
    p["emb"][vocab // 2, 3] = bad
    p["emb"][1] = bad
    p["h"][dead] = float("nan")
    o = call(b, p, piece, grads=grads)
    assert float(o["loss"][dead].abs().max()) == 0
    assert float(o["dh"][dead].float().abs().max()) == 0
    # (the others do show it)
    assert bool((~o["dh"][~dead].float().isfinite()).any(1).all())
