"""The head's gradients against differences along themselves: (loss(x + s) - loss(x - s)) / 2 for steps s of the
gradient's own signs, so that the difference is the sum of |gradient| |step| and a gradient of another size or order
shows.

x and s are whole multiples of a power of two, such that x + s and x - s are bf16 exactly.  What is left, and the
tolerance, all from 64 bits: half of both losses' bounds; the gradient's bounds along |s|; and the third derivative: a
row's is the third cumulant of its logits' moves D_v under p, at most R^3 / (6 sqrt 3) for moves within a range R, so
the difference is off by R^3 / (36 sqrt 3)."""
import math

import pytest

from tests.test_gpu_head_loss import U, call, exact, make

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


@gpu
@pytest.mark.parametrize("rows,d,vocab,piece", [(64, 64, 400, 0), (200, 64, 700, 256), (130, 800, 600, 0)])
@pytest.mark.parametrize("name", ["h", "emb"])
def test_gradients_along_themselves(b, name, rows, d, vocab, piece):
    import torch
    p = make(rows, d, vocab, rows + 1, weights=True, seed=rows, know=3.0)
    # s, and x in twice that: x and s together below 256 of them; in E small enough for the third derivative
    grid = 2.0 ** -6 if name == "h" else (2.0 ** -9 if d <= 64 else 2.0 ** -11)
    p[name] = ((p[name].float() / (2 * grid)).round() * (2 * grid)).clamp(-120 * grid, 120 * grid).bfloat16()
    base = p[name].clone()
    x0 = exact(p, inv=1.0)
    ref = {"h": x0["dh"], "emb": x0["demb"]}[name]
    tol_of = {"h": x0["dh_tol"], "emb": x0["demb_tol"] + 8 * U * x0["demb"].abs()}[name]
    step = grid * ref.sign()
    up, down = (base.double() + step).bfloat16(), (base.double() - step).bfloat16()
    assert torch.equal((up.double() - down.double()) / 2, step)
    assert torch.equal((up.double() + down.double()) / 2, base.double())
    o = call(b, p, piece, f32=True, inv=1.0)
    grad = {"h": o["dh"], "emb": o["demb"]}[name].double()
    ends, tol = [], float((tol_of * step.abs()).sum())
    for end in (up, down):
        p[name] = end
        ends.append(call(b, p, grads="none", inv=1.0)["loss"].double().sum())
        tol += float(exact(p, inv=1.0)["loss_tol"].sum()) / 2
    p[name] = base
    moves = step @ p["emb"].double().T if name == "h" else p["h"].double() @ step.T
    span = moves.amax(1) - moves.amin(1)
    w = torch.ones(rows, device="cuda", dtype=torch.float64) if p["weight"] is None else p["weight"].double()
    tol += float((w * span ** 3).sum()) / (36 * math.sqrt(3.0))
    difference = float(ends[0] - ends[1]) / 2
    want = float((ref * step).sum())
    assert want > 0 and tol <= 0.05 * want, (tol, want)  # the test is sharp

    def off(g):
        return abs(float((g * step).sum()) - difference)
    assert off(grad) <= tol, (off(grad), tol, want)
    # and gradients that are wrong would not pass
    for wrong in (-grad, 0.5 * grad, 1.5 * grad, grad.roll(1, 0), grad.roll(1, 1)):
        assert off(wrong) > 3 * tol
