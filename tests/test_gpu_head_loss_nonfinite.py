"""The head's loss where a logit, a hidden state or an entry of the table is not finite.

Without clip the definition is that of softmax on the extended numbers: a NaN or a logit of +inf makes its row's loss
NaN (inf - inf), the target's logit of -inf makes it +inf, and -inf elsewhere is a power of 0.  With clip an infinite
logit counts as the limit.  Finite losses are near to 64 bits with the bounds of test_gpu_head_loss.py, taken over the
finite terms; finite columns of dh and rows of demb likewise."""
import pytest

from tests.test_gpu_head_loss import U, call, make

gpu = pytest.mark.gpu
BAD = 7   # row of the table with the infinity
AT = 3    # its column


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


def definition(p, clip):
    """Loss, gradient of the logits and the tolerances of both, in 64 bits; sequences are one row longer than the batch,
    so every row has a target."""
    import torch
    h, e, t = p["h"].double(), p["emb"].double(), p["tokens"][1:].long()
    z = h @ e.T
    plain = torch.where(z.isfinite(), z, torch.zeros_like(z))
    inside = torch.ones_like(z)
    if clip > 0:
        inside = (z.abs() < clip).double()
        z = z.clamp(-clip, clip)
        plain = plain.clamp(-clip, clip)
    logp = torch.log_softmax(z, 1)
    n = torch.arange(p["rows"], device="cuda")
    g = logp.exp()
    g[n, t] -= 1
    hf, ef = (torch.where(x.isfinite(), x, torch.zeros_like(x)).abs() for x in (h, e))
    dz = 2 * p["d"] * U * (hf @ ef.T).amax(1)
    e_s = 2.0 ** -20 + 2 * U * (p["vocab"] / 128 + 140)
    tol = 2 * dz + 8 * U * (plain.abs().amax(1) + plain[n, t].abs() + 1) + e_s
    off = (2 * (2 * dz + e_s) + 2.0 ** -11)[:, None] * logp.exp() + 2.0 ** -38
    slack = inside * (g.abs() * (2.0 ** -8 + 2.0 ** -10) + off)
    return -logp[n, t], g * inside, tol, slack


@gpu
@pytest.mark.parametrize("clip", [0.0, 50.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("grads", ["none", "both"])
@pytest.mark.parametrize("rows,d", [(20, 64), (300, 64), (300, 800)])
def test_an_infinity_in_the_table(b, rows, d, grads, sign, clip):
    """A fifth of the rows have the token with the infinity as their target; its logit is +inf for some of them and -inf
    for others."""
    import torch
    p = make(rows, d, 1000, rows + 1, seed=rows)
    p["tokens"][1::5] = BAD
    p["emb"][BAD, AT] = sign * float("inf")
    p["h"][:, AT] = torch.where(p["h"][:, AT] == 0, torch.ones_like(p["h"][:, AT]), p["h"][:, AT])
    p["h"][0::10, AT], p["h"][5::10, AT] = 1.0, -1.0
    o = call(b, p, clip=clip, grads=grads, inv=1.0)
    want, g, tol, slack = definition(p, clip)
    hit = p["tokens"][1:].long() == BAD
    assert bool(hit.any()) and bool((~hit).any())
    nan, inf = want.isnan(), want.isinf()
    if clip > 0:
        assert bool(want.isfinite().all())
    else:
        assert bool((nan & hit).any()) and bool((nan & ~hit).any()) and bool((inf & hit).any())
    loss = o["loss"].double()
    assert torch.equal(loss.isnan(), nan)
    assert bool((loss[inf] == float("inf")).all())
    fine = want.isfinite()
    assert float(((loss - want).abs() - tol)[fine].max()) <= 0
    if grads == "none":
        return
    assert bool(o["dh"][nan].isnan().all())
    some = ~nan
    ef = torch.where(p["emb"].isfinite(), p["emb"], torch.zeros_like(p["emb"])).double()
    g, slack = g[some], slack[some]
    cols = [c for c in range(d) if c != AT]
    dh = (g @ ef)[:, cols]
    near = (o["dh"][some][:, cols].double() - dh).abs() - 1.01 * (slack @ ef.abs())[:, cols] - 2.0 ** -8 * dh.abs()
    assert float(near.max()) <= 0
    if clip > 0:  # every logit of the infinity is beyond the limit: no gradient, and h is finite
        demb = g.T @ p["h"].double()
        over = (o["demb"].double() - demb).abs() - 1.01 * (slack.T @ p["h"].double().abs()) - 2.0 ** -8 * demb.abs()
        assert float(over.max()) <= 0
    else:
        assert bool(o["demb"].isnan().all())


@gpu
@pytest.mark.parametrize("clip", [0.0, 50.0])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows,d", [(20, 64), (300, 64), (300, 800)])
def test_a_row_of_h_that_is_not_finite(b, rows, d, bad, clip):
    """Its loss and dh, and demb, which it is a term of; no other row's loss or dh.  With clip its logits count
    as the limit: a finite loss, no gradient, and 0 times the infinity in its column of demb alone."""
    import torch
    p = make(rows, d, 1000, rows + 1, seed=rows)
    p["emb"][:, AT] = torch.where(p["emb"][:, AT] == 0, torch.ones_like(p["emb"][:, AT]), p["emb"][:, AT])
    good = call(b, p, clip=clip)
    p["h"][4, AT] = bad
    for grads in ("none", "both"):
        o = call(b, p, clip=clip, grads=grads)
        rest = [r for r in range(rows) if r != 4]
        if grads == "both":
            assert torch.equal(o["loss"][rest], good["loss"][rest]) and torch.equal(o["dh"][rest], good["dh"][rest])
        else:
            assert bool(o["loss"][rest].isfinite().all())
        if clip > 0 and bad == bad:
            want, _, tol, _ = definition(p, clip)
            assert abs(float(o["loss"][4]) * rows - float(want[4])) <= float(tol[4]) + 4 * U * float(want[4])
            if grads == "both":
                assert float(o["dh"][4].float().abs().max()) == 0
                assert bool(o["demb"][:, AT].isnan().all())
                cols = [c for c in range(d) if c != AT]
                assert bool(o["demb"][:, cols].isfinite().all())
        else:
            assert bool(o["loss"][4].isnan())
            if grads == "both":
                assert bool(o["dh"][4].isnan().all()) and bool(o["demb"].isnan().all())


@gpu
@pytest.mark.parametrize("grads", ["none", "both"])
def test_the_target_alone_overflows(b, grads):
    """Finite operands whose product is +inf in fp32 for the target only, and a vocabulary of one token whose logit is
    +inf: inf - inf, not a perfect row."""
    import torch
    for rows, vocab in ((1, 1), (3, 1), (5, 600), (100, 600)):
        emb = torch.zeros(vocab, 64, device="cuda")
        emb[:, 0] = torch.linspace(-1, 1, vocab, device="cuda")
        h = torch.zeros(rows, 64, device="cuda")
        h[:, 0] = 1.0
        emb[0, 5] = 2.0 ** 60
        h[-1, 5] = 2.0 ** 100
        tokens = torch.zeros(rows + 1, device="cuda", dtype=torch.int32)
        p = dict(rows=rows, d=64, vocab=vocab, seq=rows + 1, emb=emb.bfloat16(), tokens=tokens, h=h.bfloat16(),
                 weight=None)
        o = call(b, p, grads=grads)
        assert bool(o["loss"][-1].isnan()), (rows, vocab)
        assert bool(o["loss"][:-1].isfinite().all())
        if grads == "both":
            assert bool(o["dh"][-1].isnan().all()) and bool(o["demb"].isnan().any())
