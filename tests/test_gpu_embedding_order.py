"""The embedding's gradient bit for bit: the order of additions that the header promises, in fp32.

Up to 256 rows a token's n rows are cut into quarters of ceil(n / 4).  More rows are sorted by token, stably, and cut
into runs of 8 (up to 24576 rows) or 64; a token's rows in a run are added in order, then its runs; those of more than
16 runs in eighths first.  The sum is scaled, rounded, and added to the accumulator."""
import pytest

from tests.test_gpu_embedding_sorted import error, gradient

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


def in_order(terms):
    import numpy as np
    acc = np.zeros_like(terms[0])
    for x in terms:
        acc = acc + x
    return acc


def in_groups(terms, k):
    per = -(-len(terms) // k)
    return in_order([in_order(terms[i:i + per]) for i in range(0, len(terms), per)])


def emulate(tokens, dx, before, scale):
    """The accumulator afterwards, and how many runs each token has (0 where there are none)."""
    import numpy as np
    rows, vocab = len(tokens), len(before)
    keys = np.where((tokens >= 0) & (tokens < vocab), tokens, vocab)
    order = np.argsort(keys, kind="stable")
    run = 8 if rows <= 24576 else 64
    out, spans = before.copy(), set()
    starts = np.searchsorted(keys[order], np.arange(vocab + 1))
    for v in range(vocab):
        a, z = int(starts[v]), int(starts[v + 1])
        if a == z:
            continue
        if rows <= 256:
            total = in_groups([dx[r] for r in order[a:z]], 4)
        else:
            cuts = [a] + [p for p in range(a - a % run + run, z, run)] + [z]
            parts = [in_order([dx[r] for r in order[i:j]]) for i, j in zip(cuts, cuts[1:])]
            spans.add(len(parts))
            total = parts[0] if len(parts) == 1 else in_order(parts) if len(parts) <= 16 else in_groups(parts, 8)
        out[v] = before[v] + np.float32(scale) * total
    return out, spans


def test_the_emulation_itself():
    """Groups of 2: (1 + 2^-24) + (2^-24 + 2^-24) is above 1, left to right it is 1."""
    import numpy as np
    one = [np.float32([x]) for x in (1.0, 2.0 ** -24, 2.0 ** -24, 2.0 ** -24)]
    assert in_order(one)[0] == 1 and in_groups(one, 2)[0] > 1 and in_groups(one[:3], 4)[0] == 1
    dx = np.float32([[x] for x in (1.0, 2.0 ** -24, 2.0 ** -24, 2.0 ** -24, 5.0)])
    out, _ = emulate(np.array([0, 0, 0, 0, -1]), dx, np.zeros((2, 1), np.float32), 1.0)
    assert out[0, 0] == 1 and out[1, 0] == 0


COUNTS = {
    "few": [1, 2, 3, 4, 5, 6, 7, 8, 9, 17, 40, 100],
    # (in runs of 8: two runs, 16 from a boundary on, 16 and 17 across one, hundreds)
    "rank": [16 * 8, 3, 16 * 8, 5, 16 * 8 - 8, 1, 2, 7, 6, 1200, 9, 16 * 8 + 1],
    "radix": [16 * 8, 3, 16 * 8, 5, 16 * 8 - 8, 1, 2, 7, 6, 4000, 9, 1601, 16 * 8 + 1],
    "long": [16 * 64, 3, 16 * 64, 5, 16 * 64 - 64, 1, 2, 70, 6, 20000, 9, 130, 5000, 16 * 64 + 1],
}


@gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dead", [0, 50])
@pytest.mark.parametrize("kind", COUNTS)
@pytest.mark.parametrize("d", [8, 136])
def test_bit_for_bit(b, kind, f32, dead, d):
    import numpy as np
    import torch
    counts = COUNTS[kind]
    rng = np.random.default_rng(len(counts) + dead)
    vocab = len(counts) + 3  # (tokens that never come at the end)
    tokens = np.concatenate([np.full(n, v) for v, n in enumerate(counts)] + [np.full(dead, -1)]).astype(np.int32)
    rng.shuffle(tokens)
    dx = torch.from_numpy(rng.standard_normal((len(tokens), d), dtype=np.float32))
    dx = dx if f32 else dx.bfloat16()
    before = rng.standard_normal((vocab, d), dtype=np.float32)
    want, spans = emulate(tokens, dx.float().numpy(), before, 0.7)
    if kind != "few":
        assert {1, 2, 16, 17} <= spans and max(spans) > 100
    demb = torch.from_numpy(before).cuda()
    gradient(b, torch.from_numpy(tokens).cuda(), dx.cuda(), d, demb, 0.7)
    got = demb.cpu().numpy()
    off = [v for v in range(vocab) if not np.array_equal(got[v], want[v])]
    assert not off, [(v, counts[v] if v < len(counts) else 0) for v in off]
    assert error(b) == 0


@gpu
@pytest.mark.parametrize("kind", COUNTS)
def test_subnormal_elements_count_as_zero_on_every_path(b, kind):
    """An accumulator's subnormal element that receives an addition, and a subnormal addition; others keep theirs."""
    import numpy as np
    import torch
    counts = COUNTS[kind]
    vocab = len(counts) + 1
    tokens = torch.from_numpy(np.concatenate([np.full(n, v) for v, n in enumerate(counts)]).astype(np.int32)).cuda()
    tiny = 2.0 ** -140
    for dx_value, before in ((0.0, tiny), (tiny, 0.0)):
        dx = torch.zeros(tokens.numel(), 8, device="cuda")
        first = np.cumsum([0] + counts[:-1])
        dx[torch.from_numpy(first).cuda()] = dx_value
        demb = torch.full((vocab, 8), before, device="cuda")
        gradient(b, tokens, dx, 8, demb, 1.0)
        got = demb.cpu().numpy()
        assert [v for v in range(vocab - 1) if np.any(got[v] != 0)] == []
        assert np.array_equal(got[-1], np.full(8, before, np.float32))
