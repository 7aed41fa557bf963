"""The distillation loss at the ends of what its arguments allow, against fp64."""
import numpy as np
import pytest

from tests.test_gpu_window_distill import Distill, b  # noqa: F401

pytestmark = pytest.mark.gpu

# a row in registers, through the ring, across a cluster, and read twice
LENGTHS = [600, 9000, 100001, 270001]


@pytest.mark.parametrize("temp", [0.5, 0.7, 3.0])
@pytest.mark.parametrize("offset", [3e4, -1e6])
@pytest.mark.parametrize("vocab", LENGTHS)
def test_teacher_logits_with_a_common_offset(b, vocab, offset, temp):  # noqa: F811
    """p depends on the teacher's logits through their distances to the largest one
    alone, so the bounds are those for the logits without the offset."""
    d = Distill(b, 3, vocab, 40, temp=temp, seq=3)
    d.tl += np.float32(offset)
    d.run()
    d.tl = d.tl.astype(np.float64) - d.tl.max(1, keepdims=True).astype(np.float64)
    d.check()


@pytest.mark.parametrize("vocab", LENGTHS)
def test_teacher_logits_far_apart(b, vocab):  # noqa: F811
    """Logits whose quotient by the temperature is no fp32 number: p is 1 and 0."""
    d = Distill(b, 3, vocab, 8, temp=1e-3, kd=1.0, seq=3)
    d.tl[:, 1:] = -1e37
    d.tl[:, 0] = 1e37
    d.run()
    d.tl = np.where(np.arange(8) == 0, 0.0, -np.inf) * np.ones((3, 1))
    d.check()
