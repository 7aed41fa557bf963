"""A head's loss that waits for its predecessor keeps no SM from another stream's kernels."""
import pytest

from tests.test_gpu_head_loss import call, make

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from micro_pipeline_re_gb300 import binding
    binding.lib()
    return binding


@gpu
@pytest.mark.parametrize("rows,grads", [(40, "none"), (2000, "none"), (600, "both")])
def test_a_waiting_call_leaves_the_gpu_to_other_streams(b, rows, grads):
    """Stream one: a kernel of one CTA that takes milliseconds and lets its successor launch at once, then the head's
    loss.  Stream two, enqueued after both: a product of whole SMs.  It ends long before the first kernel."""
    import torch
    lib, ptr = b.lib(), b._ptr
    p = make(rows, 256, 32000, 100)
    n = 1 << 23  # one warp's row
    y, t, dy, rows_loss = (torch.zeros(k, device="cuda") for k in (n, n, n, 1))
    m = 8192  # 0.7 ms on the whole GPU, tens on an SM or two
    x, w = (torch.zeros(m, m, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    c = torch.empty(m, m, device="cuda", dtype=torch.bfloat16)
    buf = call(b, p, grads=grads)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()

    def long_kernel():
        b._check(lib.gpipe_op_mse(1, n, ptr(y), ptr(t), 1.0, ptr(rows_loss), ptr(dy), b.current_stream()))

    def product():
        b._check(lib.gpipe_op_gemm(1, m, m, m, ptr(x), m, 1, ptr(w), m, 1, 0, ptr(c), m, None, None, 0, None, None, 0,
                                   b.current_stream()))
    long_kernel()
    product()
    torch.cuda.synchronize()  # everything is loaded
    start, last, other = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    with torch.cuda.stream(one):
        start.record()
        long_kernel()
        call(b, p, grads=grads, buf=buf)
        last.record()
    with torch.cuda.stream(two):
        product()
        other.record()
    torch.cuda.synchronize()
    # (far longer than the product, and than the host needs for these calls)
    assert start.elapsed_time(last) > 4.0
    assert start.elapsed_time(other) < 0.5 * start.elapsed_time(last), (start.elapsed_time(other), start.elapsed_time(last))
