"""What a clipping call leaves in L2 for the work behind it, on the GPU."""
import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

pytestmark = pytest.mark.gpu


def median_us(before, work, n=31):
    times = []
    for _ in range(n):
        before()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        work()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[n // 2]


@pytest.mark.parametrize("form,limit", [("in place, nothing to clip", 1.15), ("into a bucket", 1.25)])
def test_the_next_operator_has_l2_to_itself(form, limit):
    """Six passes over 90 MB, which L2 holds, directly behind a clipping call, against the same behind
    the norm alone. Lines of the gradients that L2 kept by priority would make it 1.33 and 1.45
    times as long; a bucket's entries still to be written to memory alone, 1.12. The best of three
    comparisons, as the clock may change between two."""
    dgc.build()
    src = [torch.randn(205_000_000 // 8, device="cuda").bfloat16() * 1e-4 for _ in range(8)]
    bucket = torch.empty(8 * src[0].numel(), device="cuda")
    a = dgc.TensorList(src)
    to = None if form.startswith("in place") else dgc.TensorList(list(bucket.split(src[0].numel())))
    ws = torch.empty(dgc.dgc_grad_workspace(a), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, device="cuda")
    x = torch.randn(90 << 18, device="cuda")

    def passes():
        for _ in range(6):
            x.sum()

    def norm():
        dgc.dgc_grad_norm(a, 1e9, out[:1], out[1:], ws)

    def clip():
        dgc.dgc_grad_clip(a, to, 1e9, out[:1], out[1:], ws)

    ratios = []
    for _ in range(3):
        ratios.append(median_us(clip, passes) / median_us(norm, passes))
        if ratios[-1] <= limit:
            return
    pytest.fail(f"{form}: {ratios}")
