"""dgc_grad_norm and dgc_grad_clip on the GPU against sums in 64 bits.

Tolerances. The norm: squares of at most 64 entries in binary32 chains of 16 (relative error of
a sum of positive terms <= 16 * 2^-24 < 1e-6, halved by the root), then one rounding to binary32:
1e-6. The scale: the norm's error once more and a rounding, 2e-6. A clipped entry: one binary32
product with the scale that the call reports, so given that scale it is exact: bitwise."""
import math
import random

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def call(src, max_norm, dst="norm", stream=None):
    """(norm, scale) as Python floats; dst: "norm" (no clipping), None (in place) or a list."""
    a = dgc.TensorList(src)
    out = torch.full((2,), 7.0, device="cuda")
    ws = torch.full((dgc.dgc_grad_workspace(a),), 0xA5, dtype=torch.uint8, device="cuda")
    if isinstance(dst, str):
        dgc.dgc_grad_norm(a, max_norm, out[:1], out[1:], ws, stream=stream)
    else:
        b = None if dst is None else dgc.TensorList(dst)
        dgc.dgc_grad_clip(a, b, max_norm, out[:1], out[1:], ws, stream=stream)
    return out[0].item(), out[1].item()


def norm64(src):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in src))


def expected_scale(norm, c):
    return c / norm if norm > c > 0 and math.isfinite(c) else 1.0


def make(sizes, dtype, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dts = dtype if isinstance(dtype, (list, tuple)) else [dtype] * len(sizes)
    return [(torch.randn(n, generator=g, device="cuda") * sigma).to(dt)
            for n, dt in zip(sizes, dts)]


def check_norm(src, c, got):
    want = norm64(src)
    assert got[0] == pytest.approx(want, rel=1e-6, abs=0.0)
    assert got[1] == pytest.approx(expected_scale(want, c), rel=2e-6, abs=0.0)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("sizes", [[], [0], [1], [7, 0, 1, 33], [2047], [2048], [2049],
                                   [2048 * 24 + 5] * 3, [1 << 20], [3] * 23, [5] * 191,
                                   [1000, 1] * 480, [17] * 961, [2100] * 2500])
def test_norm_and_clip(sizes, dtype):
    src = make(sizes, dtype, 3 + len(sizes))
    check_norm(src, 0.5, call(src, 0.5))
    for to in (F32, dtype):
        dst = [torch.full_like(t, 9.0, dtype=to) for t in src]
        got = call(src, 0.5, dst)
        check_norm(src, 0.5, got)
        s = torch.tensor(got[1], device="cuda")
        for a, b in zip(src, dst):
            assert torch.equal(b, (a.float() * s).to(to))


@pytest.mark.parametrize("c", [0.0, -1.0, math.inf, 1e30])
def test_no_clipping(c):
    src = make([5000, 3], F32, 1)
    keep = [t.clone() for t in src]
    got = call(src, c, None)
    check_norm(src, c, got)
    assert got[1] == 1.0
    assert all(torch.equal(a, b) for a, b in zip(src, keep))


def test_in_place_and_mixed_types():
    src = make([4097, 100001, 64, 2048], [F32, BF16, F16, F32], 5, 0.3)
    keep = [t.clone() for t in src]
    got = call(src, 1.0, None)
    check_norm(keep, 1.0, got)
    s = torch.tensor(got[1], device="cuda")
    for a, k in zip(src, keep):
        assert torch.equal(a, (k.float() * s).to(k.dtype))
    again = call(src, 1.0)
    assert again[0] == pytest.approx(1.0, rel=0.01)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_flat_bucket_with_odd_pieces(dtype, shift):
    """Pieces of a flat bucket and sources that start off every 16-byte boundary."""
    sizes = [1, 4099, 2048, 7, 30001]
    big = make([sum(sizes) + shift], dtype, 11)[0]
    src = list(big[shift:].split(sizes))
    bucket = torch.full((sum(sizes) + 2 * shift,), 3.0, device="cuda")
    got = call(src, 0.25, list(bucket[shift:-shift].split(sizes)))
    check_norm(src, 0.25, got)
    s = torch.tensor(got[1], device="cuda")
    assert torch.equal(bucket[shift:-shift], big[shift:].float() * s)
    assert bucket[:shift].eq(3.0).all() and bucket[-shift:].eq(3.0).all()


@pytest.mark.parametrize("dtype,values", [
    (F32, [1e-45, 3e-42, 1e-40]), (F32, [1e-30, 1e-28]), (F32, [1e19, 3e19]),
    (F32, [3.4e38]), (F32, [1e-44, 1.0, 1e25]), (BF16, [1e-39, 1e-38]), (BF16, [1e30, 1e-20]),
    (F16, [6e-8, 65504.0]), (F32, [2.0 ** -45, 2.0 ** -44]), (F32, [2.0 ** 60, 2.0 ** 63])])
def test_magnitudes_at_the_ends_of_the_range(dtype, values):
    t = torch.tensor(values, device="cuda").to(dtype).repeat(700)[:2048 * len(values) // 3 + 5]
    if norm64([t]) < 3.4e38:
        assert call([t], 0.0)[0] == pytest.approx(norm64([t]), rel=1e-6, abs=1e-45)
    else:  # past binary32: the norm is +inf, the scale still comes from the 64-bit norm
        got = call([t], 1.0)
        assert got[0] == math.inf
        assert got[1] == pytest.approx(1.0 / norm64([t]), rel=2e-6, abs=1e-45)


def test_all_zero():
    assert call([torch.zeros(100000, device="cuda")], 1.0) == (0.0, 1.0)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n", [3, 2048, 70001])
def test_not_finite(dtype, n):
    src = make([n, 50], dtype, 9)
    src[0][n - 1] = -math.inf
    assert call(src, 1.0) == (math.inf, 0.0)
    keep = src[1].clone()
    call(src, 1.0, None)
    assert torch.equal(src[1], keep * 0)
    assert torch.isnan(src[0][n - 1])
    src = make([n, 50], dtype, 9)
    src[0][0] = math.inf
    src[1][7] = math.nan
    norm, scale = call(src, 1.0)
    assert math.isnan(norm) and scale == 1.0


def test_runs_agree_bitwise_and_streams_are_respected():
    src = make([3_000_001, 17, 1_000_000], BF16, 21)
    first = call(src, 1.0)
    side = torch.cuda.Stream()
    a, out = dgc.TensorList(src), torch.zeros(2, device="cuda")
    ws = torch.empty(dgc.dgc_grad_workspace(a), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            dgc.dgc_grad_norm(a, 1.0, out[:1], out[1:], ws)
    side.synchronize()
    assert (out[0].item(), out[1].item()) == first


def test_graph_replays_on_fresh_gradients():
    src = make([300_000, 77], F32, 2)
    dst = [torch.empty_like(t) for t in src]
    a, b = dgc.TensorList(src), dgc.TensorList(dst)
    out = torch.zeros(2, device="cuda")
    ws = torch.empty(dgc.dgc_grad_workspace(a), dtype=torch.uint8, device="cuda")
    dgc.dgc_grad_clip(a, b, 1.0, out[:1], out[1:], ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgc.dgc_grad_clip(a, b, 1.0, out[:1], out[1:], ws)
    for seed in (5, 6):
        for t, v in zip(src, make([300_000, 77], F32, seed, 0.01 * seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        check_norm(src, 1.0, (out[0].item(), out[1].item()))
        for x, y in zip(src, dst):
            assert torch.equal(y, x * out[1])


@pytest.mark.parametrize("seed", range(6))
def test_random_lists(seed):
    r = random.Random(seed)
    count = r.randrange(1, 300)
    sizes = [int(2 ** r.uniform(0, 17)) for _ in range(count)]
    dts = [r.choice((F32, F16, BF16)) for _ in range(count)]
    src = make(sizes, dts, seed, 10.0 ** r.uniform(-3, 1))
    dst = [torch.empty(n, dtype=r.choice((F32, F16, BF16)), device="cuda") for n in sizes]
    got = call(src, 1.0, dst)
    check_norm(src, 1.0, got)
    s = torch.tensor(got[1], device="cuda")
    for a, b in zip(src, dst):
        assert torch.equal(b, (a.float() * s).to(b.dtype))


@pytest.mark.slow
def test_entries_past_32_bits():
    """A list whose entries pass 2^32, in one tensor of 16-bit entries."""
    n = (1 << 32) + 4099
    t = torch.zeros(n, dtype=BF16, device="cuda")
    t[-1] = 3.0
    t[1 << 31] = 4.0
    got = call([t], 1.0, None)
    assert got[0] == 5.0
    assert t[-1].item() == torch.tensor(3.0 * got[1]).bfloat16().item()
