"""Dropout on the GPU: the mask bit for bit against the generator's definition, the values in 64 bits
(a product and an addition in binary32, one rounding)."""
import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc
from layer_helpers import (BF16, E, F16, F32, bits, buffer, dropout_kept, generator, near, normal,
                           outside_is_untouched)

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 3), (5, 4), (9, 5), (33, 1024), (64, 63), (31, 1001), (700, 20), (3, 40001),
         (1025, 17)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def check(m, d, type_, p=0.3, seed=11, step=None, residual=True, pad=0, alias=None):
    gen = generator(m + d)
    x = normal(gen, m, d, type_, pad=pad)
    r = normal(gen, m, d, type_, pad=pad) if residual else None
    X, R = x.double(), r.double() if residual else torch.zeros(m, d, device="cuda").double()
    out = {"x": x, "r": r, None: None}[alias]
    out = buffer(m, d, type_, pad) if out is None else out
    word = None if step is None else torch.tensor([step], dtype=torch.int64, device="cuda")
    dgc.dgc_dropout(x, r, p, seed, word, out)
    kept = dropout_kept(m, d, p, seed, 0 if step is None else step).cuda()
    share = (65536 - int(p * 65536 + 0.5)) / 65536
    value = X / share if share else torch.zeros_like(X)
    want = torch.where(kept, value, torch.zeros_like(X)) + R
    near(out, want, 2 * E * value.abs() + E * want.abs())
    assert torch.equal(out[~kept].double(), R[~kept])  # dropped: the residual's own bits, or zero
    if not residual:
        assert ((out != 0) | (X == 0) | ~kept).all()   # kept: no other zeros
    outside_is_untouched(out)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("m,d", SIZES)
def test_values_and_mask(m, d, type_, residual):
    check(m, d, type_, residual=residual)


@pytest.mark.parametrize("pad", [1, "odd", "packed"])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
def test_strides(type_, pad):
    for m, d in ((1, 1), (17, 9), (40, 250), (31, 1001)):
        check(m, d, type_, pad=pad)
        check(m, d, type_, pad=pad, residual=False, alias="x")
        check(m, d, type_, pad=pad, alias="r")
        check(m, d, type_, pad=pad, alias="x")


@pytest.mark.parametrize("p", [0.0, 1e-6, 2 ** -17, 2 ** -16, 0.1, 0.5, 0.9999, 1 - 2 ** -17, 1.0])
def test_shares(p):
    check(40, 300, BF16, p=p)
    check(40, 300, F32, p=p, residual=False)


@pytest.mark.parametrize("seed,step", [(0, 0), (2**64 - 1, 1), (5, -1), (-3, 2**62), (1 << 40, 7)])
def test_seeds_and_steps(seed, step):
    """The words are taken modulo 2^64."""
    gen = generator(1)
    x, out = normal(gen, 30, 100, F32), buffer(30, 100, F32)
    dgc.dgc_dropout(x, None, 0.5, seed, torch.tensor([step], device="cuda"), out)
    kept = dropout_kept(30, 100, 0.5, seed % 2**64, step % 2**64).cuda()
    assert torch.equal(out != 0, kept)


def test_what_is_dropped_does_not_matter():
    x = torch.full((20, 64), float("nan"), dtype=F16, device="cuda")
    x[::2] = float("inf")
    r, out = normal(generator(2), 20, 64, F16), buffer(20, 64, F16)
    dgc.dgc_dropout(x, r, 0.5, 3, None, out)
    kept = dropout_kept(20, 64, 0.5, 3, 0).cuda()
    assert torch.equal(out[~kept], r[~kept]) and not torch.isfinite(out[kept]).any()
    dgc.dgc_dropout(x, None, 1.0, 3, None, out)
    assert (out == 0).all()


def test_backward_is_the_same_call():
    """The gradient of sum(w out) with the mask that the forward pass drew, and by differences."""
    gen = generator(4)
    x, w, v = (torch.randn(50, 130, generator=gen, device="cuda") for _ in range(3))
    out, dx, up, down = (torch.empty_like(x) for _ in range(4))
    step = torch.tensor([9], device="cuda")
    dgc.dgc_dropout(x, None, 0.25, 77, step, out)
    dgc.dgc_dropout(w, None, 0.25, 77, step, dx)
    assert torch.equal(dx != 0, out != 0)
    dgc.dgc_dropout(x + v, None, 0.25, 77, step, up)   # linear: a difference of any size is exact
    dgc.dgc_dropout(x - v, None, 0.25, 77, step, down)
    slope = (w.double() * (up.double() - down.double())).sum().item() / 2
    terms = (w.double() * (up.double().abs() + down.double().abs())).abs().sum().item()
    assert abs((dx.double() * v.double()).sum().item() - slope) <= 4 * E * terms


def test_share_over_many_entries():
    """2^24 draws at p = 0.1: the share of zeros is within five deviations (6e-4) of its
    expectation 6554 / 65536, and neighbours in a row and a column are independent."""
    x = torch.ones(4096, 4096, dtype=BF16, device="cuda")
    out = torch.empty_like(x)
    dgc.dgc_dropout(x, None, 0.1, 12345, None, out)
    z = (out == 0).double()
    q = 6554 / 65536
    bound = 5 * (q * (1 - q) / 2**24) ** 0.5
    assert abs(z.mean().item() - q) < bound
    for a, b in ((z[:, 1:], z[:, :-1]), (z[1:], z[:-1])):
        assert abs(((a - q) * (b - q)).mean().item()) < 5 * q * (1 - q) / 2**12


def test_a_captured_call_draws_anew():
    x, out = torch.ones(64, 512, dtype=BF16, device="cuda"), buffer(64, 512, BF16)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    dgc.dgc_dropout(x, None, 0.5, 6, step, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgc.dgc_dropout(x, None, 0.5, 6, step, out)
        step += 1
    for i in range(3):
        graph.replay()
        assert torch.equal(out != 0, dropout_kept(64, 512, 0.5, 6, i).cuda())


def test_masks_do_not_depend_on_the_type():
    m, d = 300, 333
    zeros = []
    for type_, pad in ((F32, 0), (BF16, "odd"), (F16, "packed")):
        out = buffer(m, d, type_, pad)
        x = buffer(m, d, type_, pad, fill=1.0)
        dgc.dgc_dropout(x, None, 0.4, 8, None, out)
        zeros.append(out == 0)
    assert torch.equal(zeros[0], zeros[1]) and torch.equal(zeros[0], zeros[2])
    assert bits(out).shape == (m, d)


def test_rows_past_two_to_the_32():
    m, d = 70000, 65536
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.ones(m, d, dtype=torch.float16, device="cuda")
    dgc.dgc_dropout(x, None, 0.5, 21, None, x)
    last = x[-2:]
    words = d // 4
    # the last two rows' words, by their numbers
    import numpy as np
    g = np.array([0x9E3779B97F4A7C15], np.uint64)

    def mix(z):
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))

    key = mix(g + np.uint64(21))
    n = np.arange((m - 2) * words + 1, m * words + 1, dtype=np.uint64)
    draw = mix(n * g + key).astype("<u8").view("<u2").reshape(2, d)
    assert np.array_equal((last != 0).cpu().numpy(), draw >= 32768)
