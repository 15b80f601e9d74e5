"""Layer norm and its backward pass on the GPU against their definitions in 64 bits.

Bounds, in units of E = 2^-24. A row's sums are chains of at most 64 additions in a lane (rows of up
to 16384; 128 covers the longer ones of these tests) and 10 across lanes and warps: a sum is off by
L = 160 E of its terms' magnitudes. With the mean's rounding taken out, x - mean is off by E of
itself and L of the deviation, rstd by L of itself: xhat by L (2 |xhat| + 1)."""
import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc
from layer_helpers import (BF16, E, F16, F32, bits, buffer, generator, near, normal,
                           outside_is_untouched, workspace)

pytestmark = pytest.mark.gpu

EPS = 1e-5
L = 160 * E
SIZES = [(1, 1), (3, 2), (9, 7), (33, 64), (70, 255), (50, 256), (40, 257), (777, 1001),
         (19, 1024), (23, 2049), (17, 4096), (13, 4097), (11, 8192), (5, 8193), (7, 12288),
         (5, 16384), (4, 16385), (3, 30001)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def weights(d, gen, odd=False):
    """A piece of a larger array, off 16-byte boundaries if odd."""
    flat = torch.randn(d + 8, generator=gen, device="cuda") * 0.2 + 1.0
    return flat[1:1 + d] if odd else flat[:d]


def statistics(x):
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + torch.tensor(EPS, dtype=F32).double().item())
    return mean, var.sqrt(), rstd


def forward(m, d, type_, sigma=1.0, mean=0.3, pad=0, beta=True, save=True, odd=False, in_place=False):
    gen = generator(m + d)
    x = normal(gen, m, d, type_, sigma, mean, pad)
    gamma, b = weights(d, gen, odd), weights(d, gen, odd) - 1.0 if beta else None
    X = x.double()
    y = x if in_place else buffer(m, d, type_, pad)
    mu, rs = (torch.full((m,), float("nan"), device="cuda") if save else None for _ in range(2))
    dgc.dgc_layer_norm(x, gamma, b, EPS, y, mu, rs)
    avg, dev, rstd = statistics(X)
    xhat = (X - avg) * rstd
    want = xhat * gamma.double()
    near_error = L * (2 * xhat.abs() + 1) * gamma.double().abs() + 2 * E * want.abs()
    if beta:
        want = want + b.double()
        near_error = near_error + 2 * E * b.double().abs()
    near(y, want, near_error)
    if save:
        near(mu, avg[:, 0], L * dev[:, 0])
        near(rs, rstd[:, 0], L * rstd[:, 0])
    outside_is_untouched(y)


@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("m,d", SIZES)
def test_forward(m, d, type_):
    forward(m, d, type_)


@pytest.mark.parametrize("pad", [1, "odd", "packed"])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
def test_forward_strides(type_, pad):
    for m, d in ((1, 1), (21, 63), (35, 250), (40, 1001), (5, 8192), (3, 8200), (3, 17001)):
        forward(m, d, type_, pad=pad, beta=d != 63, save=d != 250, odd=d in (1001, 17001))
        forward(m, d, type_, pad=pad, in_place=True)


@pytest.mark.parametrize("d", [200, 1500, 5000, 20000])
def test_forward_of_rows_far_from_zero(d):
    """A mean of 2^14 deviations: the deviations, which binary32 holds to 2^-10, are not lost in the
    mean's own rounding."""
    forward(30, d, F32, sigma=1.0, mean=16384.0)
    forward(30, d, F32, sigma=2.0 ** -10, mean=-3.0)


def test_forward_of_constant_rows():
    x = torch.full((4, 300), 0.1, dtype=F32, device="cuda")
    y, beta = torch.empty_like(x), torch.randn(300, device="cuda")
    dgc.dgc_layer_norm(x, torch.ones(300, device="cuda"), beta, EPS, y, None, None)
    # 0.1 - mean is at most the mean's rounding, and its average is taken out again
    near(y, beta.double().expand(4, 300), 2.0 ** -20)


def backward(m, d, type_, residual=True, accumulate=False, pad=0, odd=False, which=(True, True),
             alias=None, mean=0.3):
    gen = generator(m * 3 + d)
    x, dy = normal(gen, m, d, type_, 1.0, mean, pad), normal(gen, m, d, type_, 0.5, pad=pad)
    r = normal(gen, m, d, type_, 0.5, pad=pad) if residual else None
    gamma = weights(d, gen, odd)
    dgamma, dbeta = weights(d, gen, odd) if which[0] else None, (
        weights(d, gen, not odd) if which[1] else None)
    X, Y, R = x.double(), dy.double(), r.double() if residual else 0.0
    G = gamma.double()
    was = [None if t is None else t.double() if accumulate else torch.zeros_like(G)
           for t in (dgamma, dbeta)]
    avg, dev, rstd = statistics(X)
    mu, rs = avg[:, 0].float(), rstd[:, 0].float()
    dx = {"dy": dy, "x": x, "r": r, None: None}[alias]
    dx = buffer(m, d, type_, pad) if dx is None else dx
    ws = workspace(dgc.dgc_layer_norm_backward_workspace(m, d))
    dgc.dgc_layer_norm_backward(dy, x, gamma, mu, rs, r, dx, dgamma, dbeta, accumulate, ws)
    xhat, g = (X - avg) * rstd, Y * G
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xhat).abs().mean(1, keepdim=True)
    want = rstd * (g - m1 - xhat * m2)
    # m1 is off by L a1; m2 by L (3 a2 + a1); xhat by L (2 |xhat| + 1); the rest by 4 E
    h = xhat.abs()
    error = rstd * (L * a1 + h * L * (3 * a2 + a1) + L * (2 * h + 1) * m2.abs()
                    + (L + 8 * E) * (g.abs() + m1.abs() + h * m2.abs()))
    near(dx, want + R, error + 2 * E * (R.abs() if residual else 0.0) + 2 * E * want.abs())
    outside_is_untouched(dx)
    # m roundings of a sum over m rows, and each term's own
    chain = (m + 16) * E
    for t, w, term, own in ((dgamma, was[0], Y * xhat, L * (2 * h + 1) * Y.abs()),
                            (dbeta, was[1], Y, torch.zeros_like(Y))):
        if t is not None:
            near(t, w + term.sum(0), chain * term.abs().sum(0) + own.sum(0) + E * w.abs())


@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("m,d", SIZES + [(3000, 40), (2500, 600), (700, 2048), (650, 4096)])
def test_backward(m, d, type_):
    backward(m, d, type_)
    backward(m, d, type_, residual=False, accumulate=True)


@pytest.mark.parametrize("pad", [1, "odd", "packed"])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
def test_backward_strides(type_, pad):
    for m, d in ((1, 1), (21, 63), (35, 250), (400, 1001), (5, 8192), (3, 8200)):
        backward(m, d, type_, pad=pad, odd=True)
        for alias in ("dy", "x", "r"):
            backward(m, d, type_, pad=pad, alias=alias)


def test_backward_parts():
    for which in ((True, False), (False, True), (False, False)):
        for m, d in ((50, 700), (5, 9000)):
            backward(m, d, BF16, which=which)
    backward(40, 900, F32, mean=16384.0)


def test_no_rows():
    none = buffer(0, 40, BF16)
    gamma = torch.ones(40, device="cuda")
    dg, db = (torch.full((40,), 3.0, device="cuda") for _ in range(2))
    ws = workspace(dgc.dgc_layer_norm_backward_workspace(0, 40))
    dgc.dgc_layer_norm(none, gamma, None, EPS, none, None, None)
    dgc.dgc_layer_norm_backward(none, none, gamma, None, None, None, none, dg, db, True, ws)
    assert (dg == 3).all() and (db == 3).all()
    dgc.dgc_layer_norm_backward(none, none, gamma, None, None, None, none, dg, db, False, ws)
    assert (dg == 0).all() and (db == 0).all()


def test_bad_rows_stay_alone():
    """A row with a NaN or an infinity is NaN, the others do not see it."""
    for d in (100, 3000, 20000):
        x = normal(generator(d), 6, d, F32)
        x[1, 5], x[4, d - 1] = float("nan"), float("inf")
        y, gamma = torch.empty_like(x), torch.ones(d, device="cuda")
        mu, rs = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
        dgc.dgc_layer_norm(x, gamma, None, EPS, y, mu, rs)
        good = torch.tensor([0, 2, 3, 5], device="cuda")
        assert torch.isfinite(y[good]).all() and torch.isfinite(rs[good]).all()
        assert y[1].isnan().all() and y[4].isnan().all() and rs[[1, 4]].isnan().all()


def test_deterministic():
    m, d = 5000, 1111
    x, dy = normal(generator(1), m, d, BF16), normal(generator(2), m, d, BF16)
    gamma = torch.ones(d, device="cuda")
    mu, rs = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    y = buffer(m, d, BF16)
    dgc.dgc_layer_norm(x, gamma, None, EPS, y, mu, rs)
    ws = workspace(dgc.dgc_layer_norm_backward_workspace(m, d))
    runs = []
    for _ in range(3):
        dx, dg, db = buffer(m, d, BF16), torch.empty_like(gamma), torch.empty_like(gamma)
        dgc.dgc_layer_norm_backward(dy, x, gamma, mu, rs, None, dx, dg, db, False, ws)
        runs.append((dx, dg, db))
    for r in runs[1:]:
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(runs[0], r))


def test_gradient_against_differences():
    """The gradient of sum(w y) along a direction, by central differences of the definition in 64
    bits: the step's error is its square times third derivatives of order one, 1e-8; the kernel's dx
    and dgamma are binary32's, 1e-5 of the terms' sum."""
    m, d = 12, 90
    gen = generator(9)
    x, w, v = (torch.randn(m, d, generator=gen, device="cuda") for _ in range(3))
    gamma, vg = (torch.randn(d, generator=gen, device="cuda") for _ in range(2))

    def loss(t):
        X = x.double() + t * v.double()
        avg, _, rstd = statistics(X)
        return ((X - avg) * rstd * (gamma.double() + t * vg.double()) * w.double()).sum().item()

    step = 1e-4
    slope = (loss(step) - loss(-step)) / (2 * step)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mu, rs = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    dg = torch.empty_like(gamma)
    dgc.dgc_layer_norm(x, gamma, None, EPS, y, mu, rs)
    ws = workspace(dgc.dgc_layer_norm_backward_workspace(m, d))
    dgc.dgc_layer_norm_backward(w, x, gamma, mu, rs, None, dx, dg, None, False, ws)
    terms = (dx.double() * v.double()).abs().sum() + (dg.double() * vg.double()).abs().sum()
    got = (dx.double() * v.double()).sum() + (dg.double() * vg.double()).sum()
    assert abs(got.item() - slope) <= 1e-5 * terms.item()


# Rows enough for every block to come round many times, the statistics' loads of 32 rows among them
# (304 blocks of 8, 4 or 1 rows at once, or 152 of one row of 16 warps; the forward pass 456 of them).
MANY = [(50000, 520), (90000, 250), (14000, 2041), (14000, 4096), (6000, 4104), (5600, 8184)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("type_", [F32, BF16])
@pytest.mark.parametrize("m,d", MANY)
def test_forward_of_many_rows(m, d, type_, in_place):
    forward(m, d, type_, in_place=in_place)


@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("m,d", [(20000, 251), (6000, 2041), (3000, 4101)])
def test_forward_of_many_rows_off_boundaries(m, d, type_):
    forward(m, d, type_, pad="packed")
    forward(m, d, type_, pad="odd", in_place=True)


@pytest.mark.parametrize("type_", [F32, BF16])
@pytest.mark.parametrize("m,d", MANY)
def test_backward_of_many_rows(m, d, type_):
    for alias in (None, "dy", "x", "r"):
        backward(m, d, type_, alias=alias)


@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("m,d", [(20000, 251), (6000, 2041), (4000, 4101)])
def test_backward_of_many_rows_off_boundaries(m, d, type_):
    backward(m, d, type_, pad="packed")
    backward(m, d, type_, pad="odd", alias="x")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad", [0, "odd"])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("m,d", [(50000, 520), (14000, 2042), (14000, 4096), (6000, 4104),
                                 (6000, 8184), (1000, 9000), (3, 250), (257, 60)])
def test_whole_numbers_are_exact(m, d, type_, pad, accumulate):
    """Rows of whole numbers whose deviations add up to nothing, a power of two as the reciprocal
    deviation: every sum of the weights' gradients is a whole number below 2^24, exact in any order.
    No row is left out, taken twice or given another one's statistics."""
    gen = generator(m + d)
    row, col = torch.arange(m, device="cuda")[:, None], torch.arange(d, device="cuda")
    dev = (1 - 2 * (col % 2)) * ((col // 2 + row) % 3 + 1)
    mean, rstd = (row % 7 - 3).double(), 2.0 ** (row % 3).double()
    x, dy = buffer(m, d, type_, pad), buffer(m, d, type_, pad)
    x.copy_(dev + mean)
    dy.copy_(torch.randint(-3, 4, (m, d), generator=gen, device="cuda"))
    dgamma, dbeta = (torch.randint(-9, 10, (d,), generator=gen, device="cuda").float()
                     for _ in range(2))
    want = [t.double() if accumulate else torch.zeros(d, device="cuda").double()
            for t in (dgamma, dbeta)]
    want[0] = want[0] + (dy.double() * dev.double() * rstd).sum(0)
    want[1] = want[1] + dy.double().sum(0)
    assert 36 * m + 9 < 2**24
    ws = workspace(dgc.dgc_layer_norm_backward_workspace(m, d))
    dx, gamma = buffer(m, d, type_, pad), torch.ones(d, device="cuda")
    dgc.dgc_layer_norm_backward(dy, x, gamma, mean[:, 0].float(), rstd[:, 0].float(), None, dx,
                                dgamma, dbeta, accumulate, ws)
    assert torch.equal(dgamma.double(), want[0]) and torch.equal(dbeta.double(), want[1])


@pytest.mark.parametrize("cols,ld", [(520, 1 << 24), (521, (1 << 24) + 1), (8200, 1 << 24)])
def test_rows_past_two_to_the_32(cols, ld):
    """Rows far apart, the last of them behind 2^32 entries: on and off 16-byte boundaries, and the
    kernels of long rows."""
    m = 300
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    flat = torch.empty(m * ld, dtype=BF16, device="cuda").view(m, ld)
    x, y, dy, r, dx = (flat[:, i * 65536:i * 65536 + cols] for i in range(5))
    gen = generator(40)
    for t in (x, dy, r):
        t.copy_(torch.randn(m, cols, generator=gen, device="cuda"))
    near_x, near_dy, near_r = x.contiguous(), dy.contiguous(), r.contiguous()
    gamma, beta = weights(cols, gen), weights(cols, gen)
    mu, rs = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    dgc.dgc_layer_norm(x, gamma, beta, EPS, y, mu, rs)
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = workspace(dgc.dgc_layer_norm_backward_workspace(m, cols))
    dgc.dgc_layer_norm_backward(dy, x, gamma, mu, rs, r, dx, dg, db, False, ws)
    X, DY, G = near_x.double(), near_dy.double(), gamma.double()
    avg, _, rstd = statistics(X)
    xhat, g = (X - avg) * rstd, DY * G
    h = xhat.abs()
    near(y, xhat * G + beta.double(), (L * (2 * h + 1) + 4 * E * h) * G.abs()
         + 4 * E * beta.double().abs())
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xhat).abs().mean(1, keepdim=True)
    want = rstd * (g - m1 - xhat * m2)
    # as in backward() above, and the given rstd and mean are themselves off by L
    error = rstd * (2 * L * a1 + h * L * (4 * a2 + 2 * a1) + 2 * L * (2 * h + 1) * m2.abs()
                    + (2 * L + 8 * E) * (g.abs() + m1.abs() + h * m2.abs()))
    R = near_r.double()
    near(dx, want + R, error + 2 * E * R.abs() + 2 * E * want.abs())
    chain = (m + 16) * E
    near(dg, (DY * xhat).sum(0), chain * (DY * xhat).abs().sum(0)
         + (2 * L * (2 * h + 1) * DY.abs()).sum(0))
    near(db, DY.sum(0), chain * DY.abs().sum(0))
