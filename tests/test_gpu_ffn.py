"""The gated feed-forward block's five calls on the GPU against the formulas in 64 bits.

Tolerances, all of them fixed by the arithmetic. u = 2^-8 (bfloat16, 8 significand bits) or 2^-11
(float16, 11 bits, normal range) is a half unit in the last place, relative. A product with K terms is summed in binary32:
its error is within K * 2^-23 of the sum of its terms' magnitudes (S). A result r is then rounded
once: |error| <= u |r| + 2^-25 (float16's subnormals) + its sum's error carried through the
epilogue's smooth functions, whose slopes are below 1.13, plus 4e-6 of the value for the fast
exponential and division."""
import math
import random

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
ACTS = {"silu": dgc.ACT_SILU, "gelu": dgc.ACT_GELU, "gelu_tanh": dgc.ACT_GELU_TANH,
        "relu": dgc.ACT_RELU}
HALF_ULP = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def padded(rows, cols, dtype, pad=0, fill=float("nan")):
    """A view whose rows start on 16-byte boundaries, in a buffer filled with NaN; pad "odd": an odd
    number of entries from row to row, the first one off every boundary."""
    if pad == "odd":
        ld = cols | 1
        flat = torch.full((rows * ld + 2,), fill, dtype=dtype, device="cuda")
        return flat[1:1 + rows * ld].view(rows, ld)[:, :cols]
    ld = -(-cols // 8) * 8 + pad
    return torch.full((max(rows, 1), max(ld, 8)), fill, dtype=dtype, device="cuda")[:rows, :cols]


def rand(gen, rows, cols, dtype, sigma=1.0, pad=0):
    t = padded(rows, cols, dtype, pad)
    t.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * sigma)
    return t


def value_slope(act, g):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), (0.5 * (1 + t)
                                   + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g))
    return torch.relu(g), (g > 0).double()


def near(got, want, sum_error, dtype):
    assert got.dtype == dtype and got.shape == want.shape
    tol = HALF_ULP[dtype] * want.abs() * 1.001 + 2.0 ** -25 + sum_error + 4e-6 * want.abs()
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float((got.double() - want).abs().max()))


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def product(a, b):
    """a b and the bound on its binary32 sum's error."""
    k = a.shape[1]
    return a @ b, (a.abs() @ b.abs()) * (k * 2.0 ** -23)


def forward(m, d, f, act, dtype, seed=0, pad=0, save=True, residual=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = rand(gen, m, d, dtype, 1.0, pad)
    wg, wu = (rand(gen, f, d, dtype, max(d, 1) ** -0.5, pad) for _ in range(2))
    wd = rand(gen, d, f, dtype, max(f, 1) ** -0.5, pad)
    hidden, gate, up = (padded(m, f, dtype, pad) for _ in range(3))
    y, st = padded(m, d, dtype, pad), status_word()
    dgc.dgc_ffn_gate(x, wg, wu, ACTS[act], hidden, gate if save else None, up if save else None,
                     st)
    g, ge = product(x.double(), wg.double().t())
    u, ue = product(x.double(), wu.double().t())
    v, _ = value_slope(act, g)
    near(hidden, v * u, 1.13 * ge * u.abs() + v.abs() * ue + 1.13 * ge * ue, dtype)
    if save:
        near(gate, g, ge, dtype)
        near(up, u, ue, dtype)
    dgc.dgc_ffn_down(hidden, wd, x if residual else None, y, st)
    p, pe = product(hidden.double(), wd.double().t())
    near(y, p + x.double() if residual else p, pe + 2.0 ** -23 * (p.abs() + x.double().abs()),
         dtype)
    assert dgc.dgc_read_status(st) == 0


def backward(m, d, f, act, dtype, seed=0, pad=0, residual=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dy = rand(gen, m, d, dtype, 0.5, pad)
    wg, wu = (rand(gen, f, d, dtype, max(d, 1) ** -0.5, pad) for _ in range(2))
    wd = rand(gen, d, f, dtype, max(f, 1) ** -0.5, pad)
    gate, up = (rand(gen, m, f, dtype, 1.5, pad) for _ in range(2))
    dg, du = (padded(m, f, dtype, pad) for _ in range(2))
    dx, st = padded(m, d, dtype, pad), status_word()
    dgc.dgc_ffn_down_backward(dy, wd, gate, up, ACTS[act], dg, du, st)
    dh, he = product(dy.double(), wd.double())
    v, s = value_slope(act, gate.double())
    # a slope that nearly cancels is off by a few 2^-24 of its terms (below 2 in magnitude)
    near(dg, dh * up.double() * s, (he * 1.13 + dh.abs() * 4e-6) * up.double().abs(), dtype)
    near(du, dh * v, he * v.abs() + 4e-6 * dh.abs(), dtype)
    dgc.dgc_ffn_gate_backward(dg, du, wg, wu, dy if residual else None, dx, st)
    p, pe = product(torch.cat([dg, du], 1).double(), torch.cat([wg, wu], 0).double())
    near(dx, p + dy.double() if residual else p, pe + 2.0 ** -23 * (p.abs() + dy.double().abs()),
         dtype)
    assert dgc.dgc_read_status(st) == 0


def weight_grad(tokens, rows, cols, dtype, accumulate, seed=0, pad=0, shift=0, extra=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dy, x = rand(gen, tokens, rows, dtype, 0.5, pad), rand(gen, tokens, cols, dtype, 1.0, pad)
    n = rows * (cols + extra)
    bucket = torch.randn(shift + n + 64, generator=gen, device="cuda")
    dw = bucket[shift:shift + n].view(rows, cols + extra)[:, :cols]
    before, keep = dw.clone().double(), bucket.clone()
    if not accumulate and rows and cols:
        dw.fill_(float("nan"))
    st = status_word()
    nb = dgc.dgc_ffn_weight_grad_workspace(rows, cols, tokens)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda") if nb else None
    dgc.dgc_ffn_weight_grad(dy, x, dw, accumulate, st, ws)
    assert dgc.dgc_read_status(st) == 0
    p, pe = product(dy.double().t(), x.double())
    want = p + before if accumulate else p
    err = (dw.double() - want).abs()
    assert (err <= pe + 2.0 ** -22 * (p.abs() + want.abs()) + 1e-40).all(), float(err.max())
    dw.copy_(keep[shift:shift + n].view(rows, cols + extra)[:, :cols])
    assert torch.equal(bucket, keep)  # nothing written outside the matrix


SHAPES = [(1, 8, 8), (1, 64, 128), (3, 1, 1), (5, 7, 9), (1, 1024, 4096), (8, 100, 33),
          (127, 65, 129), (128, 64, 256), (129, 200, 257), (300, 1001, 515), (2048, 256, 640),
          (1000, 328, 2721), (20000, 64, 72)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d,f", SHAPES)
def test_forward(m, d, f, dtype):
    forward(m, d, f, list(ACTS)[(m + f) % 4], dtype, seed=m + d + f)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d,f", SHAPES)
def test_backward(m, d, f, dtype):
    backward(m, d, f, list(ACTS)[(m + f) % 4], dtype, seed=m + d + f)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m", [1, 2, 3])
@pytest.mark.parametrize("d,f", [(1, 1), (7, 3), (33, 65), (264, 1000), (1027, 333), (3000, 2049)])
def test_one_to_three_tokens(m, d, f, dtype):
    forward(m, d, f, list(ACTS)[(d + f) % 4], dtype, seed=d, pad=8, save=m != 2,
            residual=d % 2 == 1)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d,f", [(1, 1, 1), (2, 9, 5), (7, 33, 64), (130, 65, 129), (300, 129, 257),
                                   (65, 1001, 333), (1000, 70, 900)])
def test_rows_off_16_byte_boundaries(m, d, f, dtype):
    act = list(ACTS)[(m + d) % 4]
    forward(m, d, f, act, dtype, m, "odd", m % 2 == 0, m != 7)
    backward(m, d, f, act, dtype, m, "odd", m != 7)
    for accumulate in (False, True):
        weight_grad(m, d, f, dtype, accumulate, m, "odd", 1, 2)


def test_long_sum_off_16_byte_boundaries():
    weight_grad(9000, 65, 130, BF16, True, 3, "odd")


@pytest.mark.parametrize("which", range(8))
def test_one_matrix_off_16_byte_boundaries(which):
    """Each operand, input and result in turn: the same values as with all of them on."""
    gen = torch.Generator(device="cuda").manual_seed(which)
    m, d, f = 200, 72, 136
    x, dy = rand(gen, m, d, BF16), rand(gen, m, d, BF16)
    wg, wu, wd = rand(gen, f, d, BF16, 0.1), rand(gen, f, d, BF16, 0.1), rand(gen, d, f, BF16, 0.1)

    def run(off):
        def moved(t, i):
            if i != off:
                return t
            o = padded(*t.shape, t.dtype, "odd")
            o.copy_(t)
            return o

        out = [moved(padded(m, f, BF16), 4 if i == 0 else 5 if i == 1 else -2) for i in range(5)]
        hidden, gate, up, dg, du = out
        y, dx = moved(padded(m, d, BF16), 6), moved(padded(m, d, BF16), 7)
        st = status_word()
        X, D, G, W = moved(x, 0), moved(dy, 1), moved(wg, 2), moved(wd, 3)
        dgc.dgc_ffn_gate(X, G, wu, dgc.ACT_SILU, hidden, gate, up, st)
        dgc.dgc_ffn_down(hidden, W, X, y, st)
        dgc.dgc_ffn_down_backward(D, W, gate, up, dgc.ACT_SILU, dg, du, st)
        dgc.dgc_ffn_gate_backward(dg, du, G, wu, D, dx, st)
        dw = torch.empty(f, d, device="cuda")
        dgc.dgc_ffn_weight_grad(dg, X, dw, False, st, None)
        assert dgc.dgc_read_status(st) == 0
        return [t.double() for t in (hidden, gate, up, dg, du, y, dx, dw)]

    for got, want in zip(run(which), run(-1)):  # two orders of sums and one or two roundings each
        assert (got - want).norm() <= 2.0 ** -7 * want.norm()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_activations(act, dtype):
    forward(70, 96, 200, act, dtype, seed=5, pad=16, save=act != "gelu", residual=False)
    backward(70, 96, 200, act, dtype, seed=5, pad=16, residual=False)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 1), (1, 64, 64), (33, 128, 256), (63, 130, 70), (64, 7, 1000), (65, 257, 513),
    (1000, 384, 132), (4096, 128, 256), (5000, 200, 300), (16384, 64, 8), (700, 2560, 3000)])
def test_weight_grad(tokens, rows, cols, accumulate, dtype):
    weight_grad(tokens, rows, cols, dtype, accumulate, seed=tokens)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows,cols", [(65536, 300, 390), (40001, 500, 301)])
def test_weight_grad_in_parts_of_wide_tiles(tokens, rows, cols, accumulate):
    """Sums long enough that the parts go to the workspace from 256 x 256 tiles."""
    assert dgc.dgc_ffn_weight_grad_workspace(rows, cols, tokens) > 0
    weight_grad(tokens, rows, cols, BF16, accumulate, seed=1, pad=8)


@pytest.mark.parametrize("shift,extra", [(1, 0), (4, 1), (3, 3), (0, 4), (8, 2)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens", [100, 3000])
def test_weight_grad_in_odd_pieces_of_a_bucket(tokens, accumulate, shift, extra):
    weight_grad(tokens, 150, 201, BF16, accumulate, 3, 8, shift, extra)


@pytest.mark.parametrize("m,d,f", [(0, 16, 16), (4, 0, 16), (4, 16, 0), (0, 0, 0), (200, 0, 300),
                                   (200, 300, 0)])
def test_empty(m, d, f):
    forward(m, d, f, "silu", BF16)
    backward(m, d, f, "silu", BF16)
    for acc in (False, True):
        weight_grad(m, d, f, BF16, acc)
        weight_grad(m, f, d, BF16, acc)


@pytest.mark.parametrize("seed", range(10))
def test_random_shapes(seed):
    r = random.Random(seed)
    size = lambda hi: int(2 ** r.uniform(0, math.log2(hi)))  # noqa: E731
    m, d, f = size(3000), size(1500), size(3000)
    dtype, act, pad = r.choice((F16, BF16)), r.choice(list(ACTS)), 8 * r.randrange(3)
    forward(m, d, f, act, dtype, seed, pad, r.random() < 0.5, r.random() < 0.5)
    backward(m, d, f, act, dtype, seed, pad, r.random() < 0.5)
    weight_grad(m, d, f, dtype, r.random() < 0.5, seed, pad, r.randrange(5), r.randrange(5))


@pytest.mark.parametrize("cols", [1, 31, 33, 64, 97, 100])
def test_results_that_are_columns_of_a_wider_matrix(cols):
    """Nothing is written beside a result's own columns, whatever their number."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    m, k = 150, 72
    wide = [torch.full((m, 128), 7.0, dtype=BF16, device="cuda") for _ in range(7)]
    hidden, gate, up, y, dg, du, dx = (w[:, 8:8 + cols] for w in wide)
    x, w1, w2 = rand(gen, m, k, BF16), rand(gen, cols, k, BF16), rand(gen, cols, k, BF16)
    wd, st = rand(gen, k, cols, BF16), status_word()
    dgc.dgc_ffn_gate(x, w1, w2, dgc.ACT_SILU, hidden, gate, up, st)
    dgc.dgc_ffn_down(x, w1, None, y, st)
    dgc.dgc_ffn_down_backward(x, wd, gate, up, dgc.ACT_SILU, dg, du, st)
    w3 = rand(gen, m, cols, BF16)
    dgc.dgc_ffn_gate_backward(rand(gen, m, m, BF16), rand(gen, m, m, BF16), w3, w3, y, dx, st)
    wide32 = torch.full((k, 128), 7.0, device="cuda")
    for acc in (False, True):
        dgc.dgc_ffn_weight_grad(x, y, wide32[:, 4:4 + cols], acc, st, None)
    assert dgc.dgc_read_status(st) == 0
    for w, at in [(w, 8) for w in wide] + [(wide32, 4)]:
        assert w[:, :at].eq(7.0).all() and w[:, at + cols:].eq(7.0).all()
        assert not w[:, at:at + cols].eq(7.0).all()


def test_results_in_place():
    """y over the residual, d_gate and d_up over gate and up, dx over the residual: the same bits
    as into fresh buffers."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    m, d, f = 333, 192, 520
    x, dy = rand(gen, m, d, BF16), rand(gen, m, d, BF16)
    hidden, gate, up = (rand(gen, m, f, BF16) for _ in range(3))
    wd, wg, wu = rand(gen, d, f, BF16), rand(gen, f, d, BF16), rand(gen, f, d, BF16)
    st = status_word()
    y, dx, dg, du = padded(m, d, BF16), padded(m, d, BF16), padded(m, f, BF16), padded(m, f, BF16)
    dgc.dgc_ffn_down(hidden, wd, x, y, st)
    dgc.dgc_ffn_down_backward(dy, wd, gate, up, dgc.ACT_SILU, dg, du, st)
    dgc.dgc_ffn_gate_backward(dg, du, wg, wu, dy, dx, st)
    dgc.dgc_ffn_down(hidden, wd, x, x, st)
    dgc.dgc_ffn_down_backward(dy, wd, gate, up, dgc.ACT_SILU, gate, up, st)
    dgc.dgc_ffn_gate_backward(gate, up, wg, wu, dy, dy, st)
    assert dgc.dgc_read_status(st) == 0
    for a, b in ((x, y), (gate, dg), (up, du), (dy, dx)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_entries_that_are_not_finite_stay_in_their_rows(bad):
    gen = torch.Generator(device="cuda").manual_seed(1)
    m, d, f = 140, 72, 130
    x, wg, wu = rand(gen, m, d, BF16), rand(gen, f, d, BF16, 0.1), rand(gen, f, d, BF16, 0.1)
    hidden, gate, up = (padded(m, f, BF16) for _ in range(3))
    st = status_word()
    dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_SILU, hidden, gate, up, st)
    clean = hidden.clone()
    x[137, 70] = bad
    dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_SILU, hidden, gate, up, st)
    rows = torch.arange(m, device="cuda") != 137
    assert torch.equal(hidden[rows], clean[rows])
    assert not torch.isfinite(gate[137]).any() and not torch.isfinite(up[137]).any()
    want = (x[137].double() * wg.double()).sum(1)
    assert torch.equal(torch.isnan(gate[137]), torch.isnan(want))
    # a NaN in a gradient's row reaches that row of the weight gradient alone
    dy, xs = rand(gen, 100, 80, BF16), rand(gen, 100, 40, BF16)
    dy[3, 5] = float("nan")
    dw = torch.zeros(80, 40, device="cuda")
    dgc.dgc_ffn_weight_grad(dy, xs, dw, False, st, None)
    assert torch.isnan(dw[5]).all() and torch.isfinite(dw[torch.arange(80) != 5]).all()


@pytest.mark.parametrize("act", list(ACTS))
def test_activations_far_out(act):
    """Gates of every magnitude, both signs, zero and subnormal."""
    g = torch.tensor([0.0, -0.0, 1e-8, -1e-8, 0.5, -0.5, 3.0, -3.0, 20.0, -20.0, 89.0, -89.0,
                      300.0, -300.0, 3e4, -3e4], device="cuda")
    m, d = 2, 16
    x = torch.zeros(m, d, device="cuda")
    x[:, 0] = 1.0
    x = x.to(BF16)
    wg, wu = torch.zeros(16, d, device="cuda"), torch.zeros(16, d, device="cuda")
    wg[:, 0], wu[:, 0] = g, 1.0
    wg, wu = wg.to(BF16), wu.to(BF16)
    hidden, st = padded(m, 16, BF16), status_word()
    dgc.dgc_ffn_gate(x, wg, wu, ACTS[act], hidden, None, None, st)
    v, s = value_slope(act, wg[:, 0].double())
    near(hidden[0], v, 1e-30, BF16)
    assert torch.equal(hidden[0], hidden[1])
    gate = wg[:, 0].repeat(m, 1).contiguous()
    up = torch.ones_like(gate)
    dg, du = torch.empty_like(gate), torch.empty_like(gate)
    dgc.dgc_ffn_down_backward(x[:, :1].repeat(1, 8), torch.eye(8, 16, device="cuda").to(BF16) * 0
                              + (torch.arange(8, device="cuda")[:, None] == 0).to(BF16),
                              gate, up, ACTS[act], dg, du, st)
    near(dg[1], s, torch.full_like(s, 8e-6), BF16)
    near(du[1], v, torch.full_like(v, 4e-6), BF16)
    assert dgc.dgc_read_status(st) == 0


def test_gradients_against_differences():
    """The whole block's gradients against central differences of its 64-bit forward pass along
    random directions. The float16 roundings of the saved tensors and of the gradients, each an
    error of about 2^-11 / sqrt 3 of a norm, bound the agreement: 9 * 2^-12 of the gradient's
    norm, several times their root-mean-square sum."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    m, d, f, dtype = 96, 80, 136, F16
    x = rand(gen, m, d, dtype)
    wg, wu, wd = (rand(gen, f, d, dtype, 0.1), rand(gen, f, d, dtype, 0.1),
                  rand(gen, d, f, dtype, 0.1))
    dy = rand(gen, m, d, dtype)
    hidden, gate, up, dg, du = (padded(m, f, dtype) for _ in range(5))
    y, dx, st = padded(m, d, dtype), padded(m, d, dtype), status_word()
    dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_SILU, hidden, gate, up, st)
    dgc.dgc_ffn_down(hidden, wd, x, y, st)
    dgc.dgc_ffn_down_backward(dy, wd, gate, up, dgc.ACT_SILU, dg, du, st)
    dgc.dgc_ffn_gate_backward(dg, du, wg, wu, dy, dx, st)
    grads = [dx]
    for a, b in ((dg, x), (du, x), (dy, hidden)):
        dw = torch.empty(a.shape[1], b.shape[1], device="cuda")
        dgc.dgc_ffn_weight_grad(a, b, dw, False, st, None)
        grads.append(dw)
    assert dgc.dgc_read_status(st) == 0

    def loss(x, wg, wu, wd):
        h = value_slope("silu", x @ wg.t())[0] * (x @ wu.t())
        return ((h @ wd.t() + x) * dy.double()).sum()

    at = [t.double() for t in (x, wg, wu, wd)]
    for i, grad in enumerate(grads):
        for _ in range(3):
            v = torch.randn(at[i].shape, generator=gen, device="cuda").double()
            e = 1e-5
            hi, lo = ([t + s * e * v if j == i else t for j, t in enumerate(at)] for s in (1, -1))
            diff = float((loss(*hi) - loss(*lo)) / (2 * e))
            got = float((grad.double() * v).sum())
            assert abs(got - diff) <= 3 * 2.0 ** -12 * float(grad.double().norm()) * 3.0


def test_runs_agree_bitwise_on_a_side_stream():
    gen = torch.Generator(device="cuda").manual_seed(2)
    dy, x = rand(gen, 9000, 264, BF16), rand(gen, 9000, 200, BF16)
    ws = torch.empty(dgc.dgc_ffn_weight_grad_workspace(264, 200, 9000), dtype=torch.uint8,
                     device="cuda")
    assert ws.numel() > 0  # the sum over the tokens is split
    st, outs = status_word(), []
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side, side):
        with torch.cuda.stream(s):
            dw = torch.empty(264, 200, device="cuda")
            dgc.dgc_ffn_weight_grad(dy, x, dw, False, st, ws)
            outs.append(dw)
        s.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[1], outs[2])


def test_calls_on_several_streams_at_once():
    """Two streams of this library's calls and one of library products, all using the tensor cores:
    the same bits as one after the other."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    sets, st = [], status_word()
    for m, d, f in ((700, 256, 1000), (1500, 512, 520)):
        x, dy = rand(gen, m, d, BF16), rand(gen, m, d, BF16)
        w = [rand(gen, f, d, BF16, 0.05) for _ in range(2)] + [rand(gen, d, f, BF16, 0.05)]
        sets.append((x, dy, w, [padded(m, f, BF16) for _ in range(5)],
                     [padded(m, d, BF16) for _ in range(2)], torch.empty(f, d, device="cuda")))

    def run(s):
        x, dy, (wg, wu, wd), (hidden, gate, up, dg, du), (y, dx), dw = s
        dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_GELU_TANH, hidden, gate, up, st)
        dgc.dgc_ffn_down(hidden, wd, x, y, st)
        dgc.dgc_ffn_down_backward(dy, wd, gate, up, dgc.ACT_GELU_TANH, dg, du, st)
        dgc.dgc_ffn_gate_backward(dg, du, wg, wu, dy, dx, st)
        dgc.dgc_ffn_weight_grad(dg, x, dw, False, st, None)
        return [hidden, gate, up, dg, du, y, dx, dw]

    want = [[t.clone() for t in run(s)] for s in sets]
    a = rand(gen, 2048, 2048, BF16)
    product_alone = a @ a
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                run(s)
        with torch.cuda.stream(streams[2]):
            b = a @ a
    torch.cuda.synchronize()
    assert dgc.dgc_read_status(st) == 0
    assert torch.equal(b, product_alone)
    for s, w in zip(sets, want):
        x, dy, _, inner, outer, dw = s
        for got, ref in zip([*inner, *outer, dw], w):
            assert torch.equal(got, ref)


def test_graph_replays():
    gen = torch.Generator(device="cuda").manual_seed(3)
    m, d, f = 200, 136, 264
    x, wg, wu, wd = (rand(gen, m, d, BF16), rand(gen, f, d, BF16, 0.1),
                     rand(gen, f, d, BF16, 0.1), rand(gen, d, f, BF16, 0.1))
    hidden, y, st = padded(m, f, BF16), padded(m, d, BF16), status_word()

    def step():
        dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_GELU, hidden, None, None, st)
        dgc.dgc_ffn_down(hidden, wd, x, y, st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(rand(gen, m, d, BF16))
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone()
    step()
    assert torch.equal(got, y) and dgc.dgc_read_status(st) == 0


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Results and operands of more than 2^32 entries, their last rows against binary64."""
    m, d, f = 530_000, 64, 8200
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, wg, wu = rand(gen, m, d, BF16), rand(gen, f, d, BF16, 0.1), rand(gen, f, d, BF16, 0.1)
    hidden, st = torch.empty(m, f, dtype=BF16, device="cuda"), status_word()
    assert hidden.numel() > 1 << 32
    dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_RELU, hidden, None, None, st)
    last = slice(m - 300, m)
    g, ge = product(x[last].double(), wg.double().t())
    u, ue = product(x[last].double(), wu.double().t())
    near(hidden[last], torch.relu(g) * u, ge * u.abs() + g.abs() * ue + ge * ue, BF16)
    wd, y = rand(gen, 40, f, BF16, 0.01), torch.empty(m, 40, dtype=BF16, device="cuda")
    dgc.dgc_ffn_down(hidden, wd, None, y, st)
    p, pe = product(hidden[last].double(), wd.double().t())
    near(y[last], p, pe, BF16)
    del y
    # a weight gradient of more than 2^32 entries, from rows of the same big matrix
    dy = rand(gen, 8, 530_000, BF16)
    dw = torch.empty(530_000, f, device="cuda")
    dgc.dgc_ffn_weight_grad(dy, hidden[:8], dw, False, st, None)
    p, pe = product(dy[:, last].double().t(), hidden[:8].double())
    assert ((dw[last].double() - p).abs() <= pe + 2.0 ** -22 * p.abs() + 1e-40).all()
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("m,n,k", [
    (100, 512, 200),      # single blocks, each a whole sum
    (100, 1024, 4096),    # a cluster's blocks, a part of the sum each
    (4096, 4096, 256),    # pairs of blocks, several tiles each
    (512, 2048, 8192)])   # few tiles of long sums
def test_a_copy_that_never_arrives(m, n, k):
    """The waits give up, the status says so, and the next call finds everything in order."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    h, w, y = rand(gen, m, k, BF16), rand(gen, n, k, BF16, k ** -0.5), padded(m, n, BF16)
    st = status_word()
    dgc.dgc_selftest_ffn_timeout(h, w, y, st, 20)
    assert dgc.dgc_read_status(st) == dgc.ETIMEOUT
    st.zero_()
    dgc.dgc_ffn_down(h, w, None, y, st)
    p, pe = product(h.double(), w.double().t())
    near(y, p, pe, BF16)
    assert dgc.dgc_read_status(st) == 0
