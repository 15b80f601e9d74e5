"""The feed-forward calls at the ends of their ranges, on the GPU: gates of every magnitude on every
route of the products."""
import math

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
ACTS = {"silu": dgc.ACT_SILU, "gelu": dgc.ACT_GELU, "gelu_tanh": dgc.ACT_GELU_TANH,
        "relu": dgc.ACT_RELU}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def rows(t, odd):
    """t's entries in rows on 16-byte boundaries, or off them."""
    r, c = t.shape
    if not odd:
        o = torch.zeros(r, -(-c // 8) * 8, dtype=t.dtype, device="cuda")[:, :c]
    else:
        ld = c | 1
        o = torch.zeros(r * ld + 1, dtype=t.dtype, device="cuda")[1:].view(r, ld)[:, :c]
    o.copy_(t)
    return o


def block_of_gates(act, terms, m, odd):
    """What the two calls that evaluate the activation make of gates that are given as sums of
    bfloat16 terms (len(terms[0]) of them each), with up, dh = 1: hidden, and from the gates' first
    terms alone d_gate and d_up, of m equal rows. Every sum but the gate's is exact."""
    f, k = len(terms), len(terms[0])
    t = torch.tensor(terms, dtype=torch.float64, device="cuda").to(BF16)
    x = rows(torch.ones(m, k, dtype=BF16, device="cuda"), odd)
    wu = torch.zeros(f, k, dtype=BF16, device="cuda")
    wu[:, 0] = 1.0
    hidden = rows(torch.full((m, f), 7.0, dtype=BF16, device="cuda"), odd)
    st = status_word()
    dgc.dgc_ffn_gate(x, rows(t, odd), rows(wu, odd), ACTS[act], hidden, None, None, st)
    gate = rows(t[:, 0].repeat(m, 1), odd)
    up = rows(torch.ones_like(gate), odd)
    dg, du = rows(torch.full_like(gate, 7.0), odd), rows(torch.full_like(gate, 7.0), odd)
    dy, wd = torch.zeros(m, 8, dtype=BF16, device="cuda"), torch.zeros(8, f, dtype=BF16,
                                                                       device="cuda")
    dy[:, 0], wd[0] = 1.0, 1.0
    dgc.dgc_ffn_down_backward(rows(dy, odd), rows(wd, odd), gate, up, ACTS[act], dg, du, st)
    assert dgc.dgc_read_status(st) == 0
    return t.double(), hidden, dg, du


ROUTES = [(1, False), (2, True), (3, False), (3, True), (200, False), (300, True)]


@pytest.mark.parametrize("m,odd", ROUTES)
@pytest.mark.parametrize("act", list(ACTS))
def test_gates_up_to_the_largest(act, m, odd):
    """From 1e4 on the activations are the identity and 0, their slopes 1 and 0, to the last bit."""
    g = [s * v for v in (1e4, 1e10, 1.8e19, 1.9e19, 2e19, 1e20, 1e30, 3e38) for s in (1, -1)]
    t, hidden, dg, du = block_of_gates(act, [[v] for v in g], m, odd)
    value = t[:, 0].clamp_min(0.0).to(BF16).expand(m, -1)
    slope = (t[:, 0] > 0).to(BF16).expand(m, -1)
    assert torch.equal(hidden, value)
    assert torch.equal(du, value)
    assert torch.equal(dg, slope)


def off_by(got, want):
    return ((got.double() - want).abs() / want.abs()).max().item()


@pytest.mark.parametrize("m,odd", ROUTES)
def test_silu_where_the_sigmoid_is_subnormal(m, odd):
    """Gates from -87.3 down to -88.7: the sigmoid is below 2^-126, its product with the gate is not.
    Error: bfloat16's rounding (2^-8), and the exponent's in binary32 (up to 128 * 2^-24 * ln 2)
    with the instructions' 2^-22: below 2^-16 in all."""
    t, hidden, dg, du = block_of_gates("silu", [[-g] for g in (88.5, 88.0, 87.5, 87.0, 80.0)], m,
                                       odd)
    g = t[:, 0]
    s = torch.exp(g) / (1 + torch.exp(g))
    tol = 2.0 ** -8 + 2.0 ** -16
    assert off_by(hidden, g * s) <= tol
    assert off_by(du, g * s) <= tol
    assert off_by(dg, s * (1 + g * (1 - s))) <= tol


@pytest.mark.parametrize("m,odd", ROUTES)
def test_tanh_gelu_where_the_sigmoid_is_subnormal(m, odd):
    """The same of the sigmoid in tanh GELU, between two bfloat16 gates: -10 - 1/32 and their like.
    The argument, about 88, takes five roundings more: 2^-14 in all."""
    terms = [[-10.0, -1 / 32], [-10.0, -3 / 64], [-10.0, 1 / 32]]
    t, hidden, _, _ = block_of_gates("gelu_tanh", terms, m, odd)
    g = t.sum(1)
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    assert off_by(hidden, g * torch.exp(z) / (1 + torch.exp(z))) <= 2.0 ** -8 + 2.0 ** -14


@pytest.mark.parametrize("ld", [0, 2**62])
def test_a_weight_gradient_of_one_row(ld):
    dy = torch.full((3, 8), 2.0, dtype=BF16, device="cuda")[:, :1]
    x = torch.arange(72, device="cuda").view(3, 24).to(BF16)
    flat, st = torch.full((32,), 7.0, device="cuda"), status_word()
    dgc.dgc_ffn_weight_grad(dy, x, dgc.dgc_matrix(flat.data_ptr(), 1, 24, ld, dgc.F32, 0), False,
                            st, None)
    assert torch.equal(flat[:24], 2 * x.float().sum(0)) and flat[24:].eq(7.0).all()
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
@pytest.mark.parametrize("m", [1, 2])
@pytest.mark.parametrize("d,f", [(65, 300), (257, 511), (1027, 333), (3000, 2049), (4095, 70),
                                 (4901, 2603)])
def test_one_and_two_tokens_off_16_byte_boundaries(d, f, m, dtype):
    """Long sums read entry by entry: steps of 256 entries with a short last one, a sum in eight parts
    and, from 2432 rows of weights on (4864 of the down projection's), in one."""
    from test_gpu_ffn import ACTS as names, forward

    forward(m, d, f, list(names)[(d + f) % 4], dtype, d, "odd", m == 2, d % 2 == 1)


@pytest.mark.parametrize("m", [1, 2])
@pytest.mark.parametrize("which", range(3))
def test_one_operand_of_few_tokens_off_16_byte_boundaries(which, m):
    """x, the gate's and the up projection's weights in turn, within the roundings of the sums of
    those that all lie on them."""
    gen = torch.Generator(device="cuda").manual_seed(which)
    k, f = 1999, 301
    t = [(torch.randn(r, k, generator=gen, device="cuda") * s).to(BF16)
         for r, s in ((m, 1.0), (f, k ** -0.5), (f, k ** -0.5))]
    st, outs = status_word(), []
    for off in (which, None):
        x, wg, wu = (rows(a, i == off) for i, a in enumerate(t))
        out = [torch.empty(m, f, dtype=BF16, device="cuda") for _ in range(3)]
        dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_RELU, *out, st)
        outs.append([o.double() for o in out])
    assert dgc.dgc_read_status(st) == 0
    x, wg, wu = (a.double() for a in t)
    for i, w in ((1, wg), (2, wu)):  # two binary32 sums, each rounded: K 2^-23 of the terms, a unit
        terms = x.abs() @ w.abs().t()
        assert ((outs[0][i] - outs[1][i]).abs()
                <= 2 * k * 2.0 ** -23 * terms + 2.0 ** -7 * outs[1][i].abs()).all()


@pytest.mark.parametrize("tokens,cols,shift,odd", [
    (8, 64, 0, False),       # added by the bulk reduction
    (8, 61, 0, False),       # its last columns one by one
    (8, 64, 1, False),       # every column
    (8, 64, 0, True),        # on the ordinary cores
    (1 << 16, 64, 0, False)])  # by the parts' join
def test_subnormal_sums_are_kept(tokens, cols, shift, odd):
    """dw = 2^-130 + 2^-130 and 1.5 * 2^-126 - 2^-126, exact on every route of the addition."""
    for start, left, right, want in ((2.0 ** -130, 2.0 ** -65, 2.0 ** -65, 2.0 ** -129),
                                     (1.5 * 2.0 ** -126, -2.0 ** -63, 2.0 ** -63, 2.0 ** -127)):
        dy, x = torch.zeros(tokens, 64, dtype=BF16), torch.zeros(tokens, cols, dtype=BF16)
        dy[tokens // 2], x[tokens // 2] = left, right
        flat = torch.full((64 * 64 + 8,), start, device="cuda")
        dw, st = flat[shift:shift + 64 * 64].view(64, 64)[:, :cols], status_word()
        ws = torch.empty(max(1, dgc.dgc_ffn_weight_grad_workspace(64, cols, tokens)),
                         dtype=torch.uint8, device="cuda")
        dgc.dgc_ffn_weight_grad(rows(dy, odd), rows(x, odd), dw, True, st, ws)
        assert dgc.dgc_read_status(st) == 0
        assert torch.equal(dw.double().cpu(), torch.full((64, cols), want, dtype=torch.float64))
