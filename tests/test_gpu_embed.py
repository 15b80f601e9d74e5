"""Embedding lookup and its gradient on the GPU against their definitions in 64 bits."""
import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc
from layer_helpers import (BF16, E, F16, F32, bits, buffer, generator, near, normal,
                           outside_is_untouched, status_word, workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def tokens_of(kind, n, vocab, gen):
    if kind == "one":
        t = torch.full((n,), vocab // 2, device="cuda")
    elif kind == "head":  # half of them the same word
        t = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
        t[torch.rand(n, generator=gen, device="cuda") < 0.5] = vocab - 1
    elif kind == "runs":  # words met 31, 32, 33, 64, 65 and 97 times
        t = torch.arange(vocab, device="cuda").repeat_interleave(
            torch.tensor([31, 32, 33, 64, 65, 97, 0, 1], device="cuda").repeat(vocab)[:vocab])
        t = t.repeat(-(-n // max(t.numel(), 1)))[:n]
        t = t[torch.randperm(n, generator=gen, device="cuda")]
    else:
        t = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    return t


@pytest.mark.parametrize("pad", [0, 1, "odd", "packed"])
@pytest.mark.parametrize("table_type,type_", [(BF16, BF16), (F32, BF16), (F32, F16), (F16, F32),
                                              (F32, F32), (BF16, F16)])
def test_lookup(table_type, type_, pad):
    """One product in binary32 (E of it), rounded once."""
    for n, vocab, d, scale, wide in ((1, 1, 1, 1.0, True), (7, 50, 3, 22.6, False),
                                     (300, 1000, 64, 8.0, True), (1029, 333, 1001, 0.37, False),
                                     (5, 9, 4100, 1.0, True)):
        gen = generator(n)
        table = normal(gen, vocab, d, table_type, pad=pad)
        out, st = buffer(n, d, type_, pad), status_word()
        tok = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
        dgc.dgc_embed(table, tok if wide else tok.int(), scale, out, st)
        scale = torch.tensor(scale, dtype=F32).double().item()
        want = table.double()[tok] * scale
        near(out, want, E * want.abs())
        outside_is_untouched(out)
        assert dgc.dgc_read_status(st) == 0


def test_lookup_of_unknown_words():
    """Their rows are zeros whatever the scale, and the status says so."""
    table = normal(generator(1), 10, 24, BF16)
    tok = torch.tensor([3, -1, 9, 10, 2**40, -2**63, 0], device="cuda")
    out, st = buffer(7, 24, BF16), status_word()
    dgc.dgc_embed(table, tok, float("inf"), out, st)
    assert dgc.dgc_read_status(st) == dgc.EINVAL
    for i in (1, 3, 4, 5):
        assert (out[i] == 0).all()
    st.zero_()
    dgc.dgc_embed(table, tok, 1.0, out, st)
    assert torch.equal(out[[0, 2, 6]], table[[3, 9, 0]])
    empty = torch.zeros(0, 24, dtype=BF16, device="cuda")  # no vocabulary: every word is unknown
    st.zero_()
    dgc.dgc_embed(empty, tok, 1.0, out, st)
    assert dgc.dgc_read_status(st) == dgc.EINVAL and (out == 0).all()


def gradient(n, vocab, d, type_, kind="any", scale=1.0, accumulate=False, padding=None, wide=True,
             pad=0, table_pad=0, seed=0):
    gen = generator(seed + n)
    tok = tokens_of(kind, n, vocab, gen)
    dy = normal(gen, n, d, type_, pad=pad)
    dt = normal(gen, vocab, d, F32, pad=table_pad)
    was, st = dt.double(), status_word()
    ws = workspace(dgc.dgc_embed_backward_workspace(n, vocab, d))
    dgc.dgc_embed_backward(tok if wide else tok.int(), dy, scale, padding, dt, accumulate, st, ws)
    scale = torch.tensor(scale, dtype=F32).double().item()
    use = tok != (-1 if padding is None else padding)
    total, size = (torch.zeros(vocab, d, dtype=torch.float64, device="cuda").index_add_(
        0, tok[use], scale * v) for v in (dy.double()[use], dy.double()[use].abs()))
    met = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(
        0, tok[use], torch.ones(int(use.sum()), dtype=torch.float64, device="cuda"))
    # one rounding for each addition and the scale's product; the addition to what was there
    error = (met[:, None] + 2) * E * size
    want = total + was if accumulate else total
    near(dt, want, error + (E * was.abs() if accumulate else 0))
    if accumulate:  # words that are not met keep their bits
        assert torch.equal(dt[met == 0].double(), was[met == 0])
    else:
        assert (dt[met == 0] == 0).all()
    outside_is_untouched(dt)
    assert dgc.dgc_read_status(st) == 0
    return tok, dy, dt


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["any", "one", "head", "runs"])
def test_gradient(kind, type_, accumulate):
    for n, vocab, d, scale in ((1, 1, 1, 1.0), (2, 600, 5, 2.0), (31, 7, 64, 1.0),
                               (32, 511, 129, 1.0), (33, 512, 260, 0.5), (64, 3, 513, 11.3),
                               (65, 2, 1001, 1.0), (1000, 90, 72, 1.0), (4097, 300, 1030, 31.6)):
        gradient(n, vocab, d, type_, kind, scale, accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad,table_pad", [("odd", 0), (0, "odd"), ("odd", "odd"), (1, 2),
                                           ("packed", "packed")])
def test_gradient_strides(pad, table_pad, accumulate):
    for type_ in (F32, BF16):
        gradient(777, 130, 301, type_, "head", 1.0, accumulate, pad=pad, table_pad=table_pad)
        gradient(90, 41, 1, type_, "head", 1.0, accumulate, pad=pad, table_pad=table_pad)


@pytest.mark.parametrize("vocab", [510, 511, 512, 513, 262143, 262144, 300000])
def test_gradient_digits(vocab):
    """Vocabularies around one, two and three digits of the sort; several blocks of it."""
    gradient(9000, vocab, 16, BF16, "any", wide=False)
    gradient(9000, vocab, 16, BF16, "head", accumulate=True)
    gradient(70000, vocab, 8, F16, "head", padding=vocab - 1)


def test_gradient_padding_and_unknown_words():
    gradient(500, 40, 33, BF16, "head", padding=39)
    gradient(500, 40, 33, F32, "one", padding=20)            # nothing left
    gradient(500, 40, 33, F32, "one", padding=20, accumulate=True)
    gradient(500, 40, 33, F32, "any", padding=1000)          # no such word
    tok = torch.tensor([3, -1, 5, 6, 3, 2**35], device="cuda")
    dy, dt, st = normal(generator(2), 6, 9, F32), buffer(6, 9, F32), status_word()
    ws = workspace(dgc.dgc_embed_backward_workspace(6, 6, 9))
    dgc.dgc_embed_backward(tok, dy, 1.0, None, dt, False, st, ws)
    assert dgc.dgc_read_status(st) == dgc.EINVAL
    assert torch.equal(dt[3], dy[0] + dy[4]) and torch.equal(dt[5], dy[2])
    assert (dt[[0, 1, 2, 4]] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_padded_rows_reach_nothing(bad):
    n, vocab, d = 200, 30, 40
    tok = tokens_of("head", n, vocab, generator(3))
    dy, dt, st = normal(generator(4), n, d, BF16), buffer(vocab, d, F32), status_word()
    dy[tok == vocab - 1] = bad
    ws = workspace(dgc.dgc_embed_backward_workspace(n, vocab, d))
    dgc.dgc_embed_backward(tok, dy, 1.0, vocab - 1, dt, False, st, ws)
    assert torch.isfinite(dt).all() and dgc.dgc_read_status(st) == 0


def test_no_tokens():
    none, dy = torch.zeros(0, dtype=torch.int64, device="cuda"), buffer(0, 12, BF16)
    dt, st = buffer(50, 12, F32, fill=7.0), status_word()
    ws = workspace(dgc.dgc_embed_backward_workspace(0, 50, 12))
    dgc.dgc_embed_backward(none, dy, 1.0, None, dt, True, st, ws)
    assert (dt == 7).all()
    dgc.dgc_embed_backward(none, dy, 1.0, None, dt, False, st, ws)
    assert (dt == 0).all()
    dgc.dgc_embed(dt, none, 1.0, buffer(0, 12, F32), st)
    assert dgc.dgc_read_status(st) == 0


def test_gradient_is_deterministic_and_shares_its_workspace():
    """The same bits again, after the workspace served another problem."""
    n, vocab, d = 20000, 5000, 200
    gen = generator(5)
    tok, other = tokens_of("head", n, vocab, gen), tokens_of("one", n, vocab, gen)
    dy, st = normal(gen, n, d, BF16), status_word()
    ws = workspace(dgc.dgc_embed_backward_workspace(n, vocab, d))
    first, again, third = (buffer(vocab, d, F32) for _ in range(3))
    dgc.dgc_embed_backward(tok, dy, 1.0, None, first, False, st, ws)
    dgc.dgc_embed_backward(other, dy, 1.0, None, third, False, st, ws)
    dgc.dgc_embed_backward(tok, dy, 1.0, None, again, False, st, ws)
    assert torch.equal(bits(first), bits(again))
    assert dgc.dgc_read_status(st) == 0


def test_rows_past_two_to_the_32():
    """A table whose last rows lie behind 2^32 entries."""
    vocab, d = 530000, 8192
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    table = torch.zeros(vocab, d, dtype=BF16, device="cuda")
    tok = torch.tensor([vocab - 1, 0, vocab - 2], device="cuda")
    table[tok] = normal(generator(6), 3, d, BF16)
    out, st = buffer(3, d, BF16), status_word()
    dgc.dgc_embed(table, tok, 1.0, out, st)
    assert torch.equal(out, table[tok])
    dt = table.float()
    del table
    ws = workspace(dgc.dgc_embed_backward_workspace(3, vocab, d))
    dgc.dgc_embed_backward(tok, out, 1.0, None, dt, True, st, ws)
    assert torch.equal(dt[tok], out.float() * 2)
    assert dgc.dgc_read_status(st) == 0


def chunk_tokens(n, vocab, d):
    """How many sorted tokens a warp of the gradient sums, 8 or 32, read off the workspace's size: the
    sort's two lists and its counts, the list of chunks, two rows of sums for each."""
    def up(x):
        return -(-x // 256) * 256

    def size(tokens):
        chunks = -(-n // tokens)
        return (2 * up(8 * n) + up(256 * 512 * 4) + up(4 * (chunks + 1))
                + up(chunks * 2 * (-(-d // 4) * 4) * 4))

    found = [t for t in (8, 32) if size(t) == dgc.dgc_embed_backward_workspace(n, vocab, d)]
    assert len(found) == 1, (n, vocab, d)
    return found[0]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["any", "one", "head", "runs"])
def test_gradient_by_chunks_of_32(kind, type_, accumulate):
    """Sizes of which a warp sums 32 tokens: four columns a lane on and off 16-byte boundaries, eight
    of 16-bit entries."""
    for n, vocab, d, padding in ((8192, 200, 1280, None), (8190, 200, 1283, 199),
                                 (16384, 400, 2048, None), (16301, 5000, 2056, 4999)):
        assert chunk_tokens(n, vocab, d) == 32
        gradient(n, vocab, d, type_, kind, 1.5, accumulate, padding=padding)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad,table_pad", [("odd", 0), (0, "odd"), ("odd", "odd"),
                                           ("packed", "packed")])
def test_gradient_strides_by_chunks_of_32(pad, table_pad, accumulate):
    for type_ in (F32, F16, BF16):
        for kind in ("head", "runs"):
            gradient(8100, 210, 1301, type_, kind, 1.0, accumulate, pad=pad, table_pad=table_pad)


def whole_numbers(n, vocab, d, kind, type_, accumulate, padding=None):
    """Gradients of small whole numbers, whose sums are exact in any order: equal bit for bit."""
    gen = generator(n + vocab)
    tok = tokens_of(kind, n, vocab, gen)
    dy = torch.randint(-4, 5, (n, d), generator=gen, device="cuda").to(type_)
    dt = torch.randint(-9, 10, (vocab, d), generator=gen, device="cuda").float()
    use = tok != (-1 if padding is None else padding)
    want = (dt.double() if accumulate else torch.zeros(vocab, d, device="cuda").double())
    want.index_add_(0, tok[use], 2.0 * dy[use].double())
    assert want.abs().max() < 2**24
    st, ws = status_word(), workspace(dgc.dgc_embed_backward_workspace(n, vocab, d))
    dgc.dgc_embed_backward(tok, dy, 2.0, padding, dt, accumulate, st, ws)
    assert torch.equal(dt.double(), want)
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["any", "one", "head", "runs"])
@pytest.mark.parametrize("n,vocab,d", [(8192, 200, 1280), (8190, 200, 1283), (16384, 400, 2048),
                                       (5001, 300, 1001), (40000, 3000, 260)])
def test_whole_numbers_are_exact(n, vocab, d, kind, accumulate):
    """No row is left out or taken twice, however often its word is met."""
    for type_ in (F32, BF16):
        whole_numbers(n, vocab, d, kind, type_, accumulate, padding=vocab // 3)


@pytest.mark.parametrize("n", [2**20 + 1, 2**21 + 12345])
def test_a_sort_of_several_tiles_a_block(n):
    """More tokens than 256 blocks have in a tile of 4096 each: a block goes on with its digits'
    places from tile to tile."""
    for vocab, d, kind in ((300000, 3, "any"), (500, 4, "head"), (1 << 20, 1, "any")):
        whole_numbers(n, vocab, d, kind, BF16, False, padding=7)
        whole_numbers(n, vocab, d, kind, F32, True)
