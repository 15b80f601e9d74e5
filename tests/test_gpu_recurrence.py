"""The gated linear recurrence and its backward pass on the GPU against the definition, row by row in
64 bits (the bounds are derived with it, in layer_helpers)."""
import numpy as np
import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc
from layer_helpers import (BF16, E, F16, F32, bits, buffer, generator, near, normal,
                           outside_is_untouched, scan64, scan64_backward, status_word, workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def numpy64(t):
    return None if t is None else t.double().cpu().numpy()


def inside(rows, ends):
    m = torch.zeros(rows, dtype=torch.bool)
    m[ends[0]:ends[-1]] = True
    return m


def run(rows, cols, ends, type_, state=True, pad=0, gate_mean=1.5, gate_sigma=2.0, alias=False,
        outside=float("nan"), backward=True, seed=0, state_pad="packed"):
    """Forward and backward; the rows of no sequence hold `outside` in every operand."""
    gen = generator(seed + rows + cols)
    n = len(ends) - 1
    x, dy = normal(gen, rows, cols, type_, pad=pad), normal(gen, rows, cols, type_, 0.5, pad=pad)
    gate = normal(gen, rows, cols, type_, gate_sigma, gate_mean, pad)
    ok = inside(rows, ends)
    for t in (x, gate, dy):
        t[~ok.cuda()] = outside
    h0, d_last = (normal(gen, n, cols, F32, pad=state_pad) if state else None for _ in range(2))
    off = torch.tensor(ends, dtype=torch.int64, device="cuda")
    X, G, DY, H0, DL = (numpy64(t) for t in (x, gate, dy, h0, d_last))
    y = buffer(rows, cols, type_, pad)
    h_last = buffer(n, cols, F32, state_pad)
    saved = torch.full((dgc.dgc_recurrence_saved_rows(rows), cols), float("nan"), device="cuda")
    st, ws = status_word(), workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, h0, y, h_last, saved, st, ws)
    h, _, err, last, last_err = scan64(X, G, ends, H0)
    T = torch.from_numpy
    near(y.cpu()[ok], T(h)[ok], T(err)[ok])
    assert torch.isnan(y.cpu()[~ok]).all()  # the buffer's fill
    near(h_last.cpu(), T(last), T(last_err))
    outside_is_untouched(y)
    outside_is_untouched(h_last)
    if backward:
        if alias:
            dx, dgate, d_h0 = dy, gate, d_last
        else:
            dx, dgate = buffer(rows, cols, type_, pad), buffer(rows, cols, type_, pad)
            d_h0 = buffer(n, cols, F32, state_pad) if state else None
        dgc.dgc_recurrence_backward(dy, x, gate, off, h0, saved, d_last, dx, dgate, d_h0, st, ws)
        (wx, ex), (wg, eg), (wh, eh) = scan64_backward(X, G, ends, H0, DY, DL)
        near(dx.cpu()[ok], T(wx)[ok], T(ex)[ok])
        near(dgate.cpu()[ok], T(wg)[ok], T(eg)[ok])
        if state:
            near(d_h0.cpu(), T(wh), T(eh))
        if not alias:
            assert torch.isnan(dx.cpu()[~ok]).all() and torch.isnan(dgate.cpu()[~ok]).all()
            outside_is_untouched(dx)
            outside_is_untouched(dgate)
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_one_sequence(rows, type_):
    for cols in (1, 2, 64, 67):
        run(rows, cols, [0, rows], type_)
    run(rows, 130, [0, rows], type_, state=False)


@pytest.mark.parametrize("type_", [F32, BF16])
def test_long_sequences(type_):
    """Several groups of chunks in both directions."""
    run(4229, 66, [0, 4229], type_, gate_mean=5.0)
    run(9000, 3, [0, 9000], type_, gate_mean=8.0, gate_sigma=0.5)
    run(8192, 65, [0, 100, 4096, 4097, 8192], type_)
    run(6000, 2, [17, 17, 5000, 5000, 5990], type_, gate_mean=4.0)


TABLES = [
    [0, 64], [0, 1, 2, 3], [0, 0, 0, 5], [0, 5, 5, 5], [3, 3], [3, 9], [0, 63, 64, 65, 130],
    [0, 128, 256], [1, 127, 129, 255, 256], [0, 127, 128, 129], [5, 64, 128, 190, 192, 192, 300],
    list(range(0, 200)), list(range(0, 400, 2)), [0] * 70 + [40] * 70 + [90] * 40 + [91],
]


@pytest.mark.parametrize("type_", [F32, BF16])
@pytest.mark.parametrize("i", range(len(TABLES)))
def test_packed_sequences(i, type_):
    ends = TABLES[i]
    for rows in (ends[-1], ends[-1] + 1, ends[-1] + 77):
        run(rows, 70, ends, type_, seed=i)
        run(rows, 5, ends, type_, seed=i, state=False, outside=float("inf"))


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("pad", [1, "odd", "packed"])
@pytest.mark.parametrize("type_", [F32, F16, BF16])
def test_strides(type_, pad, alias):
    for cols in (1, 31, 65, 100):
        run(150, cols, [2, 70, 70, 150], type_, pad=pad, alias=alias, state_pad=pad)


@pytest.mark.parametrize("type_", [F32, F16, BF16])
def test_gates_at_their_ends(type_):
    """Gates of +-30, +-100 and the infinities: open, closed, and nothing in between is lost."""
    rows, cols = 90, 8
    gen = generator(3)
    x, dy = normal(gen, rows, cols, type_), normal(gen, rows, cols, type_)
    gate = buffer(rows, cols, type_, fill=0.0)
    ends = [0, 40, rows]
    values = [30.0, -30.0, 100.0, -100.0, float("inf"), -float("inf"), 0.0, 88.0]
    for c, v in enumerate(values):
        gate[:, c] = v
    gate[20], gate[60] = -float("inf"), float("inf")
    h0, d_last = normal(gen, 2, cols, F32), normal(gen, 2, cols, F32)
    off = torch.tensor(ends, device="cuda")
    y, dx, dgate = (buffer(rows, cols, type_) for _ in range(3))
    h_last, d_h0 = buffer(2, cols, F32), buffer(2, cols, F32)
    saved, st = torch.empty(2, cols, device="cuda"), status_word()
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, h0, y, h_last, saved, st, ws)
    dgc.dgc_recurrence_backward(dy, x, gate, off, h0, saved, d_last, dx, dgate, d_h0, st, ws)
    args = [numpy64(t) for t in (x, gate)] + [ends, numpy64(h0)]
    h, _, err, last, last_err = scan64(*args)
    (wx, ex), (wg, eg), (wh, eh) = scan64_backward(*args, numpy64(dy), numpy64(d_last))
    T = torch.from_numpy
    near(y.cpu(), T(h), T(err))
    near(h_last.cpu(), T(last), T(last_err))
    # factors below 2^-126 are zero here: 1e-37 of the terms, whose magnitudes are below 1000
    near(dx.cpu(), T(wx), T(ex) + 1e-34)
    near(dgate.cpu(), T(wg), T(eg) + 1e-34)
    near(d_h0.cpu(), T(wh), T(eh) + 1e-34)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_sequence(bad):
    rows, cols, ends = 700, 66, [0, 300, 301, 500, 700]
    gen = generator(8)
    x, gate, dy = (normal(gen, rows, cols, BF16) for _ in range(3))
    x[120, 7], dy[420, 9] = bad, bad
    off, st = torch.tensor(ends, device="cuda"), status_word()
    y, dx, dgate = (buffer(rows, cols, BF16) for _ in range(3))
    h_last, d_h0 = buffer(4, cols, F32), buffer(4, cols, F32)
    h0 = normal(gen, 4, cols, F32)
    h0[2, 11] = bad
    saved = torch.empty(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, h0, y, h_last, saved, st, ws)
    dgc.dgc_recurrence_backward(dy, x, gate, off, h0, saved, None, dx, dgate, d_h0, st, ws)
    good = torch.ones(rows, cols, dtype=torch.bool, device="cuda")
    good[120:300, 7] = False
    good[301:500, 11] = False
    assert torch.isfinite(y[good]).all() and not torch.isfinite(y[~good]).any()
    back = torch.ones_like(good)
    back[301:421, 9] = False
    assert torch.isfinite(dx[back]).all() and not torch.isfinite(dx[~back]).any()
    back[120:300, 7] = False
    back[301:500, 11] = False
    assert torch.isfinite(dgate[back]).all()
    assert dgc.dgc_read_status(st) == 0


def test_steps_of_a_model_that_answers():
    """One row a sequence, state in place, against the whole sequences at once: each step's state
    passes on in binary32."""
    n, cols, steps = 9, 200, 40
    gen = generator(5)
    x, gate = normal(gen, n * steps, cols, BF16), normal(gen, n * steps, cols, BF16)
    off = torch.arange(0, n * steps + 1, steps, device="cuda")
    y, h_last, st = buffer(n * steps, cols, BF16), buffer(n, cols, F32), status_word()
    ws = workspace(dgc.dgc_recurrence_workspace(n * steps, cols))
    dgc.dgc_recurrence(x, gate, off, None, y, h_last, None, st, ws)
    state, out = torch.zeros(n, cols, device="cuda"), buffer(n, cols, BF16)
    one = torch.arange(n + 1, device="cuda")
    X, G = x.view(n, steps, cols), gate.view(n, steps, cols)
    ends = [steps * i for i in range(n + 1)]
    h, _, err, last, last_err = scan64(numpy64(x), numpy64(gate), ends, None)
    ws1 = workspace(dgc.dgc_recurrence_workspace(n, cols))
    for t in range(steps):
        dgc.dgc_recurrence(X[:, t], G[:, t], one, state, out, state, None, st, ws1)
        near(out.cpu(), torch.from_numpy(h.reshape(n, steps, cols)[:, t]),
             torch.from_numpy(err.reshape(n, steps, cols)[:, t]))
    near(state.cpu(), torch.from_numpy(last), torch.from_numpy(last_err))
    assert dgc.dgc_read_status(st) == 0


def test_in_place_over_many_rows():
    rows, cols, ends = 5000, 70, [0, 900, 900, 4999]
    gen = generator(6)
    x, gate, h0 = normal(gen, rows, cols, BF16), normal(gen, rows, cols, BF16), normal(gen, 3, cols,
                                                                                       F32)
    off, st = torch.tensor(ends, device="cuda"), status_word()
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    y, last = buffer(rows, cols, BF16), buffer(3, cols, F32)
    dgc.dgc_recurrence(x, gate, off, h0, y, last, None, st, ws)
    for out in ("x", "gate"):
        a, b, h = x.clone(), gate.clone(), h0.clone()
        dgc.dgc_recurrence(a, b, off, h, a if out == "x" else b, h, None, st, ws)
        assert torch.equal(bits((a if out == "x" else b)[:4999]), bits(y[:4999].contiguous()))
        assert torch.equal((a if out == "x" else b)[4999], (x if out == "x" else gate)[4999])
        assert torch.equal(h, last)
    assert dgc.dgc_read_status(st) == 0


def test_deterministic_and_shares_its_workspace():
    rows, cols = 20000, 130
    gen = generator(7)
    x, gate, dy = (normal(gen, rows, cols, BF16, mean=m) for m in (0.0, 4.0, 0.0))
    off, st = torch.tensor([0, rows], device="cuda"), status_word()
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    saved = torch.empty(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
    runs = []
    for _ in range(4):
        y, dx, dgate = (buffer(rows, cols, BF16, "packed") for _ in range(3))
        dgc.dgc_recurrence(x, gate, off, None, y, None, saved, st, ws)
        dgc.dgc_recurrence_backward(dy, x, gate, off, None, saved, None, dx, dgate, None, st, ws)
        runs.append((y, dx, dgate))
    for r in runs[1:]:
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(runs[0], r))
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("ends", [[-1, 5], [0, 6, 5], [0, 201], [0, 2**40], [-2**63, 200],
                                  [200, 0], [0, 500, 3, 200]])
@pytest.mark.parametrize("rows", [200])
def test_bad_tables_are_reported(rows, ends):
    x, gate = (normal(generator(1), rows, 70, BF16) for _ in range(2))
    y, st = buffer(rows, 70, BF16), status_word()
    n = len(ends) - 1
    h0, saved = torch.zeros(n, 70, device="cuda"), torch.zeros(4, 70, device="cuda")
    off = torch.tensor(ends, device="cuda")
    ws = workspace(dgc.dgc_recurrence_workspace(rows, 70))
    dgc.dgc_recurrence(x, gate, off, h0, y, h0, saved, st, ws)
    assert dgc.dgc_read_status(st) == dgc.EINVAL
    st.zero_()
    dgc.dgc_recurrence_backward(x, x, gate, off, h0, saved, h0, y, y, h0, st, ws)
    assert dgc.dgc_read_status(st) == dgc.EINVAL


def test_nothing_to_scan():
    st = status_word()
    h0 = torch.ones(2, 9, device="cuda")
    last, d_h0 = torch.zeros_like(h0), torch.zeros_like(h0)
    none, off = buffer(0, 9, BF16), torch.zeros(3, dtype=torch.int64, device="cuda")
    saved = torch.empty(0, 9, device="cuda")
    dgc.dgc_recurrence(none, none, off, h0, none, last, saved, st, None)
    assert torch.equal(last, h0)
    dgc.dgc_recurrence_backward(none, none, none, off, h0, saved, h0, none, none, d_h0, st, None)
    assert torch.equal(d_h0, h0)
    x, y = normal(generator(1), 5, 9, BF16), buffer(5, 9, BF16)
    dgc.dgc_recurrence(x, x, off[:1], None, y, None, None, st, None)  # no sequence
    assert torch.isnan(y).all() and dgc.dgc_read_status(st) == 0


def test_gradient_against_differences():
    """Of sum(w y) + sum(c h_last) along a direction, by central differences of the definition in 64
    bits (the step's error: its square, 1e-8, times third derivatives of order one)."""
    rows, cols, ends = 150, 20, [0, 60, 60, 150]
    gen = generator(12)
    x, gate, w = (normal(gen, rows, cols, F32, pad="packed") for _ in range(3))
    h0, c = normal(gen, 3, cols, F32, pad="packed"), normal(gen, 3, cols, F32, pad="packed")
    vx, vg, vh = (numpy64(torch.randn(t.shape, generator=gen, device="cuda")) for t in (x, gate, h0))
    X, G, W, H, C = (numpy64(t) for t in (x, gate, w, h0, c))

    def loss(t):
        h, _, _, last, _ = scan64(X + t * vx, G + t * vg, ends, H + t * vh)
        return (h * W).sum() + (last * C).sum()

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    off, st = torch.tensor(ends, device="cuda"), status_word()
    y, dx, dgate, d_h0 = (torch.empty_like(t) for t in (x, x, x, h0))
    saved = torch.empty(3, cols, device="cuda")
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, h0, y, None, saved, st, ws)
    dgc.dgc_recurrence_backward(w, x, gate, off, h0, saved, c, dx, dgate, d_h0, st, ws)
    parts = [numpy64(a) * b for a, b in ((dx, vx), (dgate, vg), (d_h0, vh))]
    got, terms = sum(p.sum() for p in parts), sum(np.abs(p).sum() for p in parts)
    assert abs(got - slope) <= 1e-5 * terms
    assert dgc.dgc_read_status(st) == 0


def test_a_wait_that_runs_out():
    """The first chunk's map never arrives: the status says so, and the next call is right."""
    rows, cols = 700, 130
    gen = generator(13)
    x, gate = normal(gen, rows, cols, BF16), normal(gen, rows, cols, BF16)
    off, st, y = torch.tensor([0, rows], device="cuda"), status_word(), buffer(rows, cols, BF16)
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_selftest_recurrence_timeout(x, gate, off, y, st, ws, 2000)
    assert dgc.dgc_read_status(st) == dgc.ETIMEOUT
    run(rows, cols, [0, rows], BF16)


def test_captured_calls_on_their_own_streams():
    """Two graphs with their own workspaces, replayed on two streams at once, and the bits of plain
    calls."""
    rows, cols = 3000, 64
    sets = []
    for i in range(2):
        gen = generator(20 + i)
        x, gate, dy = (normal(gen, rows, cols, F16) for _ in range(3))
        off = torch.tensor([0, 1000 * (i + 1), rows], device="cuda")
        y, dx, dgate = (buffer(rows, cols, F16) for _ in range(3))
        saved = torch.empty(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
        st, ws = status_word(), workspace(dgc.dgc_recurrence_workspace(rows, cols))

        def step(x=x, gate=gate, dy=dy, off=off, y=y, dx=dx, dgate=dgate, saved=saved, st=st, ws=ws):
            dgc.dgc_recurrence(x, gate, off, None, y, None, saved, st, ws)
            dgc.dgc_recurrence_backward(dy, x, gate, off, None, saved, None, dx, dgate, None, st, ws)

        step()
        want = [t.clone() for t in (y, dx, dgate)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        sets.append((graph, (y, dx, dgate), want, torch.cuda.Stream(), st, step))  # step: its inputs
    for _ in range(3):
        for _, outs, *_ in sets:
            for t in outs:
                t.fill_(1.0)
        torch.cuda.synchronize()
        for graph, _, _, stream, *_ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _, st, _ in sets:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            assert dgc.dgc_read_status(st) == 0


def test_rows_past_two_to_the_32():
    """Long rows far apart: the last rows lie behind 2^32 entries."""
    rows, cols, ld = 400, 70, 1 << 24
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    flat = torch.empty(rows * ld, dtype=BF16, device="cuda")
    x = flat.view(rows, ld)[:, :cols]
    gate = flat.view(rows, ld)[:, 4096:4096 + cols]
    y = flat.view(rows, ld)[:, 8192:8192 + cols]
    gen = generator(30)
    x.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
    gate.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
    off, st = torch.tensor([0, rows], device="cuda"), status_word()
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, None, y, None, None, st, ws)
    h, _, err, _, _ = scan64(numpy64(x), numpy64(gate), [0, rows], None)
    near(y.cpu(), torch.from_numpy(h), torch.from_numpy(err))
    assert dgc.dgc_read_status(st) == 0 and E > 0


@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("nseq", [33, 300, 1023, 1024, 1100, 5000])
def test_many_sequences(nseq, type_):
    """Tables that are searched in one, two and three steps, most of whose sequences have no rows; over
    columns enough for groups of 16 chunks, and over a few."""
    ends = np.sort(np.random.default_rng(nseq).integers(3, 691, nseq + 1)).tolist()
    run(700, 520, ends, type_, seed=nseq)
    run(690, 6, ends, type_, seed=nseq, state=False)


@pytest.mark.parametrize("type_", [F32, BF16])
def test_empty_sequences_alone(type_):
    """No sequence has a row: states pass through, y, dx and dgate stay as they were."""
    run(300, 600, [7] * 3001, type_)
    run(300, 70, [300] * 40, type_)


@pytest.mark.parametrize("type_", [F32, BF16])
@pytest.mark.parametrize("rows", [0, 90, 400])
def test_slots_of_a_model_that_answers(rows, type_):
    """One token for some of 1024 slots, or none; the others keep their state, which may be kept where
    it is."""
    slots, cols = 1024, 130
    order = np.random.default_rng(rows).permutation(slots)[:rows]
    with_row = np.zeros(slots, dtype=np.int64)
    with_row[order] = 1
    ends = np.concatenate([[0], np.cumsum(with_row)]).tolist()
    if rows:
        run(rows, cols, ends, type_, seed=rows)
    gen = generator(rows)
    x, gate = normal(gen, rows, cols, type_), normal(gen, rows, cols, type_)
    h0 = normal(gen, slots, cols, F32)
    off = torch.tensor(ends, dtype=torch.int64, device="cuda")
    y, h_last = buffer(rows, cols, type_), buffer(slots, cols, F32)
    st, ws = status_word(), workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, h0, y, h_last, None, st, ws)
    empty = torch.from_numpy(with_row == 0).cuda()
    assert torch.equal(h_last[empty], h0[empty])
    again = buffer(rows, cols, type_)
    dgc.dgc_recurrence(x, gate, off, h0, again, h0, None, st, ws)
    assert torch.equal(h0, h_last) and torch.equal(bits(again), bits(y))
    assert dgc.dgc_read_status(st) == 0


def ragged(rows, n, seed):
    """n packed sequences of unequal length, one of them empty, over all rows."""
    cuts = np.sort(np.random.default_rng(seed).integers(1, rows, n - 2)).tolist()
    return [0] + cuts[:n // 2] + cuts[n // 2 - 1:n // 2] + cuts[n // 2:] + [rows]


# Tiles enough for a block to take several of them, chunks enough for several groups: of 16 chunks
# from 512 columns on, of 32 below (chunks have 128 rows forward in 16 bits, else 64).
@pytest.mark.parametrize("type_", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(5000, 1024), (9001, 576), (20000, 130)])
def test_several_groups_and_tiles(rows, cols, type_):
    # a memory of a thousand rows and more: the state goes through every group
    run(rows, cols, [0, rows], type_, gate_mean=8.0, gate_sigma=0.5)
    run(rows, cols, ragged(rows, 40, cols), type_, gate_mean=5.0, alias=True)
    run(rows, cols, [70, 900, 900, 2048, rows - 3], type_, state=False, gate_mean=6.0)


@pytest.mark.parametrize("pad", [1, "odd", "packed"])
@pytest.mark.parametrize("type_", [F32, BF16])
def test_several_groups_of_strided_rows(type_, pad):
    run(9001, 571, [0, 4000, 9001], type_, pad=pad, gate_mean=7.0, state_pad=pad)
    run(6000, 66, ragged(6000, 9, 1), type_, pad=pad, gate_mean=7.0, alias=True)


@pytest.mark.parametrize("type_", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(5000, 1024), (20000, 130)])
def test_in_place_over_several_groups(rows, cols, type_):
    """y on x or on gate, h_last on h0, over many tiles a block: the bits of results elsewhere."""
    gen = generator(rows)
    ends = ragged(rows, 30, 2)
    x, gate = normal(gen, rows, cols, type_), normal(gen, rows, cols, type_, mean=6.0)
    h0 = normal(gen, 30, cols, F32)
    off, st = torch.tensor(ends, device="cuda"), status_word()
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    y, last = buffer(rows, cols, type_), buffer(30, cols, F32)
    dgc.dgc_recurrence(x, gate, off, h0, y, last, None, st, ws)
    for out in (0, 1):
        a = [x.clone(), gate.clone()]
        h = h0.clone()
        dgc.dgc_recurrence(a[0], a[1], off, h, a[out], h, None, st, ws)
        assert torch.equal(bits(a[out]), bits(y.clone())) and torch.equal(h, last)
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("type_", [F32, BF16])
@pytest.mark.parametrize("place", ["ahead", "between", "behind"])
@pytest.mark.parametrize("rows,cols", [(40, 66), (100, 66), (300, 5), (700, 520)])
def test_idle_slots_at_one_place(rows, cols, place, type_):
    """A thousand and more sequences without rows that share an offset: ahead of the rows, at a border
    within a chunk, at a chunk's, and behind the rows."""
    for idle, at in ((1500, 33), (31, 17), (32, 16), (33, 64), (5000, 128)):
        at = {"ahead": 0, "between": min(at, rows - 1), "behind": rows}[place]
        tail = [rows] if at < rows else []
        head = list(range(0, at, 3))
        ends = head + [at] * (idle + 1) + tail
        run(rows, cols, ends, type_, seed=idle)


def test_idle_slots_at_one_place_are_passed_at_once():
    """A step for 100 of 2^20 slots, and a batch of 5000 rows in 100 of them, with the idle ones behind
    the others, or ten thousand between any two: below 3 ms each, both directions, where looking at
    them 32 at a time took 5 to 31 (the states' copies alone take some 0.1 to 1 ms)."""
    slots, busy, cols = 1 << 20, 100, 16
    h0, last = torch.zeros(slots, cols, device="cuda"), torch.zeros(slots, cols, device="cuda")
    st = status_word()
    for each in (1, 50):
        rows = busy * each
        gen = generator(each)
        x, gate, dy = (normal(gen, rows, cols, BF16) for _ in range(3))
        y, dx, dgate = (buffer(rows, cols, BF16) for _ in range(3))
        saved = torch.empty(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
        ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
        times = []
        for spread in (True, False):
            with_rows = torch.zeros(slots, dtype=torch.int64, device="cuda")
            with_rows[::slots // busy][:busy] = each
            if not spread:
                with_rows = with_rows.sort(descending=True).values
            off = torch.cat([with_rows.new_zeros(1), with_rows.cumsum(0)])
            assert off[-1] == rows
            for call in (lambda: dgc.dgc_recurrence(x, gate, off, h0, y, last, saved, st, ws),
                         lambda: dgc.dgc_recurrence_backward(dy, x, gate, off, h0, saved, h0, dx,
                                                             dgate, last, st, ws)):
                took = []
                for _ in range(5):
                    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                    a.record()
                    call()
                    b.record()
                    b.synchronize()
                    took.append(a.elapsed_time(b))
                times.append(min(took))
        assert dgc.dgc_read_status(st) == 0
        assert max(times) < 3.0, times


@pytest.mark.parametrize("cols", [130, 520])
def test_a_wait_of_the_backward_pass_that_runs_out(cols):
    """The last rows' map never arrives: the status says so, and the next call is right."""
    rows = 2500
    gen = generator(14)
    x, gate, dy = (normal(gen, rows, cols, BF16) for _ in range(3))
    off, st = torch.tensor([0, rows], device="cuda"), status_word()
    y, dx, dgate = (buffer(rows, cols, BF16) for _ in range(3))
    saved = torch.empty(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
    ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
    dgc.dgc_recurrence(x, gate, off, None, y, None, saved, st, ws)

    def backward():
        dgc.dgc_recurrence_backward(dy, x, gate, off, None, saved, None, dx, dgate, None, st, ws)
        assert dgc.dgc_read_status(st) == 0
        return bits(dx.contiguous()).clone(), bits(dgate.contiguous()).clone()

    want = backward()
    dgc.dgc_selftest_recurrence_backward_timeout(dy, x, gate, off, saved, dx, dgate, st, ws, 2000)
    assert dgc.dgc_read_status(st) == dgc.ETIMEOUT
    st.zero_()
    assert all(torch.equal(a, b) for a, b in zip(backward(), want))


@pytest.mark.parametrize("rows", [0, 1, 64, 65, 300])
def test_few_rows_of_many_sequences_backward(rows):
    """More blocks than tiles: the states' gradients of those without rows pass, the others' are the
    definition's."""
    n, cols = 3000, 130
    gen = generator(rows + 1)
    if rows:
        run(rows, cols, [0] * 1000 + list(range(rows)) + [rows] * (n - 999 - rows), F32)
    x, gate, dy = (normal(gen, rows, cols, BF16) for _ in range(3))
    ends = [0] * 2000 + [rows] * 1001
    h0, d_last = normal(gen, n, cols, F32), normal(gen, n, cols, F32)
    off, st = torch.tensor(ends, device="cuda"), status_word()
    y, dx, dgate = (buffer(rows, cols, BF16) for _ in range(3))
    saved = torch.empty(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
    ws, d_h0 = workspace(dgc.dgc_recurrence_workspace(rows, cols)), buffer(n, cols, F32)
    dgc.dgc_recurrence(x, gate, off, h0, y, None, saved, st, ws)
    dgc.dgc_recurrence_backward(dy, x, gate, off, h0, saved, d_last, dx, dgate, d_h0, st, ws)
    empty = torch.ones(n, dtype=torch.bool, device="cuda")
    empty[1999] = rows == 0
    assert torch.equal(d_h0[empty], d_last[empty])
    last = d_last.clone()  # in its place
    dgc.dgc_recurrence_backward(dy, x, gate, off, h0, saved, last, dx, dgate, last, st, ws)
    assert torch.equal(last, d_h0)
    assert dgc.dgc_read_status(st) == 0


@pytest.mark.parametrize("rows", [100, 700])
def test_bad_tables_of_many_sequences_are_reported(rows):
    """Offsets in no order, runs of equal ones among them; nothing outside the operands is written."""
    n, cols = 5000, 70
    for seed in range(4):
        rng = np.random.default_rng(seed)
        ends = rng.integers(-3, rows + 50, n + 1)
        ends[1000:2500] = rows // 2
        ends[3000:3100] = rng.integers(-2**62, 2**62, 100)
        x, gate = (normal(generator(seed), rows, cols, BF16) for _ in range(2))
        y, st = buffer(rows, cols, BF16), status_word()
        h0, last = torch.zeros(n, cols, device="cuda"), buffer(n, cols, F32)
        saved = torch.zeros(dgc.dgc_recurrence_saved_rows(rows), cols, device="cuda")
        off = torch.from_numpy(ends).cuda()
        ws = workspace(dgc.dgc_recurrence_workspace(rows, cols))
        dgc.dgc_recurrence(x, gate, off, h0, y, last, saved, st, ws)
        assert dgc.dgc_read_status(st) == dgc.EINVAL
        st.zero_()
        dgc.dgc_recurrence_backward(x, x, gate, off, h0, saved, h0, y, y, last, st, ws)
        assert dgc.dgc_read_status(st) == dgc.EINVAL
        for t in (y, last):
            t.fill_(float("nan"))
            outside_is_untouched(t)
