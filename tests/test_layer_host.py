"""The operators around the feed-forward block on the host (no GPU): argument errors are returned
before any CUDA call, sizes of workspaces, and the Python binding's checks."""
import ctypes
import math

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

FAKE = 1 << 40  # aligned non-null address that is never dereferenced
BIG = 1 << 41


@pytest.fixture(scope="module")
def L():
    dgc.build()
    return dgc.lib()


def mat(rows, cols, ld=None, dtype=dgc.BF16, data=FAKE, reserved=0):
    return ctypes.byref(dgc.dgc_matrix(data, rows, cols, -(-cols // 8) * 8 if ld is None else ld,
                                       dtype, reserved))


def vec(n, dtype=dgc.F32, data=FAKE, reserved=0):
    return ctypes.byref(dgc.dgc_tensor(data, n, dtype, reserved))


M, D, V, Q = 200, 16, 30, 3
F32 = dict(dtype=dgc.F32)
# call: its arguments by name, in order; matrices as (rows, cols, type), vectors as (n, type)
CALLS = {
    "dgc_embed": dict(table=("m", V, D, dgc.BF16), tokens=("v", M, dgc.I64), scale=1.0,
                      out=("m", M, D, dgc.BF16), status=FAKE, stream=None),
    "dgc_embed_backward": dict(tokens=("v", M, dgc.I32), dy=("m", M, D, dgc.BF16), scale=1.0,
                               padding=-1, accumulate=0, dtable=("m", V, D, dgc.F32), status=FAKE,
                               ws=FAKE, ws_bytes=BIG, stream=None),
    "dgc_layer_norm": dict(x=("m", M, D, dgc.BF16), gamma=("v", D, dgc.F32),
                           beta=("v", D, dgc.F32), eps=1e-5, y=("m", M, D, dgc.BF16), mean=FAKE,
                           rstd=FAKE, stream=None),
    "dgc_layer_norm_backward": dict(dy=("m", M, D, dgc.BF16), x=("m", M, D, dgc.BF16),
                                    gamma=("v", D, dgc.F32), mean=FAKE, rstd=FAKE,
                                    residual=("m", M, D, dgc.BF16), dx=("m", M, D, dgc.BF16),
                                    dgamma=("v", D, dgc.F32), dbeta=("v", D, dgc.F32),
                                    accumulate=0, ws=FAKE, ws_bytes=BIG, stream=None),
    "dgc_dropout": dict(x=("m", M, D, dgc.BF16), residual=("m", M, D, dgc.BF16), p=0.5, seed=1,
                        step=FAKE, out=("m", M, D, dgc.BF16), stream=None),
    "dgc_recurrence": dict(x=("m", M, D, dgc.BF16), gate=("m", M, D, dgc.BF16), offsets=FAKE,
                           nseq=Q, h0=("m", Q, D, dgc.F32), y=("m", M, D, dgc.BF16),
                           h_last=("m", Q, D, dgc.F32), saved=("m", 4, D, dgc.F32), status=FAKE,
                           ws=FAKE, ws_bytes=BIG, stream=None),
    "dgc_recurrence_backward": dict(dy=("m", M, D, dgc.BF16), x=("m", M, D, dgc.BF16),
                                    gate=("m", M, D, dgc.BF16), offsets=FAKE, nseq=Q,
                                    h0=("m", Q, D, dgc.F32), saved=("m", 4, D, dgc.F32),
                                    d_last=("m", Q, D, dgc.F32), dx=("m", M, D, dgc.BF16),
                                    dgate=("m", M, D, dgc.BF16), d_h0=("m", Q, D, dgc.F32),
                                    status=FAKE, ws=FAKE, ws_bytes=BIG, stream=None),
    "dgc_selftest_recurrence_timeout": dict(x=("m", M, D, dgc.BF16), gate=("m", M, D, dgc.BF16),
                                            offsets=FAKE, nseq=Q, y=("m", M, D, dgc.BF16),
                                            status=FAKE, ws=FAKE, ws_bytes=BIG, spins=100,
                                            stream=None),
}
OPTIONAL = {"dgc_layer_norm": {"beta"}, "dgc_dropout": {"residual", "step"},
            "dgc_layer_norm_backward": {"residual", "dgamma", "dbeta"},
            "dgc_recurrence": {"h0", "h_last", "saved"},
            "dgc_recurrence_backward": {"h0", "d_last", "d_h0"}}
OWN_TYPE = {("dgc_embed", "table"), ("dgc_embed", "out"), ("dgc_embed_backward", "dy")}


def call(L, name, **change):
    args = []
    for k, v in CALLS[name].items():
        v = change.get(k, v)
        if isinstance(v, tuple):
            v = mat(v[1], v[2], dtype=v[3]) if v[0] == "m" else vec(v[1], v[2])
        args.append(v)
    return getattr(L, name)(*args)


@pytest.mark.parametrize("name", CALLS)
def test_every_matrix_is_checked(L, name):
    for k, v in CALLS[name].items():
        if not isinstance(v, tuple) or v[0] != "m":
            continue
        _, r, c, t = v
        bad = [mat(-1, c, dtype=t), mat(r, -1, dtype=t), mat(r, c, c - 1, dtype=t),
               mat(r, c, data=None, dtype=t), mat(r, c, data=FAKE + 1, dtype=t),
               mat(r, c, dtype=7), mat(r, c, dtype=dgc.I32), mat(r, c, dtype=t, reserved=1),
               mat(r, c + 1, dtype=t)]
        if (name, k) != ("dgc_embed", "table") and k != "dtable":
            bad.append(mat(r + 1, c, dtype=t))
        if (name, k) not in OWN_TYPE:
            bad.append(mat(r, c, dtype=dgc.F16))
        for b in bad:
            assert call(L, name, **{k: b}) == dgc.EINVAL, (k, b._obj.rows, b._obj.cols)
        assert call(L, name, **{k: mat(2**24 + 1, c, dtype=t)}) == dgc.EUNSUPPORTED, k
        assert call(L, name, **{k: mat(r, 2**24 + 8, dtype=t)}) == dgc.EUNSUPPORTED, k
        assert call(L, name, **{k: mat(r, c, 2**37, dtype=t)}) == dgc.EUNSUPPORTED, k


@pytest.mark.parametrize("name", CALLS)
def test_every_vector_and_address_is_checked(L, name):
    for k, v in CALLS[name].items():
        if isinstance(v, tuple) and v[0] == "v":
            _, n, t = v
            for b in (vec(n + 1, t), vec(n - 1, t), vec(-1, t), vec(n, dgc.BF16), vec(n, 9),
                      vec(n, t, data=None), vec(n, t, data=FAKE + 2), vec(n, t, reserved=1)):
                assert call(L, name, **{k: b}) == dgc.EINVAL, k
        if isinstance(v, tuple) or v == FAKE:
            if k not in OPTIONAL.get(name, ()):
                assert call(L, name, **{k: None}) == dgc.EINVAL, k
    if name in ("dgc_embed", "dgc_embed_backward"):
        t = CALLS[name]["tokens"][2]
        assert call(L, name, tokens=vec(2**24 + 1, t)) == dgc.EUNSUPPORTED


def test_settings(L):
    for p in (-0.1, 1.1, math.nan, math.inf):
        assert call(L, "dgc_dropout", p=p) == dgc.EINVAL
    assert call(L, "dgc_dropout", step=FAKE + 4) == dgc.EINVAL
    for eps in (0.0, -1e-5, math.nan, math.inf):
        assert call(L, "dgc_layer_norm", eps=eps) == dgc.EINVAL
    assert call(L, "dgc_layer_norm", mean=None) == dgc.EINVAL
    assert call(L, "dgc_layer_norm", rstd=FAKE + 2) == dgc.EINVAL
    assert call(L, "dgc_layer_norm_backward", mean=FAKE + 1) == dgc.EINVAL
    assert call(L, "dgc_embed_backward", padding=-2) == dgc.EINVAL
    for name in ("dgc_recurrence", "dgc_recurrence_backward"):
        assert call(L, name, nseq=-1) == dgc.EINVAL
        assert call(L, name, nseq=Q + 1) == dgc.EINVAL
        assert call(L, name, nseq=2**24 + 1) == dgc.EUNSUPPORTED
        assert call(L, name, offsets=FAKE + 4) == dgc.EINVAL
    for spins in (0, 2**31):
        assert call(L, "dgc_selftest_recurrence_timeout", spins=spins) == dgc.EINVAL


SIZED = {"dgc_embed_backward": lambda: dgc.dgc_embed_backward_workspace(M, V, D),
         "dgc_layer_norm_backward": lambda: dgc.dgc_layer_norm_backward_workspace(M, D),
         "dgc_recurrence": lambda: dgc.dgc_recurrence_workspace(M, D),
         "dgc_recurrence_backward": lambda: dgc.dgc_recurrence_workspace(M, D)}


@pytest.mark.parametrize("name", SIZED)
def test_workspaces(L, name):
    need = SIZED[name]()
    assert need > 0
    assert call(L, name, ws_bytes=need - 1) == dgc.EINVAL
    assert call(L, name, ws=FAKE + 16) == dgc.EINVAL
    assert call(L, name, ws=None) == dgc.EINVAL


def test_size_queries(L):
    out, n = ctypes.c_size_t(0), ctypes.c_int64(0)
    for q, k in ((L.dgc_embed_backward_workspace, 3), (L.dgc_layer_norm_backward_workspace, 2),
                 (L.dgc_recurrence_workspace, 2)):
        for i in range(k):
            sizes = [8] * k
            sizes[i] = -1
            assert q(*sizes, ctypes.byref(out)) == dgc.EINVAL
            sizes[i] = 2**24 + 1
            assert q(*sizes, ctypes.byref(out)) == dgc.EUNSUPPORTED
        assert q(*[8] * k, None) == dgc.EINVAL
        assert q(*[0] * k, ctypes.byref(out)) == 0
        assert q(*[2**24] * k, ctypes.byref(out)) == 0 and out.value > 2**32
    assert L.dgc_recurrence_saved_rows(-1, ctypes.byref(n)) == dgc.EINVAL
    assert L.dgc_recurrence_saved_rows(4, None) == dgc.EINVAL
    assert L.dgc_recurrence_saved_rows(2**24 + 1, ctypes.byref(n)) == dgc.EUNSUPPORTED
    assert [dgc.dgc_recurrence_saved_rows(r) for r in (0, 1, 64, 65)] == [0, 1, 1, 2]
    assert dgc.dgc_recurrence_workspace(64, 1000) == 0


def test_nothing_to_do_makes_no_cuda_call(L):
    none = dict(data=None)
    assert L.dgc_embed(mat(V, D), vec(0, dgc.I64, None), 1.0, mat(0, D, **none), FAKE, None) == 0
    assert L.dgc_embed(mat(V, 0, **none), vec(M, dgc.I64), 1.0, mat(M, 0, **none), FAKE, None) == 0
    ws = dgc.dgc_embed_backward_workspace(0, V, D)
    assert L.dgc_embed_backward(vec(0, dgc.I32, None), mat(0, D, **none), 1.0, -1, 1,
                                mat(V, D, **F32), FAKE, FAKE, ws, None) == 0
    assert L.dgc_layer_norm(mat(0, D, **none), vec(D), None, 1e-5, mat(0, D, **none), None, None,
                            None) == 0
    assert L.dgc_layer_norm_backward(mat(0, D, **none), mat(0, D, **none), vec(D), None, None, None,
                                     mat(0, D, **none), vec(D), None, 1, FAKE, BIG, None) == 0
    assert L.dgc_dropout(mat(M, 0, **none), None, 0.5, 0, None, mat(M, 0, **none), None) == 0
    assert L.dgc_recurrence(mat(9, 0, **none), mat(9, 0, **none), FAKE, 1, None, mat(9, 0, **none),
                            None, None, FAKE, None, 0, None) == 0


def refused(call, *args, **kw):
    with pytest.raises(dgc.DGCError) as e:
        call(*args, stream=0, **kw)
    assert e.value.code == dgc.EINVAL
    return str(e.value)


def python_args(name):
    args = {}
    for k, v in CALLS[name].items():
        if k in ("stream", "ws_bytes", "nseq"):
            continue
        if isinstance(v, tuple) and v[0] == "m":
            v = dgc.dgc_matrix(FAKE, v[1], v[2], -(-v[2] // 8) * 8, v[3], 0)
        elif isinstance(v, tuple):
            v = dgc.dgc_tensor(FAKE, v[1], v[2], 0)
        args[k] = None if k == "padding" else v
    return args


def host_tensor(v):
    if not isinstance(v, tuple):
        return torch.zeros(256, dtype=torch.uint8)
    types = {dgc.F32: torch.float32, dgc.BF16: torch.bfloat16, dgc.I32: torch.int32,
             dgc.I64: torch.int64}
    return torch.zeros(v[1:-1], dtype=types[v[-1]])


@pytest.mark.parametrize("view", [False, True])
@pytest.mark.parametrize("name", [n for n in CALLS if "selftest" not in n])
def test_host_tensors_are_refused(L, name, view):
    sized = dict(ws_bytes=BIG) if "ws" in CALLS[name] else {}
    if "offsets" in CALLS[name]:
        sized["nseq"] = Q
    for k, v in CALLS[name].items():
        if not (isinstance(v, tuple) or v == FAKE):
            continue
        args = python_args(name)
        t = host_tensor(v)
        if k in ("mean", "rstd"):
            t = torch.zeros(M)
        elif k in ("offsets", "step"):
            t = torch.zeros(Q + 1, dtype=torch.int64)
        elif view and isinstance(v, tuple):
            t = (dgc.matrix if v[0] == "m" else dgc.vector)(t)
        args[k] = t
        assert "host tensor" in refused(getattr(dgc, name), **args, **sized), k


def test_binding_checks(L):
    for bad in (torch.zeros(4, 6)[:, :3], torch.zeros(4, dtype=torch.float64),
                torch.zeros(4, dtype=torch.int16)):
        with pytest.raises(dgc.DGCError):
            dgc.vector(bad)
    v = dgc.vector(torch.zeros(4, 6, dtype=torch.int64))
    assert (v.n, v.dtype) == (24, dgc.I64)
    assert dgc.vector(torch.zeros(3, dtype=torch.int32)).dtype == dgc.I32
    for k, t in (("mean", torch.zeros(M - 1)), ("mean", torch.zeros(M, dtype=torch.float64)),
                 ("rstd", torch.zeros(2 * M)[::2])):
        args = python_args("dgc_layer_norm")
        args[k] = t
        refused(dgc.dgc_layer_norm, **args)
    args = python_args("dgc_recurrence")
    args["offsets"] = torch.zeros(Q + 1, dtype=torch.int32)
    refused(dgc.dgc_recurrence, **args, ws_bytes=BIG)
    args = python_args("dgc_embed_backward")
    args["padding"] = -1
    refused(dgc.dgc_embed_backward, **args, ws_bytes=BIG)
    args = python_args("dgc_dropout")
    args["step"] = torch.zeros(1)
    refused(dgc.dgc_dropout, **args)


def test_types_that_another_thread_is_loading(L, monkeypatch):
    """A call while another thread's first call has stored some of torch's types and not all."""
    args = python_args("dgc_dropout")
    args["step"] = torch.zeros(1, dtype=torch.int64)
    monkeypatch.setattr(dgc, "_float32", torch.float32)
    monkeypatch.setattr(dgc, "_words", ())
    assert "host tensor" in refused(dgc.dgc_dropout, **args)


def test_backward_selftest_is_checked(L):
    """Its limit, its workspace and its matrices, as the call it tests."""
    m = ("dy", "x", "gate", "dx", "dgate")

    def timeout(spins=100, ws=FAKE, ws_bytes=BIG, status=FAKE, nseq=Q, **change):
        a = {k: mat(M, D) for k in m}
        a["saved"] = mat(4, D, **F32)
        a.update(change)
        return L.dgc_selftest_recurrence_backward_timeout(
            a["dy"], a["x"], a["gate"], FAKE, nseq, a["saved"], a["dx"], a["dgate"], status, ws,
            ws_bytes, spins, None)

    for spins in (0, 2**31):
        assert timeout(spins=spins) == dgc.EINVAL
    for k in m:
        for b in (None, mat(M, D + 1), mat(M, D, data=None), mat(M, D, dtype=dgc.F16)):
            assert timeout(**{k: b}) == dgc.EINVAL
    for b in (None, mat(3, D, **F32), mat(4, D)):
        assert timeout(saved=b) == dgc.EINVAL
    need = dgc.dgc_recurrence_workspace(M, D)
    for change in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=FAKE + 16), dict(status=None),
                   dict(nseq=-1)):
        assert timeout(**change) == dgc.EINVAL
