"""The feed-forward block's calls on the host (no GPU): argument errors are returned before any
CUDA call, and the Python binding's checks."""
import ctypes

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

FAKE = 1 << 40  # aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    dgc.build()
    return dgc.lib()


def mat(rows, cols, ld=None, dtype=dgc.BF16, data=FAKE, reserved=0):
    return ctypes.byref(dgc.dgc_matrix(data, rows, cols, -(-cols // 8) * 8 if ld is None else ld,
                                       dtype, reserved))


M, D, F = 6, 16, 24
SHAPES = {  # call: the shapes of its matrices in order, and whether it takes an activation
    "dgc_ffn_gate": ([(M, D), (F, D), (F, D), (M, F), (M, F), (M, F)], 3),
    "dgc_ffn_down": ([(M, F), (D, F), (M, D), (M, D)], None),
    "dgc_ffn_down_backward": ([(M, D), (D, F), (M, F), (M, F), (M, F), (M, F)], 4),
    "dgc_ffn_gate_backward": ([(M, F), (M, F), (F, D), (F, D), (M, D), (M, D)], None),
}


def call(L, name, change=None, act=0, status=FAKE):
    """The call with one matrix changed: change = (position, matrix)."""
    shapes, at = SHAPES[name]
    args = [mat(*s) for s in shapes]
    if change:
        args[change[0]] = change[1]
    if at is not None:
        args.insert(at, act)
    return getattr(L, name)(*args, status, None)


@pytest.mark.parametrize("name", SHAPES)
def test_every_matrix_is_checked(L, name):
    for i, (r, c) in enumerate(SHAPES[name][0]):
        for bad in (mat(r + 1, c), mat(r, c + 1), mat(-1, c), mat(r, -1), mat(r, c, c - 1),
                    mat(r, c, data=None), mat(r, c, data=FAKE + 1),
                    mat(r, c, dtype=dgc.F16), mat(r, c, dtype=dgc.F32), mat(r, c, dtype=7),
                    mat(r, c, reserved=1)):
            assert call(L, name, (i, bad)) == dgc.EINVAL, (i, bad._obj.rows, bad._obj.cols)
        assert call(L, name, (i, mat(2**24 + 1, c))) == dgc.EUNSUPPORTED
        assert call(L, name, (i, mat(r, 2**24 + 8))) == dgc.EUNSUPPORTED
    assert call(L, name, status=None) == dgc.EINVAL


@pytest.mark.parametrize("name,act", [(n, a) for n in SHAPES for a in (-1, 4)
                                      if SHAPES[n][1] is not None])
def test_unknown_activations(L, name, act):
    assert call(L, name, act=act) == dgc.EINVAL


@pytest.mark.parametrize("name,i", [(n, i) for n in SHAPES for i in range(len(SHAPES[n][0]))])
def test_missing_matrices(L, name, i):
    if (name, i) in (("dgc_ffn_down", 2), ("dgc_ffn_gate_backward", 4)):
        return  # the residual may be left out
    assert call(L, name, (i, None)) == dgc.EINVAL


def test_weight_grad(L):
    g = L.dgc_ffn_weight_grad
    T, R, C = 40, 16, 24

    def call(dy=mat(T, R), x=mat(T, C), dw=mat(R, C, C, dgc.F32), status=FAKE, ws=None, nws=0):
        return g(dy, x, 0, dw, status, ws, nws, None)

    for bad in (None, mat(T, R, dtype=dgc.F32), mat(T, R, data=FAKE + 1), mat(T, R, R - 1),
                mat(T + 1, R), mat(T, R + 8)):
        assert call(dy=bad) == dgc.EINVAL
    for bad in (None, mat(T, C, dtype=dgc.F16), mat(T + 1, C), mat(T, C + 8), mat(T, C, 8)):
        assert call(x=bad) == dgc.EINVAL
    f32 = dict(dtype=dgc.F32)
    for bad in (None, mat(R, C), mat(R, C, C - 1, **f32), mat(R, C, C, data=None, **f32),
                mat(R, C, C, data=FAKE + 2, **f32), mat(C, R, R, **f32), mat(-1, C, C, **f32),
                mat(R, C, C, reserved=2, **f32)):
        assert call(dw=bad) == dgc.EINVAL
    assert call(dw=mat(R, C, 2**37, **f32)) == dgc.EUNSUPPORTED
    assert call(status=None) == dgc.EINVAL
    # a sum that is split over the tokens needs its workspace, aligned
    T = 1 << 16
    need = dgc.dgc_ffn_weight_grad_workspace(R, C, T)
    assert need > 0 and dgc.dgc_ffn_weight_grad_workspace(R, C, 40) == 0
    big = dict(dy=mat(T, R), x=mat(T, C))
    assert call(**big, ws=FAKE, nws=need - 1) == dgc.EINVAL
    assert call(**big, ws=FAKE + 16, nws=need) == dgc.EINVAL
    assert call(**big, ws=None, nws=need) == dgc.EINVAL
    out = ctypes.c_size_t(0)
    q = L.dgc_ffn_weight_grad_workspace
    assert q(-1, 1, 1, ctypes.byref(out)) == dgc.EINVAL and q(1, 1, 1, None) == dgc.EINVAL
    assert q(2**24 + 1, 1, 1, ctypes.byref(out)) == dgc.EUNSUPPORTED


def test_nothing_to_do_makes_no_cuda_call(L):
    empty = dict(data=None)
    assert L.dgc_ffn_gate(mat(0, D, **empty), mat(F, D), mat(F, D), 0, mat(0, F, **empty), None,
                          None, FAKE, None) == 0
    assert L.dgc_ffn_down(mat(M, F), mat(0, F, **empty), None, mat(M, 0, **empty), FAKE,
                          None) == 0


def test_binding_checks():
    with pytest.raises(dgc.DGCError):
        dgc.matrix(torch.zeros(4, dtype=torch.bfloat16))
    with pytest.raises(dgc.DGCError):
        dgc.matrix(torch.zeros(4, 8, dtype=torch.bfloat16).t())
    with pytest.raises(dgc.DGCError):
        dgc.matrix(torch.zeros(4, 8, dtype=torch.int16))
    m = dgc.matrix(torch.zeros(4, 16, dtype=torch.float16)[:, :5])
    assert (m.rows, m.cols, m.ld, m.dtype) == (4, 5, 16, dgc.F16)


def test_selftest_rejects_on_host(L):
    t = L.dgc_selftest_ffn_timeout
    args = (mat(M, F), mat(D, F), mat(M, D))
    assert t(*args, FAKE, 0, None) == dgc.EINVAL and t(*args, FAKE, 1001, None) == dgc.EINVAL
    assert t(*args, None, 20, None) == dgc.EINVAL
    assert t(None, args[1], args[2], FAKE, 20, None) == dgc.EINVAL
