"""dgc_grad_norm and dgc_grad_clip on the host (no GPU): argument errors are returned before any
CUDA call, and the Python binding's list checks."""
import ctypes
import math

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

FAKE = 1 << 40  # aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    dgc.build()
    return dgc.lib()


def tensors(*rows):
    a = (dgc.dgc_tensor * max(len(rows), 1))()
    for i, r in enumerate(rows):
        a[i] = dgc.dgc_tensor(*r)
    return ctypes.cast(a, ctypes.c_void_p)


def workspace(L, src, count):
    out = ctypes.c_size_t(0)
    rc = L.dgc_grad_workspace(src, count, ctypes.byref(out))
    return rc, out.value


GOOD = (FAKE, 100, 0, 0)


def test_workspace_grows_with_long_lists(L):
    rc, small = workspace(L, tensors(GOOD), 1)
    assert rc == 0 and small > 0
    rc, big = workspace(L, tensors(*[GOOD] * 5000), 5000)
    assert rc == 0 and big >= small + 5000 * 28
    assert workspace(L, None, 0) == (0, small)
    assert L.dgc_grad_workspace(None, 0, None) == dgc.EINVAL


@pytest.mark.parametrize("row,code", [
    ((FAKE, -1, 0, 0), dgc.EINVAL),
    ((FAKE, 8, 3, 0), dgc.EINVAL),
    ((FAKE, 8, -1, 0), dgc.EINVAL),
    ((FAKE, 8, 0, 1), dgc.EINVAL),
    ((None, 8, 0, 0), dgc.EINVAL),
    ((FAKE + 2, 8, 0, 0), dgc.EINVAL),
    ((FAKE + 1, 8, 1, 0), dgc.EINVAL),
    ((FAKE, 2**43, 0, 0), dgc.EUNSUPPORTED),
])
def test_lists_are_checked(L, row, code):
    assert workspace(L, tensors(GOOD, row), 2)[0] == code
    norm, clip = L.dgc_grad_norm, L.dgc_grad_clip
    bad, good = tensors(GOOD, row), tensors(GOOD, GOOD)
    assert norm(bad, 2, 1.0, FAKE, FAKE, FAKE, 1 << 30, None) == code
    assert clip(bad, None, 2, 1.0, FAKE, FAKE, FAKE, 1 << 30, None) == code
    if row[1] != 2**43:
        assert clip(good, bad, 2, 1.0, FAKE, FAKE, FAKE, 1 << 30, None) == code


def test_calls_reject_on_host(L):
    src = tensors(GOOD, (FAKE + 4096, 7, 2, 0))
    ws = workspace(L, src, 2)[1]
    n = L.dgc_grad_norm
    assert n(src, -1, 1.0, FAKE, FAKE, FAKE, ws, None) == dgc.EINVAL
    assert n(None, 2, 1.0, FAKE, FAKE, FAKE, ws, None) == dgc.EINVAL
    assert n(src, 2, math.nan, FAKE, FAKE, FAKE, ws, None) == dgc.EINVAL
    assert n(src, 2, 1.0, None, FAKE, FAKE, ws, None) == dgc.EINVAL
    assert n(src, 2, 1.0, FAKE, None, FAKE, ws, None) == dgc.EINVAL
    assert n(src, 2, 1.0, FAKE, FAKE, None, ws, None) == dgc.EINVAL
    assert n(src, 2, 1.0, FAKE, FAKE, FAKE + 16, ws, None) == dgc.EINVAL
    assert n(src, 2, 1.0, FAKE, FAKE, FAKE, ws - 1, None) == dgc.EINVAL
    assert n(src, (1 << 20) + 1, 1.0, FAKE, FAKE, FAKE, ws, None) == dgc.EUNSUPPORTED
    c = L.dgc_grad_clip
    short = tensors((FAKE + 8192, 99, 0, 0), (FAKE + 16384, 7, 0, 0))
    assert c(src, short, 2, 1.0, FAKE, FAKE, FAKE, ws, None) == dgc.EINVAL
    retyped = tensors(GOOD, (FAKE + 4096, 7, 1, 0))  # src's address with another type
    assert c(src, retyped, 2, 1.0, FAKE, FAKE, FAKE, ws, None) == dgc.EINVAL


def test_binding_checks_lists():
    with pytest.raises(dgc.DGCError):
        dgc.TensorList([torch.zeros(4, 6)[:, :3]])
    with pytest.raises(dgc.DGCError):
        dgc.TensorList([torch.zeros(4, dtype=torch.float64)])
    a = dgc.TensorList([torch.zeros(4), torch.zeros(0, dtype=torch.bfloat16)])
    assert len(a) == 2 and a.array[0].n == 4 and a.array[1].dtype == dgc.BF16
    with pytest.raises(dgc.DGCError):
        dgc.dgc_grad_clip(a, dgc.TensorList([torch.zeros(4)]), 1.0, None, None, None, ws_bytes=0,
                          stream=0)
