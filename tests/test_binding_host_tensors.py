"""Host tensors in the calls on gradient lists and feed-forward blocks (no GPU): refused by the
binding, before their addresses can reach a kernel."""
import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

FAKE = 1 << 40  # an address passed through as it is


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dgc.build()
    dgc.lib()


def refused(call, *args, **kw):
    with pytest.raises(dgc.DGCError, match="host tensor") as e:
        call(*args, stream=0, **kw)
    assert e.value.code == dgc.EINVAL


def mat(rows, cols, dtype=dgc.BF16):
    return dgc.dgc_matrix(FAKE, rows, cols, -(-cols // 8) * 8, dtype, 0)


M, D, F = 6, 16, 24
CALLS = {  # the shapes of the matrices in order, and where the activation goes
    "dgc_ffn_gate": ([(M, D), (F, D), (F, D), (M, F), (M, F), (M, F)], 3),
    "dgc_ffn_down": ([(M, F), (D, F), (M, D), (M, D)], None),
    "dgc_ffn_down_backward": ([(M, D), (D, F), (M, F), (M, F), (M, F), (M, F)], 4),
    "dgc_ffn_gate_backward": ([(M, F), (M, F), (F, D), (F, D), (M, D), (M, D)], None),
}


@pytest.mark.parametrize("view", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_matrices_and_status(name, view):
    shapes, at = CALLS[name]
    for i in range(len(shapes) + 1):  # the last one: the status word
        args = [mat(*s) for s in shapes] + [FAKE]
        if i < len(shapes):
            t = torch.zeros(shapes[i], dtype=torch.bfloat16)
            args[i] = dgc.matrix(t) if view else t
        else:
            args[i] = torch.zeros(1, dtype=torch.int32)
        if at is not None:
            args.insert(at, dgc.ACT_SILU)
        refused(getattr(dgc, name), *args)


def test_weight_grad_and_selftest():
    good = [mat(8, 16), mat(8, 24), mat(16, 24, dgc.F32)]
    bf16, i32 = torch.bfloat16, torch.int32
    for i, t in enumerate((torch.zeros(8, 16, dtype=bf16), torch.zeros(8, 24, dtype=bf16),
                           torch.zeros(16, 24))):
        args = good[:]
        args[i] = t
        refused(dgc.dgc_ffn_weight_grad, *args, False, FAKE, None)
    refused(dgc.dgc_ffn_weight_grad, *good, False, torch.zeros(1, dtype=i32), None)
    refused(dgc.dgc_ffn_weight_grad, *good, False, FAKE, torch.zeros(256, dtype=torch.uint8))
    refused(dgc.dgc_selftest_ffn_timeout, torch.zeros(4, 128, dtype=bf16), mat(8, 128), mat(4, 8),
            FAKE, 20)


def test_gradient_lists():
    host = dgc.TensorList([torch.zeros(0), torch.zeros(4)])
    none = dgc.TensorList([torch.zeros(0)])  # no entries: no address to read
    one = torch.zeros(1)
    refused(dgc.dgc_grad_norm, host, 1.0, FAKE, FAKE, FAKE, ws_bytes=1 << 20)
    refused(dgc.dgc_grad_clip, host, None, 1.0, FAKE, FAKE, FAKE, ws_bytes=1 << 20)
    refused(dgc.dgc_grad_clip, dgc.TensorList([torch.zeros(0)] * 2), host, 1.0, FAKE, FAKE, FAKE,
            ws_bytes=1 << 20)
    for i in range(3):
        args = [FAKE, FAKE, FAKE]
        args[i] = one if i < 2 else torch.zeros(1 << 20, dtype=torch.uint8)
        refused(dgc.dgc_grad_norm, none, 1.0, *args, ws_bytes=1 << 20)
        refused(dgc.dgc_grad_clip, none, None, 1.0, *args, ws_bytes=1 << 20)
    assert dgc.dgc_grad_workspace(host) > 0  # a size: no address is read
