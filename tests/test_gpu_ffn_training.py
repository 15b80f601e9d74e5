"""The feed-forward training example on the GPU: its gradients against autograd, and its learning."""
import os
import sys

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def trainer(**kw):
    from ffn_training_step import FfnTrainer

    dgc.build()
    return FfnTrainer(**kw)


def test_gradients_of_a_step_against_autograd():
    """Two micro-batches' gradients in the bucket, and dx. Autograd runs in binary64 on the same
    bfloat16 weights; the block's saved and passed-on tensors are rounded to bfloat16, five
    roundings of at most 2^-9 root-mean-square along any path: 2% of the norm is beyond them."""
    t = trainer(dim=96, ffn=160, tokens=200)
    gen = torch.Generator(device="cuda").manual_seed(5)
    wg, wu, wd = (w.double().requires_grad_(True) for w in t.weights)
    for i in range(2):
        x = torch.randn(200, 96, generator=gen, device="cuda").bfloat16()
        dy = torch.randn(200, 96, generator=gen, device="cuda").bfloat16()
        t.forward(t.weights, x, t.y, True)
        t.backward(x, dy, i == 0)
        xd = x.double().requires_grad_(True)
        y = xd + (torch.nn.functional.silu(xd @ wg.t()) * (xd @ wu.t())) @ wd.t()
        (y * dy.double()).sum().backward()
        assert (t.y.double() - y).norm() < 0.02 * y.norm()
        assert (t.dx.double() - xd.grad).norm() < 0.02 * xd.grad.norm()
    for got, w in zip(t.grads, (wg, wu, wd)):
        assert (got.double() - w.grad).norm() < 0.02 * w.grad.norm()
    assert dgc.dgc_read_status(t.status) == 0


def test_learns_with_one_percent_of_the_gradient():
    t = trainer()
    losses = [t.step().item() for _ in range(60)]
    assert dgc.dgc_read_status(t.status) == 0
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5]), losses
    assert t.message_bytes.item() < 0.02 * 4 * t.bucket.numel()
