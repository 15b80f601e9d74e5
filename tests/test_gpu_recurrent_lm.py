"""The recurrent language model's example on the GPU: the operators together, as they are used. Its
gradients against autograd in 64 bits, a captured step, and two models on two streams at once."""
import os
import sys

import pytest
import torch

import sparsified_gradient_compression_gb300 as dgc
from layer_helpers import dropout_kept

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def model(**kw):
    from recurrent_lm_step import RecurrentLm

    dgc.build()
    return RecurrentLm(**kw)


def inputs(m):
    from recurrent_lm_step import batch

    return batch(m)


def reference(m, tokens, d_logits):
    """The model in 64 bits on its bfloat16 weights, with the masks that it draws; the gradients of
    sum(logits d_logits)."""
    w = {k: (m.copies.get(k, m.w[k])).double().requires_grad_(True) for k in m.w}
    keep = [dropout_kept(m.rows, m.dim, m.drop, 1000 * m.seed + i, int(m.counter)).cuda()
            for i in (1, 2)]
    share = (65536 - int(m.drop * 65536 + 0.5)) / 65536
    pad = 0

    def norm(x, i):
        return torch.nn.functional.layer_norm(x, x.shape[1:], w[f"g{i}"], w[f"b{i}"], 1e-5)

    e = torch.nn.functional.embedding(tokens, w["table"], padding_idx=pad) * m.scale
    n1 = norm(e, 1)
    x, a = n1 @ w["wx"].t(), torch.sigmoid(n1 @ w["wz"].t())
    ends, rows = m.offsets.tolist(), []
    for s, t in zip(ends, ends[1:]):
        h = torch.zeros(m.dim, dtype=torch.float64, device="cuda")
        for i in range(s, t):
            h = a[i] * h + (1 - a[i]) * x[i]
            rows.append(h)
    s1 = e + torch.where(keep[0], torch.stack(rows) @ w["wo"].t() / share, 0.0)
    n2 = norm(s1, 2)
    f = (torch.nn.functional.silu(n2 @ w["wg"].t()) * (n2 @ w["wu"].t())) @ w["wd"].t()
    s2 = s1 + torch.where(keep[1], f / share, 0.0)
    logits = norm(s2, 3) @ w["table"].t()
    (logits * d_logits.double()).sum().backward()
    return logits.detach(), {k: v.grad for k, v in w.items()}


def test_gradients_of_a_step_against_autograd():
    """Along any path some 20 tensors are rounded to bfloat16, each by 2^-9 root-mean-square or less,
    independently: 20^(1/2) 2^-9 = 0.9% of the norm; the norms' and the recurrence's slopes are of
    order one: 3% is beyond them."""
    m = model(vocab=96, dim=64, ffn=128, lengths=(40, 0, 1, 75))
    tokens, _ = inputs(m)
    m.counter += 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    m.forward(tokens)
    m.d_logits.copy_(torch.randn(m.rows, m.vocab, generator=gen, device="cuda"))
    m.bucket.fill_(float("nan"))  # every gradient is written
    m.backward(tokens)
    assert dgc.dgc_read_status(m.status) == 0
    logits, grads = reference(m, tokens, m.d_logits)
    assert (m.logits.double() - logits).norm() < 0.03 * logits.norm()
    for k, want in grads.items():
        assert (m.grad[k].double() - want).norm() < 0.03 * want.norm(), k


def test_a_step_runs():
    m = model()
    before = m.master.clone()
    loss = m.step(*inputs(m))
    assert dgc.dgc_read_status(m.status) == 0 and torch.isfinite(loss)
    assert torch.isfinite(m.master).all() and not torch.equal(m.master, before)
    assert 0 < m.message_bytes.item() < 0.02 * 4 * m.bucket.numel()


def forward_backward(m, tokens):
    m.forward(tokens)
    m.backward(tokens)
    m.counter += 1


def test_captured_steps_draw_their_own_masks():
    """Forward and backward passes in a graph, with the counter advanced in it: the bits of plain
    calls, replay by replay."""
    m = model(vocab=100, dim=64, ffn=96, lengths=(300, 20, 137))
    tokens, _ = inputs(m)
    gen = torch.Generator(device="cuda").manual_seed(6)
    m.d_logits.copy_(torch.randn(m.rows, m.vocab, generator=gen, device="cuda"))
    want = []
    for _ in range(3):
        forward_backward(m, tokens)
        want.append((m.logits.clone(), m.bucket.clone()))
    assert not torch.equal(want[0][1], want[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward_backward(m, tokens)
    m.counter.zero_()
    for logits, bucket in want:
        m.bucket.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.logits, logits) and torch.equal(m.bucket, bucket)
    assert dgc.dgc_read_status(m.status) == 0


def test_two_models_on_two_streams():
    models = [model(vocab=300, dim=128, ffn=192, lengths=(900, 400, 1500), seed=i) for i in (1, 2)]
    data = [inputs(m)[0] for m in models]
    want = []
    for m, t in zip(models, data):
        m.d_logits.normal_(generator=m.gen)
        forward_backward(m, t)
        want.append(m.bucket.clone())
        m.counter.zero_()
    streams = [torch.cuda.Stream() for _ in models]
    for _ in range(4):
        for m in models:
            m.bucket.fill_(1.0)
            m.counter.zero_()
        torch.cuda.synchronize()
        for m, t, s in zip(models, data, streams):
            with torch.cuda.stream(s):
                forward_backward(m, t)
        torch.cuda.synchronize()
        for m, w in zip(models, want):
            assert torch.equal(m.bucket, w)
            assert dgc.dgc_read_status(m.status) == 0
