"""Training a small recurrent language model with compressed gradients, all of it in the library.

    e  = scale E[tokens]                                             dgc_embed
    s1 = e  + drop(rec(n1 Wx^T, n1 Wz^T) Wo^T),   n1 = norm(e)       dgc_layer_norm, dgc_recurrence,
    s2 = s1 + drop(ffn(n2)),                      n2 = norm(s1)      dgc_dropout, dgc_ffn_*
    logits = norm(s2) E^T

over a packed batch of sequences of unequal length. The loss is the mean cross-entropy of the next
token; its softmax is the only arithmetic outside the library. The gradients of all weights land in one
flat binary32 bucket, E's from both of its uses, and go from there as every learner's do: clipped by
their global norm (dgc_grad_clip), compressed, encoded, decoded and applied to the binary32 master
weights (dgc_compress, dgc_encode, dgc_decode_apply_dev). The products read bfloat16 copies of them.
A product with one weight matrix is dgc_ffn_down; its data-path backward pass dgc_ffn_gate_backward on
the matrix's two halves.

    python examples/recurrent_lm_step.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparsified_gradient_compression_gb300 as dgc  # noqa: E402

EPS = 1e-5
PAD = 0  # the padding's token: no gradient


class RecurrentLm:
    MATRICES = ("table", "wx", "wz", "wo", "wg", "wu", "wd")
    VECTORS = ("g1", "b1", "g2", "b2", "g3", "b3")

    def __init__(self, vocab=512, dim=256, ffn=512, lengths=(200, 0, 37, 512, 275), drop=0.1,
                 sparsity=0.99, lr=0.5, max_norm=1.0, seed=0):
        self.vocab, self.dim, self.drop, self.lr, self.max_norm = vocab, dim, drop, lr, max_norm
        self.seed, self.scale = seed, math.sqrt(dim)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        rows = self.rows = sum(lengths)
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        self.offsets = torch.tensor(ends, dtype=torch.int64, device="cuda")
        shapes = dict(table=(vocab, dim), wx=(dim, dim), wz=(dim, dim), wo=(dim, dim),
                      wg=(ffn, dim), wu=(ffn, dim), wd=(dim, ffn))
        shapes.update({k: (dim,) for k in self.VECTORS})
        sizes = [math.prod(s) for s in shapes.values()]
        n = sum(sizes)

        def pieces(flat):
            return {k: p.view(s) for (k, s), p in zip(shapes.items(), flat.split(sizes))}

        # master weights and the gradient bucket, flat, a piece a weight; bfloat16 copies
        self.master, self.bucket = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        self.w, self.grad = pieces(self.master), pieces(self.bucket)
        for k in self.MATRICES:
            self.w[k].copy_(torch.randn(shapes[k], generator=self.gen, device="cuda")
                            * shapes[k][1] ** -0.5)
        for k in ("g1", "g2", "g3"):
            self.w[k].fill_(1.0)
        self.copies = {k: self.w[k].bfloat16() for k in self.MATRICES}

        def bf16(cols, *names):
            for k in names:
                setattr(self, k, torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"))

        def f32(*shape):
            return torch.empty(*shape, device="cuda")

        bf16(dim, "e", "n1", "x", "z", "h", "r", "s1", "n2", "f", "s2", "n3",
             "d1", "d2", "d3", "d4")
        bf16(ffn, "hidden", "gate", "up", "d_gate", "d_up")
        bf16(vocab, "logits", "d_logits")
        self.stats = [(f32(rows), f32(rows)) for _ in range(3)]
        self.saved = f32(dgc.dgc_recurrence_saved_rows(rows), dim)
        self.counter = torch.zeros(1, dtype=torch.int64, device="cuda")  # numbers the steps' masks
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # one workspace for all: the calls are on one stream
        need = [dgc.dgc_recurrence_workspace(rows, dim),
                dgc.dgc_layer_norm_backward_workspace(rows, dim),
                dgc.dgc_embed_backward_workspace(rows, vocab, dim)]
        need += [dgc.dgc_ffn_weight_grad_workspace(*shapes[k], rows) for k in self.MATRICES]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")

        # clipping, compressor, codec and decoder over the bucket, a segment a weight
        self.list = dgc.TensorList(self.grad.values())
        self.norm, self.clip = f32(1), f32(1)
        self.clip_ws = torch.empty(dgc.dgc_grad_workspace(self.list), dtype=torch.uint8,
                                   device="cuda")
        self.params = dgc.make_params(mode=dgc.SELECT_EXACT, sparsity=sparsity, momentum=0.9)
        nseg = len(sizes)
        self.seg_off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()],
                                    dtype=torch.int64, device="cuda")
        self.u, self.v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        cap = dgc.dgc_compress_max_out(n, nseg, self.params)
        self.idx, self.val = torch.empty(cap, dtype=torch.int32, device="cuda"), f32(cap)
        self.count = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.compress_ws = torch.empty(dgc.dgc_compress_workspace(n, nseg, self.params),
                                       dtype=torch.uint8, device="cuda")
        self.most = [dgc.dgc_encode_max_bytes(cap, n)]
        self.message = torch.empty(self.most[0], dtype=torch.uint8, device="cuda")
        self.message_bytes = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.encode_ws = torch.empty(dgc.dgc_encode_workspace(cap), dtype=torch.uint8,
                                     device="cuda")
        self.decode_ws = torch.empty(dgc.dgc_decode_workspace_bound(self.most, n),
                                     dtype=torch.uint8, device="cuda")

    def dropped(self, x, residual, layer, out):
        """out = residual + drop(x); the same call on the gradient is its backward pass."""
        dgc.dgc_dropout(x, residual, self.drop, 1000 * self.seed + layer, self.counter, out)

    def normed(self, x, i, out):
        dgc.dgc_layer_norm(x, self.w[f"g{i}"], self.w[f"b{i}"], EPS, out, *self.stats[i - 1])

    def forward(self, tokens):
        c, st = self.copies, self.status
        dgc.dgc_embed(c["table"], tokens, self.scale, self.e, st)
        self.normed(self.e, 1, self.n1)
        dgc.dgc_ffn_down(self.n1, c["wx"], None, self.x, st)
        dgc.dgc_ffn_down(self.n1, c["wz"], None, self.z, st)
        dgc.dgc_recurrence(self.x, self.z, self.offsets, None, self.h, None, self.saved, st,
                           self.ws)
        dgc.dgc_ffn_down(self.h, c["wo"], None, self.r, st)
        self.dropped(self.r, self.e, 1, self.s1)
        self.normed(self.s1, 2, self.n2)
        dgc.dgc_ffn_gate(self.n2, c["wg"], c["wu"], dgc.ACT_SILU, self.hidden, self.gate, self.up,
                         st)
        dgc.dgc_ffn_down(self.hidden, c["wd"], None, self.f, st)
        self.dropped(self.f, self.s1, 2, self.s2)
        self.normed(self.s2, 3, self.n3)
        dgc.dgc_ffn_down(self.n3, c["table"], None, self.logits, st)

    def norm_backward(self, dy, x, i, residual, dx):
        dgc.dgc_layer_norm_backward(dy, x, self.w[f"g{i}"], *self.stats[i - 1], residual, dx,
                                    self.grad[f"g{i}"], self.grad[f"b{i}"], False, self.ws)

    def times(self, dy, name, dx):
        """dx = dy W, by W's two halves."""
        w, half = self.copies[name], self.copies[name].shape[0] // 2
        dgc.dgc_ffn_gate_backward(dy[:, :half], dy[:, half:], w[:half], w[half:], None, dx,
                                  self.status)

    def weight_grad(self, dy, x, name):
        dgc.dgc_ffn_weight_grad(dy, x, self.grad[name], False, self.status, self.ws)

    def backward(self, tokens):
        """The bucket's gradients from d_logits."""
        c, st = self.copies, self.status
        d1, d2, d3, d4 = self.d1, self.d2, self.d3, self.d4
        self.weight_grad(self.d_logits, self.n3, "table")
        self.times(self.d_logits, "table", d1)
        self.norm_backward(d1, self.s2, 3, None, d2)                  # d2: of s2
        self.dropped(d2, None, 2, d1)                                 # d1: of the block's result
        dgc.dgc_ffn_down_backward(d1, c["wd"], self.gate, self.up, dgc.ACT_SILU, self.d_gate,
                                  self.d_up, st)
        self.weight_grad(d1, self.hidden, "wd")
        self.weight_grad(self.d_gate, self.n2, "wg")
        self.weight_grad(self.d_up, self.n2, "wu")
        dgc.dgc_ffn_gate_backward(self.d_gate, self.d_up, c["wg"], c["wu"], None, d1, st)
        self.norm_backward(d1, self.s1, 2, d2, d2)                    # d2: of s1
        self.dropped(d2, None, 1, d1)
        self.weight_grad(d1, self.h, "wo")
        self.times(d1, "wo", d3)
        dgc.dgc_recurrence_backward(d3, self.x, self.z, self.offsets, None, self.saved, None, d3,
                                    d4, None, st, self.ws)            # d3, d4: of x and z
        self.weight_grad(d3, self.n1, "wx")
        self.weight_grad(d4, self.n1, "wz")
        dgc.dgc_ffn_gate_backward(d3, d4, c["wx"], c["wz"], None, d1, st)
        self.norm_backward(d1, self.e, 1, d2, d2)                     # d2: of e
        dgc.dgc_embed_backward(tokens, d2, self.scale, PAD, self.grad["table"], True, st, self.ws)

    def step(self, tokens, targets):
        """One step; the mean cross-entropy before it. Targets of PAD are not counted."""
        self.counter += 1
        self.forward(tokens)
        logp = torch.log_softmax(self.logits.float(), 1)
        counted = (targets != PAD).float()
        share = counted / counted.sum()
        loss = -(logp.gather(1, targets[:, None])[:, 0] * share).sum()
        d = logp.exp()
        d.scatter_add_(1, targets[:, None], -torch.ones_like(d[:, :1]))
        self.d_logits.copy_(d * share[:, None])
        self.backward(tokens)
        dgc.dgc_grad_clip(self.list, None, self.max_norm, self.norm, self.clip, self.clip_ws)
        dgc.dgc_compress(self.bucket, self.u, self.v, self.seg_off, self.params, self.idx, self.val,
                         self.count, None, self.status, self.compress_ws)
        n = self.bucket.numel()
        dgc.dgc_encode(self.idx, self.val, self.count, n, self.message, self.message_bytes,
                       self.status, self.encode_ws)
        dgc.dgc_decode_apply_dev([self.message], self.message_bytes, self.most, self.master, n,
                                 self.lr, self.status, self.decode_ws)
        for k, w in self.copies.items():
            w.copy_(self.w[k])
        return loss


def batch(model):
    """Counting sequences with a step of their own, the padding's token behind each."""
    ends = model.offsets.tolist()
    tokens = torch.empty(model.rows, dtype=torch.int64, device="cuda")
    for a, b in zip(ends, ends[1:]):
        start, stride = torch.randint(0, model.vocab, (2,), generator=model.gen,
                                      device="cuda").tolist()
        run = (start + (stride % 7 + 1) * torch.arange(b - a, device="cuda")) % (model.vocab - 1)
        tokens[a:b] = run + 1
        tokens[max(a, b - 5):b] = PAD
    targets = torch.cat([tokens[1:], tokens[:1]])
    targets[[b - 1 for a, b in zip(ends, ends[1:]) if b > a]] = PAD
    return tokens, targets


def main(steps=40):
    dgc.build()
    model = RecurrentLm()
    for i in range(steps):
        loss = model.step(*batch(model))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}  gradient norm {model.norm.item():.4f}  "
                  f"clipped by {model.clip.item():.3f}  message {model.message_bytes.item()} of "
                  f"{4 * model.bucket.numel()} bytes")
    assert dgc.dgc_read_status(model.status) == 0


if __name__ == "__main__":
    main()
