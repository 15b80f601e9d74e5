"""Training a gated feed-forward block with compressed gradients, all of it in the library.

The block y = x + (silu(x Wg^T) o (x Wu^T)) Wd^T learns to follow a fixed teacher of the same shape.
A step is what one learner does: for each micro-batch the forward pass (dgc_ffn_gate, dgc_ffn_down)
and the backward pass (dgc_ffn_down_backward), whose weight gradients (dgc_ffn_weight_grad) are
added up in the flat binary32 bucket; the bucket's pieces clipped to their global norm in place
(dgc_grad_clip); the bucket compressed, encoded, and the message decoded and applied to the
binary32 master weights (dgc_compress, dgc_encode, dgc_decode_apply_dev). The bfloat16 weights that
the products read are copies of the master weights.

    python examples/ffn_training_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparsified_gradient_compression_gb300 as dgc  # noqa: E402


class FfnTrainer:
    def __init__(self, dim=512, ffn=1536, tokens=1024, micro_batches=2, sparsity=0.99, lr=0.2,
                 max_norm=1.0, seed=0):
        self.lr, self.max_norm, self.micro_batches = lr, max_norm, micro_batches
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.dim, self.ffn = tokens, dim, ffn
        shapes = [(ffn, dim), (ffn, dim), (dim, ffn)]
        sizes = [r * c for r, c in shapes]
        n = sum(sizes)

        def pieces(flat):
            return [p.view(s) for p, s in zip(flat.split(sizes), shapes)]

        def weights():
            return torch.cat([torch.randn(s, generator=self.gen, device="cuda").flatten()
                              * s[1] ** -0.5 for s in shapes])

        # master weights and the gradient bucket: flat, one piece per matrix
        self.master, self.bucket = weights(), torch.zeros(n, device="cuda")
        self.master_pieces, self.grads = pieces(self.master), pieces(self.bucket)
        self.teacher = [w.bfloat16() for w in pieces(weights())]
        self.weights = [w.bfloat16() for w in self.master_pieces]

        def matrix(rows, cols):
            return torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")

        self.hidden, self.gate, self.up, self.d_gate, self.d_up = (matrix(tokens, ffn)
                                                                   for _ in range(5))
        self.y, self.target, self.dx = (matrix(tokens, dim) for _ in range(3))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.grad_ws = torch.empty(
            max(1, max(dgc.dgc_ffn_weight_grad_workspace(r, c, tokens) for r, c in shapes)),
            dtype=torch.uint8, device="cuda")

        # clipping: the bucket's pieces as one list
        self.list = dgc.TensorList(self.grads)
        self.norm, self.scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        self.clip_ws = torch.empty(dgc.dgc_grad_workspace(self.list), dtype=torch.uint8,
                                   device="cuda")

        # compressor, codec and decoder over the bucket, a segment per matrix
        self.params = dgc.make_params(mode=dgc.SELECT_EXACT, sparsity=sparsity, momentum=0.9)
        self.seg_off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()],
                                    dtype=torch.int64, device="cuda")
        self.u, self.v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        cap = dgc.dgc_compress_max_out(n, 3, self.params)
        self.idx = torch.empty(cap, dtype=torch.int32, device="cuda")
        self.val = torch.empty(cap, device="cuda")
        self.count = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.compress_ws = torch.empty(dgc.dgc_compress_workspace(n, 3, self.params),
                                       dtype=torch.uint8, device="cuda")
        most = dgc.dgc_encode_max_bytes(cap, n)
        self.message = torch.empty(most, dtype=torch.uint8, device="cuda")
        self.message_bytes = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.encode_ws = torch.empty(dgc.dgc_encode_workspace(cap), dtype=torch.uint8,
                                     device="cuda")
        self.most = [most]
        self.decode_ws = torch.empty(dgc.dgc_decode_workspace_bound(self.most, n),
                                     dtype=torch.uint8, device="cuda")

    def forward(self, weights, x, y, save):
        """y = x + block(x)."""
        wg, wu, wd = weights
        gate, up = (self.gate, self.up) if save else (None, None)
        dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_SILU, self.hidden, gate, up, self.status)
        dgc.dgc_ffn_down(self.hidden, wd, x, y, self.status)

    def backward(self, x, dy, first):
        """Adds the weight gradients of one micro-batch to the bucket (the first one overwrites
        it), and makes dx, which a layer below would take as its dy."""
        wg, wu, wd = self.weights
        dgc.dgc_ffn_down_backward(dy, wd, self.gate, self.up, dgc.ACT_SILU, self.d_gate, self.d_up,
                                  self.status)
        dgc.dgc_ffn_gate_backward(self.d_gate, self.d_up, wg, wu, dy, self.dx, self.status)
        for dw, a, b in zip(self.grads, (self.d_gate, self.d_up, dy), (x, x, self.hidden)):
            dgc.dgc_ffn_weight_grad(a, b, dw, not first, self.status, self.grad_ws)

    def step(self):
        """One step; the mean squared error before it."""
        loss = torch.zeros((), device="cuda")
        for i in range(self.micro_batches):
            x = torch.randn(self.tokens, self.dim, generator=self.gen, device="cuda").bfloat16()
            self.forward(self.teacher, x, self.target, False)
            self.forward(self.weights, x, self.y, True)
            error = self.y.float() - self.target.float()
            loss += error.square().mean() / self.micro_batches
            dy = (error * (2.0 / (self.tokens * self.micro_batches))).bfloat16()
            self.backward(x, dy, i == 0)
        dgc.dgc_grad_clip(self.list, None, self.max_norm, self.norm, self.scale, self.clip_ws)
        dgc.dgc_compress(self.bucket, self.u, self.v, self.seg_off, self.params, self.idx, self.val,
                         self.count, None, self.status, self.compress_ws)
        n = self.bucket.numel()
        dgc.dgc_encode(self.idx, self.val, self.count, n, self.message, self.message_bytes,
                       self.status, self.encode_ws)
        dgc.dgc_decode_apply_dev([self.message], self.message_bytes, self.most, self.master, n,
                                 self.lr, self.status, self.decode_ws)
        for w, m in zip(self.weights, self.master_pieces):
            w.copy_(m)
        return loss


def main(steps=60):
    dgc.build()
    t = FfnTrainer()
    for i in range(steps):
        loss = t.step()
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}  gradient norm {t.norm.item():.4f}  "
                  f"clipped by {t.scale.item():.3f}  message {t.message_bytes.item()} of "
                  f"{4 * t.bucket.numel()} bytes")
    assert dgc.dgc_read_status(t.status) == 0


if __name__ == "__main__":
    main()
