"""Measured cases of the training-step operators around the gradient compressor.

Two groups. The global norm of a step's gradient tensors with the clipped copy into the
compressor's flat bucket (dgc_grad_norm, dgc_grad_clip), and a gated feed-forward block whose
weight gradients land in that bucket (dgc_ffn_gate, dgc_ffn_down, dgc_ffn_down_backward,
dgc_ffn_gate_backward, dgc_ffn_weight_grad). With `own` set, run() makes the library's calls;
without it, the same mathematics in elementary torch operations, in 32 bits, rounded once.
"""
import math
import random

import torch

own = False

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm for the log of a single small tensor: latency of one call
        dict(name="norm_1m", op="norm", layout="one", n=1 << 20, dtype="float32", max_norm=1.0),
        # the norm of the whole 1B-entry bucket, one read of 4 GiB
        dict(name="norm_bucket_1g", op="norm", layout="one", n=1 << 30, dtype="float32",
             max_norm=1.0),
        # an image model's 161 gradient tensors, clipped by their global norm into the bucket
        dict(name="clip_resnet50", op="clip", layout="resnet50", n=25557032, dtype="float32",
             max_norm=1.0),
        # a language model's layers: 16-bit matrix gradients, 32-bit vectors, into the bucket
        dict(name="clip_layers_bf16", op="clip", layout="layers", n=2, dim=4096, ffn=11264,
             dtype="bfloat16", max_norm=1.0),
        # the forward pass of one token: the weights are read for a single row
        dict(name="ffn_one_token", op="forward", tokens=1, dim=1024, ffn=4096, act="silu",
             dtype="bfloat16"),
        # a short ragged batch: odd sizes, rows padded to the alignment
        dict(name="ffn_ragged", op="forward", tokens=777, dim=1001, ffn=2721, act="gelu",
             dtype="float16"),
        # a training step's batch of tokens through one large layer
        dict(name="ffn_8k_tokens", op="forward", tokens=8192, dim=4096, ffn=11264, act="silu",
             dtype="bfloat16"),
        # the data path of the backward pass of a small layer with a ragged batch
        dict(name="backward_ragged", op="backward", tokens=1531, dim=1024, ffn=2816,
             act="gelu_tanh", dtype="float16"),
        # and of the large layer
        dict(name="backward_8k_tokens", op="backward", tokens=8192, dim=4096, ffn=11264,
             act="silu", dtype="bfloat16"),
        # weight gradient of a few tokens, added to the bucket (micro-batches): latency
        dict(name="wgrad_33_tokens", op="wgrad", tokens=33, rows=1024, cols=1024,
             dtype="bfloat16", accumulate=True),
        # a small weight over many tokens: few output tiles, a long sum
        dict(name="wgrad_16k_tokens", op="wgrad", tokens=16384, rows=1024, cols=1024,
             dtype="bfloat16", accumulate=False),
        # the large layer's weight gradient, added to the bucket
        dict(name="wgrad_8k_tokens", op="wgrad", tokens=8192, rows=11264, cols=4096,
             dtype="bfloat16", accumulate=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "clip", "forward", "backward", "wgrad"))
    dtype = rng.choice(("bfloat16", "float16"))
    if op in ("norm", "clip"):
        return dict(op=op, layout="random", n=_spread(rng, 1000, 1 << 28),
                    count=_spread(rng, 1, 600), salt=rng.randrange(1 << 30),
                    dtype=rng.choice(("float32", "float16", "bfloat16")),
                    max_norm=rng.choice((0.5, 1.0, 1e9)))
    if op == "wgrad":
        return dict(op=op, tokens=_spread(rng, 1, 8192), rows=_spread(rng, 64, 8192),
                    cols=_spread(rng, 64, 4096), dtype=dtype, accumulate=rng.random() < 0.5)
    return dict(op=op, tokens=_spread(rng, 1, 8192), dim=_spread(rng, 64, 4096),
                ffn=_spread(rng, 64, 11264), act=rng.choice(ACTS), dtype=dtype)


def _resnet50_sizes():
    sizes, inp = [64 * 3 * 49, 64, 64], 64
    for blocks, width in ((3, 64), (4, 128), (6, 256), (3, 512)):
        for b in range(blocks):
            out = 4 * width
            sizes += [width * inp, width, width, 9 * width * width, width, width,
                      out * width, out, out]
            if b == 0:
                sizes += [out * inp, out, out]
            inp = out
    return sizes + [1000 * 2048, 1000]


def _tensors(case):
    """(size, dtype) of each gradient tensor."""
    dt = case["dtype"]
    if case["layout"] == "one":
        return [(case["n"], dt)]
    if case["layout"] == "resnet50":
        return [(n, dt) for n in _resnet50_sizes()]
    if case["layout"] == "layers":
        d, f = case["dim"], case["ffn"]
        return [(d, "float32"), (d * d, dt), (d * d, dt), (d * d, dt), (d * d, dt),
                (d, "float32"), (f * d, dt), (f * d, dt), (d * f, dt)] * case["n"]
    r = random.Random(case["salt"])
    part = [math.exp(r.uniform(0.0, 8.0)) for _ in range(case["count"])]
    total = sum(part)
    return [(int(case["n"] * p / total), dt) for p in part]


# ----------------------------------------------------------------------------------- prepare
def _padded(rows, cols, dtype):
    """A rows x cols view whose rows start on 16-byte boundaries."""
    return torch.empty(rows, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]


def _normal(gen, rows, cols, dtype, sigma):
    t = _padded(rows, cols, dtype)
    t.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * sigma)
    return t


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("norm", "clip"):
        # heavy-tailed over the tensors, as layers' gradients are: each has its own scale
        spread = random.Random(seed)
        s["grads"] = []
        for n, dt in _tensors(case):
            g = torch.randn(n, generator=gen, device="cuda")
            g *= 10.0 ** spread.uniform(-4.0, -1.0)
            s["grads"].append(g.to(getattr(torch, dt)))
        s["norm"] = torch.zeros(1, device="cuda")
        s["scale"] = torch.zeros(1, device="cuda")
        sizes = [g.numel() for g in s["grads"]]
        if op == "clip":
            s["bucket"] = torch.empty(sum(sizes), device="cuda")
        if own:
            import sparsified_gradient_compression_gb300 as dgc

            s["src"] = dgc.TensorList(s["grads"])
            if op == "clip":
                s["dst"] = dgc.TensorList(list(s["bucket"].split(sizes)))
            s["ws"] = torch.empty(dgc.dgc_grad_workspace(s["src"]), dtype=torch.uint8,
                                  device="cuda")
        return s
    dtype = getattr(torch, case["dtype"])
    m = case["tokens"]
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "wgrad":
        s["dy"] = _normal(gen, m, case["rows"], dtype, 0.1)
        s["x"] = _normal(gen, m, case["cols"], dtype, 1.0)
        s["dw"] = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda")
        if own:
            import sparsified_gradient_compression_gb300 as dgc

            s["m"] = {k: dgc.matrix(s[k]) for k in ("dy", "x", "dw")}
            s["ws"] = torch.empty(
                dgc.dgc_ffn_weight_grad_workspace(case["rows"], case["cols"], m),
                dtype=torch.uint8, device="cuda")
        return s
    d, f = case["dim"], case["ffn"]
    s["wg"] = _normal(gen, f, d, dtype, d ** -0.5)
    s["wu"] = _normal(gen, f, d, dtype, d ** -0.5)
    s["wd"] = _normal(gen, d, f, dtype, f ** -0.5)
    if op == "forward":
        s["x"] = _normal(gen, m, d, dtype, 1.0)
        s.update({k: _padded(m, f, dtype) for k in ("hidden", "gate", "up")})
        s["y"] = _padded(m, d, dtype)
        names = ("x", "wg", "wu", "wd", "hidden", "gate", "up", "y")
    else:
        s["dy"] = _normal(gen, m, d, dtype, 0.1)
        s["gate"] = _normal(gen, m, f, dtype, 1.0)
        s["up"] = _normal(gen, m, f, dtype, 1.0)
        s.update({k: _padded(m, f, dtype) for k in ("dgate", "dup")})
        s["dx"] = _padded(m, d, dtype)
        names = ("dy", "wg", "wu", "wd", "gate", "up", "dgate", "dup", "dx")
    if own:
        import sparsified_gradient_compression_gb300 as dgc

        s["m"] = {k: dgc.matrix(s[k]) for k in names}
    return s


# --------------------------------------------------------------------------------------- run
def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return torch.where(g > 0, g, torch.zeros_like(g))


def _act_slope(name, g):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
                + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi)))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)
    return (g > 0).to(g.dtype)


def _run_own(s):
    import sparsified_gradient_compression_gb300 as dgc

    case = s["case"]
    op = case["op"]
    if op == "norm":
        dgc.dgc_grad_norm(s["src"], case["max_norm"], s["norm"], s["scale"], s["ws"])
        return {"norm": s["norm"], "scale": s["scale"]}
    if op == "clip":
        dgc.dgc_grad_clip(s["src"], s["dst"], case["max_norm"], s["norm"], s["scale"], s["ws"])
        return {"norm": s["norm"], "scale": s["scale"], "bucket": s["bucket"]}
    m, st = s["m"], s["status"]
    if op == "wgrad":
        dgc.dgc_ffn_weight_grad(m["dy"], m["x"], m["dw"], case["accumulate"], st, s["ws"])
        return {"dw": s["dw"]}
    act = getattr(dgc, "ACT_" + case["act"].upper())
    if op == "forward":
        dgc.dgc_ffn_gate(m["x"], m["wg"], m["wu"], act, m["hidden"], m["gate"], m["up"], st)
        dgc.dgc_ffn_down(m["hidden"], m["wd"], m["x"], m["y"], st)
        return {k: s[k] for k in ("hidden", "gate", "up", "y")}
    dgc.dgc_ffn_down_backward(m["dy"], m["wd"], m["gate"], m["up"], act, m["dgate"], m["dup"], st)
    dgc.dgc_ffn_gate_backward(m["dgate"], m["dup"], m["wg"], m["wu"], m["dy"], m["dx"], st)
    return {k: s[k] for k in ("dgate", "dup", "dx")}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op in ("norm", "clip"):
        flat = torch.cat([g.float() for g in s["grads"]]) if len(s["grads"]) > 1 else (
            s["grads"][0].float())
        norm = (flat * flat).sum().sqrt()
        scale = torch.where(norm > case["max_norm"], case["max_norm"] / norm,
                            torch.ones_like(norm))
        if op == "norm":
            return {"norm": norm.reshape(1), "scale": scale.reshape(1)}
        return {"norm": norm.reshape(1), "scale": scale.reshape(1), "bucket": flat * scale}
    if op == "wgrad":
        p = s["dy"].float().t() @ s["x"].float()
        if case["accumulate"]:
            s["dw"] += p
        else:
            s["dw"].copy_(p)
        return {"dw": s["dw"]}
    dtype, act = s["wd"].dtype, case["act"]
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    if op == "forward":
        x = s["x"].float()
        gate, up = x @ wg.t(), x @ wu.t()
        hidden = _act(act, gate) * up
        y = hidden @ wd.t() + x
        return {"hidden": hidden.to(dtype), "gate": gate.to(dtype), "up": up.to(dtype),
                "y": y.to(dtype)}
    dy, gate, up = s["dy"].float(), s["gate"].float(), s["up"].float()
    dh = dy @ wd
    dgate = dh * up * _act_slope(act, gate)
    dup = dh * _act(act, gate)
    dx = dgate @ wg + dup @ wu + dy
    return {"dgate": dgate.to(dtype), "dup": dup.to(dtype), "dx": dx.to(dtype)}


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        total = 0.0
        for g in s["grads"]:
            for part in g.split(1 << 26):
                v = part.to(torch.float64)
                total += float(torch.dot(v, v))
        norm = math.sqrt(total)
        scale = min(1.0, case["max_norm"] / norm) if norm > 0 else 1.0
        out = {"norm": torch.tensor([norm], dtype=torch.float64),
               "scale": torch.tensor([scale], dtype=torch.float64)}
        if op == "clip":
            bucket = torch.empty(sum(g.numel() for g in s["grads"]), dtype=torch.float64,
                                 device="cuda")
            at = 0
            for g in s["grads"]:
                bucket[at:at + g.numel()] = g.to(torch.float64) * scale
                at += g.numel()
            out["bucket"] = bucket
        return out
    if op == "wgrad":
        dw = torch.einsum("mi,mj->ij", s["dy"].double(), s["x"].double())
        return {"dw": dw + s["dw"].double() if case["accumulate"] else dw}
    g64 = {k: v.double() for k, v in s.items()
           if isinstance(v, torch.Tensor) and k in ("x", "dy", "wg", "wu", "wd")}
    if op == "forward":
        gate = torch.einsum("md,fd->mf", g64["x"], g64["wg"])
        up = torch.einsum("md,fd->mf", g64["x"], g64["wu"])
        hidden = _value64(case["act"], gate)[0] * up
        y = g64["x"] + torch.einsum("mf,df->md", hidden, g64["wd"])
        return {"hidden": hidden, "gate": gate, "up": up, "y": y}
    gate, up = s["gate"].double(), s["up"].double()
    dh = torch.einsum("md,df->mf", g64["dy"], g64["wd"])
    value, slope = _value64(case["act"], gate)
    dgate, dup = dh * up * slope, dh * value
    dx = (g64["dy"] + torch.einsum("mf,fd->md", dgate, g64["wg"])
          + torch.einsum("mf,fd->md", dup, g64["wu"]))
    return {"dgate": dgate, "dup": dup, "dx": dx}


def _value64(act, g):
    """The activation and its derivative in 64 bits, by autograd from the definition."""
    g = g.clone().requires_grad_(True)
    if act == "silu":
        v = g * torch.sigmoid(g)
    elif act == "gelu":
        v = g * 0.5 * torch.erfc(-g / math.sqrt(2.0))
    elif act == "gelu_tanh":
        v = g * torch.sigmoid(math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3))
    else:
        v = torch.relu(g)
    slope, = torch.autograd.grad(v.sum(), g)
    return v.detach(), slope


# -------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        size = {"float32": 4, "float16": 2, "bfloat16": 2}
        read = sum(n * size[dt] for n, dt in _tensors(case))
        n = sum(n for n, _ in _tensors(case))
        return {"bytes": read + 8 + (4 * n if op == "clip" else 0),
                "flops": (3 if op == "clip" else 2) * n}
    m = case["tokens"]
    if op == "wgrad":
        r, c = case["rows"], case["cols"]
        return {"bytes": 2 * m * (r + c) + (8 if case["accumulate"] else 4) * r * c,
                "flops": 2 * m * r * c}
    d, f = case["dim"], case["ffn"]
    if op == "forward":  # x once, three weights, gate, up, hidden and y written
        return {"bytes": 2 * (m * d + 3 * d * f + 3 * m * f + m * d), "flops": 6 * m * d * f}
    # dy, three weights, gate and up read; dgate, dup and dx written
    return {"bytes": 2 * (m * d + 3 * d * f + 4 * m * f + m * d), "flops": 6 * m * d * f}
