"""Measured cases of the operators that surround a feed-forward block in a language model.

Embedding lookup with scaling and its gradient by sorted tokens (dgc_embed, dgc_embed_backward),
layer norm and its backward pass (dgc_layer_norm, dgc_layer_norm_backward), dropout from a
counter-based generator (dgc_dropout), and a gated linear recurrence over packed sequences with its
backward pass (dgc_recurrence, dgc_recurrence_backward). Their weights' gradients land in the
compressor's binary32 bucket. With `own` set, run() makes the library's calls; without it, the same
mathematics in elementary torch operations, in 32 bits, rounded once.
"""
import math
import random

import numpy as np
import torch

own = False

BITS = {"float32": 4, "float16": 2, "bfloat16": 2}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the lookup of a training step's tokens in a table of 16-bit copies, scaled by the root
        # of the width
        dict(name="embed_16k", op="embed", tokens=16384, vocab=50000, dim=4096, scale=64.0,
             table="bfloat16", dtype="bfloat16", wide=False),
        # a micro-batch with padding at its end, odd width: its gradient added to the bucket
        dict(name="embed_grad_ragged", op="embed_grad", tokens=5001, vocab=10000, dim=1001,
             scale=31.64, padded=0.1, dtype="float16", accumulate=True, wide=True),
        # a whole step's gradient of a large table, every row written
        dict(name="embed_grad_16k", op="embed_grad", tokens=16384, vocab=50000, dim=4096,
             scale=64.0, padded=0.0, dtype="bfloat16", accumulate=False, wide=False),
        # the norm of a short ragged batch
        dict(name="norm_ragged", op="norm", rows=777, cols=1001, dtype="float16", beta=True),
        # the norm ahead of a large layer
        dict(name="norm_16k", op="norm", rows=16384, cols=4096, dtype="bfloat16", beta=True),
        # its backward pass, with the gradient that went around the layer, weights' gradients
        # into the bucket
        dict(name="norm_grad_16k", op="norm_grad", rows=16384, cols=4096, dtype="bfloat16",
             residual=True, accumulate=False),
        # a few rows of a small layer: latency
        dict(name="dropout_33", op="dropout", rows=33, cols=1024, dtype="float16", p=0.1,
             residual=True),
        # a ragged batch in 32 bits, the backward direction: no residual
        dict(name="dropout_ragged", op="dropout", rows=1531, cols=2721, dtype="float32", p=0.25,
             residual=False),
        # a feed-forward block's result for a large batch, dropped on its way to the residual
        dict(name="dropout_8k", op="dropout", rows=8192, cols=11264, dtype="bfloat16", p=0.1,
             residual=True),
        # one token of each of 64 sequences: the state read and written
        dict(name="recur_step", op="recur", rows=64, cols=4096, sequences=64, even=True,
             state=True, dtype="bfloat16"),
        # one long sequence
        dict(name="recur_long", op="recur", rows=32768, cols=2048, sequences=1, even=True,
             state=True, dtype="bfloat16"),
        # a packed batch of sequences of unequal length, forward and backward
        dict(name="recur_train_ragged", op="recur_train", rows=16001, cols=2048, sequences=37,
             even=False, state=True, dtype="float16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "norm", "norm_grad", "dropout", "recur",
                     "recur_train"))
    dtype = rng.choice(("float32", "float16", "bfloat16", "bfloat16"))
    if op == "embed":
        dim = _spread(rng, 64, 4096)
        return dict(op=op, tokens=_spread(rng, 1, 16384), vocab=_spread(rng, 256, 50000), dim=dim,
                    scale=rng.choice((1.0, round(dim ** 0.5, 2))),
                    table=rng.choice(("float32", dtype)), dtype=dtype, wide=rng.random() < 0.5)
    if op == "embed_grad":
        dim = _spread(rng, 64, 4096)
        return dict(op=op, tokens=_spread(rng, 1, 16384), vocab=_spread(rng, 256, 50000), dim=dim,
                    scale=rng.choice((1.0, round(dim ** 0.5, 2))),
                    padded=rng.choice((0.0, 0.1, 0.4)), dtype=dtype,
                    accumulate=rng.random() < 0.5, wide=rng.random() < 0.5)
    if op in ("norm", "norm_grad"):
        case = dict(op=op, rows=_spread(rng, 1, 8192), cols=_spread(rng, 64, 8192), dtype=dtype)
        if op == "norm":
            return dict(case, beta=rng.random() < 0.7)
        return dict(case, residual=rng.random() < 0.5, accumulate=rng.random() < 0.5)
    if op == "dropout":
        return dict(op=op, rows=_spread(rng, 1, 8192), cols=_spread(rng, 64, 8192), dtype=dtype,
                    p=rng.choice((0.05, 0.1, 0.25, 0.5)), residual=rng.random() < 0.5)
    rows = _spread(rng, 1, 16384)
    return dict(op=op, rows=rows, cols=_spread(rng, 64, 2048),
                sequences=min(rows, _spread(rng, 1, 128)), even=rng.random() < 0.3,
                state=rng.random() < 0.5, dtype=dtype)


# ----------------------------------------------------------------------------------- prepare
def _padded(rows, cols, dtype):
    """A rows x cols view whose rows start on 16-byte boundaries."""
    return torch.empty(rows, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]


def _normal(gen, rows, cols, dtype, sigma=1.0, mean=0.0):
    t = _padded(rows, cols, dtype)
    t.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * sigma + mean)
    return t


def _frequencies(vocab):
    """Words by rank: frequency falls as 1 / (rank + 2.7)."""
    f = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return f / f.sum()


def _offsets(case, seed):
    """Where the packed sequences start, and the end of the last one. Ragged: one of them empty."""
    n, rows = case["sequences"], case["rows"]
    if case["even"]:
        return [rows * i // n for i in range(n + 1)]
    r = random.Random(seed)
    part = [r.expovariate(1.0) + 0.05 for _ in range(n)]
    if n > 3:
        part[2] = 0.0
    at, total, out = 0.0, sum(part), [0]
    for p in part:
        at += p
        out.append(min(rows, int(rows * at / total + 0.5)))
    out[-1] = rows
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    op = case["op"]
    dtype = getattr(torch, case["dtype"])
    if op in ("embed", "embed_grad"):
        m, vocab, d = case["tokens"], case["vocab"], case["dim"]
        cdf = torch.from_numpy(np.cumsum(_frequencies(vocab))).cuda()
        u = torch.rand(m, generator=gen, device="cuda", dtype=torch.float64)
        tokens = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
        if op == "embed":
            s["table"] = _normal(gen, vocab, d, getattr(torch, case["table"]), 0.02)
            s["out"] = _padded(m, d, dtype)
        else:
            tokens[m - int(m * case["padded"]):] = 0  # the padding's token
            s["dy"] = _normal(gen, m, d, dtype, 0.1)
            s["dtable"] = torch.randn(vocab, d, generator=gen, device="cuda")
        s["tokens"] = tokens if case["wide"] else tokens.int()
    elif op in ("norm", "norm_grad"):
        m, d = case["rows"], case["cols"]
        s["x"] = _normal(gen, m, d, dtype, 1.0, 0.2)
        s["gamma"] = 1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")
        if op == "norm":
            s["beta"] = 0.1 * torch.randn(d, generator=gen, device="cuda") if case["beta"] else None
            s["y"] = _padded(m, d, dtype)
            s["mean"], s["rstd"] = (torch.empty(m, device="cuda") for _ in range(2))
        else:
            x = s["x"].double()  # what the forward pass left
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + 1e-5).rsqrt().float()
            s["dy"] = _normal(gen, m, d, dtype, 0.1)
            s["residual"] = _normal(gen, m, d, dtype, 0.1) if case["residual"] else None
            s["dx"] = _padded(m, d, dtype)
            s["dgamma"], s["dbeta"] = (torch.randn(d, generator=gen, device="cuda")
                                       for _ in range(2))
    elif op == "dropout":
        m, d = case["rows"], case["cols"]
        s["x"] = _normal(gen, m, d, dtype)
        s["residual"] = _normal(gen, m, d, dtype) if case["residual"] else None
        s["out"] = _padded(m, d, dtype)
        s["seed"] = 1000003 * seed + 17
        s["step"] = torch.tensor([seed % 1000 + 5], dtype=torch.int64, device="cuda")
    else:
        m, d, n = case["rows"], case["cols"], case["sequences"]
        s["ends"] = _offsets(case, seed)
        s["offsets"] = torch.tensor(s["ends"], dtype=torch.int64, device="cuda")
        s["x"] = _normal(gen, m, d, dtype)
        s["gate"] = _normal(gen, m, d, dtype, 1.5, 2.0)  # a memory of some ten rows
        s["h0"] = torch.randn(n, d, generator=gen, device="cuda") if case["state"] else None
        s["h_last"] = torch.empty(n, d, device="cuda")
        s["y"] = _padded(m, d, dtype)
        if op == "recur_train":
            s["dy"] = _normal(gen, m, d, dtype, 0.1)
            s["d_last"] = (torch.randn(n, d, generator=gen, device="cuda") * 0.1
                           if case["state"] else None)
            s["dx"], s["dgate"] = _padded(m, d, dtype), _padded(m, d, dtype)
            s["d_h0"] = torch.empty(n, d, device="cuda") if case["state"] else None
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The views and workspaces that a program with fixed buffers keeps."""
    import sparsified_gradient_compression_gb300 as dgc

    case, op = s["case"], s["case"]["op"]
    matrices = ("table", "out", "dy", "dtable", "x", "y", "residual", "dx", "gate", "h0", "h_last",
                "dgate", "d_h0", "d_last")
    vectors = ("tokens", "gamma", "beta", "dgamma", "dbeta")
    s["m"] = {k: None if s[k] is None else dgc.matrix(s[k]) for k in matrices if k in s}
    s["m"].update({k: None if s[k] is None else dgc.vector(s[k]) for k in vectors if k in s})
    size = 0
    if op == "embed_grad":
        size = dgc.dgc_embed_backward_workspace(case["tokens"], case["vocab"], case["dim"])
    elif op == "norm_grad":
        size = dgc.dgc_layer_norm_backward_workspace(case["rows"], case["cols"])
    elif op in ("recur", "recur_train"):
        size = dgc.dgc_recurrence_workspace(case["rows"], case["cols"])
        saved = dgc.dgc_recurrence_saved_rows(case["rows"])
        s["m"]["saved"] = None
        if op == "recur_train":
            s["saved"] = torch.empty(saved, case["cols"], device="cuda")
            s["m"]["saved"] = dgc.matrix(s["saved"])
    s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------------------- run
EPS = 1e-5
PADDING = 0


def _run_own(s):
    import sparsified_gradient_compression_gb300 as dgc

    case, m, st = s["case"], s["m"], s["status"]
    op = case["op"]
    if op == "embed":
        dgc.dgc_embed(m["table"], m["tokens"], case["scale"], m["out"], st)
        return {"out": s["out"]}
    if op == "embed_grad":
        dgc.dgc_embed_backward(m["tokens"], m["dy"], case["scale"],
                               PADDING if case["padded"] else None, m["dtable"],
                               case["accumulate"], st, s["ws"])
        return {"dtable": s["dtable"]}
    if op == "norm":
        dgc.dgc_layer_norm(m["x"], m["gamma"], m["beta"], EPS, m["y"], s["mean"], s["rstd"])
        return {k: s[k] for k in ("y", "mean", "rstd")}
    if op == "norm_grad":
        dgc.dgc_layer_norm_backward(m["dy"], m["x"], m["gamma"], s["mean"], s["rstd"],
                                    m["residual"], m["dx"], m["dgamma"], m["dbeta"],
                                    case["accumulate"], s["ws"])
        return {k: s[k] for k in ("dx", "dgamma", "dbeta")}
    if op == "dropout":
        dgc.dgc_dropout(m["x"], m["residual"], case["p"], s["seed"], s["step"], m["out"])
        return {"out": s["out"]}
    dgc.dgc_recurrence(m["x"], m["gate"], s["offsets"], m["h0"], m["y"], m["h_last"], m["saved"],
                       st, s["ws"])
    out = {"y": s["y"], "h_last": s["h_last"]}
    if op == "recur_train":
        dgc.dgc_recurrence_backward(m["dy"], m["x"], m["gate"], s["offsets"], m["h0"], m["saved"],
                                    m["d_last"], m["dx"], m["dgate"], m["d_h0"], st, s["ws"])
        out.update({k: s[k] for k in ("dx", "dgate", "d_h0") if s[k] is not None})
    return out


def _logical_shift(z, k):
    return (z >> k) & ((1 << (64 - k)) - 1)


def _mix(z):
    """SplitMix64's output function on int64 tensors, whose products wrap as unsigned ones do."""
    z = (z ^ _logical_shift(z, 30)) * (0xBF58476D1CE4E5B9 - (1 << 64))
    z = (z ^ _logical_shift(z, 27)) * (0x94D049BB133111EB - (1 << 64))
    return z ^ _logical_shift(z, 31)


GOLDEN = 0x9E3779B97F4A7C15 - (1 << 64)


def _signed(v):
    v &= (1 << 64) - 1
    return v - (1 << 64) if v >> 63 else v


def _threshold(p):
    return int(p * 65536.0 + 0.5)


def _mask(s, rows, cols):
    """What is kept: 16 random bits an entry, four entries of a row to a 64-bit word."""
    words = -(-cols // 4)
    key = _mix((s["step"] + 1) * GOLDEN + _signed(s["seed"]))
    word = torch.arange(1, rows * words + 1, device="cuda")
    word = _mix(word * GOLDEN + key).view(rows, words, 1)
    shift = torch.arange(0, 64, 16, device="cuda")
    bits = ((word >> shift) & 0xFFFF).view(rows, 4 * words)[:, :cols]
    return bits >= _threshold(s["case"]["p"])


def _forward_scan(s, x, a, keep):
    """h of every row by doubling: after a step of k rows, (a, b) of a row spans 2k rows."""
    start, seq = s["starts"]
    b = keep * x
    if s["h0"] is not None:
        b[start] += a[start] * s["h0"][seq]
    a = a.clone()
    a[start] = 0.0
    k = 1
    while k < s["longest"]:
        b[k:] = b[k:] + a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _sequence_rows(s):
    ends = s["ends"]
    full = [i for i in range(len(ends) - 1) if ends[i + 1] > ends[i]]
    s["longest"] = max(ends[i + 1] - ends[i] for i in full)
    dev = dict(dtype=torch.int64, device="cuda")
    seq = torch.tensor(full, **dev)
    s["starts"] = torch.tensor([ends[i] for i in full], **dev), seq
    s["lasts"] = torch.tensor([ends[i + 1] - 1 for i in full], **dev), seq


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return {"out": (s["table"][s["tokens"].long()].float() * case["scale"]).to(s["out"].dtype)}
    if op == "embed_grad":
        dy, tokens = s["dy"].float(), s["tokens"].long()
        if case["padded"]:
            dy = torch.where((tokens == PADDING)[:, None], torch.zeros_like(dy), dy)
        grad = torch.zeros_like(s["dtable"]).index_add_(0, tokens, dy) * case["scale"]
        if case["accumulate"]:
            s["dtable"] += grad
        else:
            s["dtable"].copy_(grad)
        return {"dtable": s["dtable"]}
    if op == "norm":
        x = s["x"].float()
        mean = x.sum(1) / x.shape[1]
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).sum(1) / x.shape[1] + EPS)
        y = d * rstd[:, None] * s["gamma"]
        if s["beta"] is not None:
            y = y + s["beta"]
        return {"y": y.to(s["y"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        x, dy, cols = s["x"].float(), s["dy"].float(), s["x"].shape[1]
        xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gamma"]
        c1, c2 = g.sum(1, keepdim=True) / cols, (g * xhat).sum(1, keepdim=True) / cols
        dx = (g - c1 - xhat * c2) * s["rstd"][:, None]
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        dgamma, dbeta = (dy * xhat).sum(0), dy.sum(0)
        if case["accumulate"]:
            s["dgamma"] += dgamma
            s["dbeta"] += dbeta
        else:
            s["dgamma"].copy_(dgamma)
            s["dbeta"].copy_(dbeta)
        return {"dx": dx.to(s["dx"].dtype), "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "dropout":
        x = s["x"].float()
        kept = 65536 - _threshold(case["p"])
        y = torch.where(_mask(s, *x.shape), x * (65536.0 / kept), torch.zeros_like(x))
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"out": y.to(s["out"].dtype)}
    if "starts" not in s:
        _sequence_rows(s)  # host arithmetic on the lengths, which a program has from its batch
    x, g = s["x"].float(), s["gate"].float()
    a, keep = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    h = _forward_scan(s, x, a, keep)
    last, seq = s["lasts"]
    h_last = torch.zeros_like(s["h_last"]) if s["h0"] is None else s["h0"].clone()
    h_last[seq] = h[last]
    out = {"y": h.to(s["y"].dtype), "h_last": h_last}
    if op == "recur_train":
        start, _ = s["starts"]
        before = torch.zeros_like(h)
        before[1:] = h[:-1]
        before[start] = 0.0 if s["h0"] is None else s["h0"][seq]
        dh = s["dy"].float()
        if s["d_last"] is not None:
            dh[last] += s["d_last"][seq]
        c = torch.zeros_like(a)
        c[:-1] = a[1:]
        c[last] = 0.0
        k = 1
        while k < s["longest"]:
            dh[:-k] = dh[:-k] + c[:-k] * dh[k:]
            c[:-k] = c[:-k] * c[k:]
            k *= 2
        out["dx"] = (dh * keep).to(s["dx"].dtype)
        out["dgate"] = (dh * (before - x) * a * keep).to(s["dgate"].dtype)
        if s["d_h0"] is not None:
            d_h0 = s["d_last"].clone()  # of an empty sequence: its last state is its first
            d_h0[seq] = a[start] * dh[start]
            out["d_h0"] = d_h0
    return out


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    w = {k: v.to(torch.float64) for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "embed":
        return {"out": torch.nn.functional.embedding(s["tokens"].long(), w["table"])
                * case["scale"]}
    if op == "embed_grad":
        grad = w["dtable"] if case["accumulate"] else torch.zeros_like(w["dtable"])
        order = torch.argsort(s["tokens"].long(), stable=True)
        words, counts = torch.unique_consecutive(s["tokens"].long()[order], return_counts=True)
        ends = counts.cumsum(0).tolist()
        at = 0
        for word, end in zip(words.tolist(), ends):
            if not (case["padded"] and word == PADDING):
                grad[word] += case["scale"] * w["dy"][order[at:end]].sum(0)
            at = end
        return {"dtable": grad}
    if op == "norm":
        x = w["x"]
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + EPS) * w["gamma"]
        return {"y": y + w["beta"] if case["beta"] else y, "mean": mean[:, 0],
                "rstd": (var[:, 0] + EPS) ** -0.5}
    if op == "norm_grad":
        out = {"dx": torch.empty_like(w["x"]), "dgamma": w["dgamma"], "dbeta": w["dbeta"]}
        if not case["accumulate"]:
            out["dgamma"], out["dbeta"] = (torch.zeros_like(w["dgamma"]) for _ in range(2))
        for at in range(0, case["rows"], 1024):  # the definition, differentiated
            x = w["x"][at:at + 1024].clone().requires_grad_(True)
            gamma = w["gamma"].clone().requires_grad_(True)
            beta = torch.zeros_like(gamma).requires_grad_(True)
            y = torch.nn.functional.layer_norm(x, x.shape[1:], gamma, beta, EPS)
            dx, dg, db = torch.autograd.grad(y, (x, gamma, beta), w["dy"][at:at + 1024])
            out["dx"][at:at + 1024] = dx
            out["dgamma"] += dg
            out["dbeta"] += db
        if case["residual"]:
            out["dx"] += w["residual"]
        return out
    if op == "dropout":
        m, d = case["rows"], case["cols"]

        def mix(z):
            z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
            z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
            return z ^ (z >> np.uint64(31))

        golden = np.array([0x9E3779B97F4A7C15], np.uint64)
        step = np.uint64(int(s["step"].item()))
        key = mix(golden * (step + np.uint64(1)) + np.uint64(s["seed"] % 2**64))
        lanes = -(-d // 4)
        words = mix(golden * np.arange(1, m * lanes + 1, dtype=np.uint64) + key)
        bits = words.astype("<u8").view("<u2").reshape(m, 4 * lanes)[:, :d]
        kept = torch.from_numpy(bits.astype(np.int32)).cuda() >= _threshold(case["p"])
        share = (65536 - _threshold(case["p"])) / 65536.0
        out = w["x"].div(share).masked_fill(~kept, 0.0)
        return {"out": out + w["residual"] if case["residual"] else out}
    return _exact_recurrence(case, s, w)


def _exact_recurrence(case, s, w):
    """Row after row of all sequences at once."""
    ends = torch.tensor(s["ends"], device="cuda")
    first, length = ends[:-1], ends[1:] - ends[:-1]
    longest = int(length.max())
    if longest * case["cols"] > 1 << 27 or longest > 1 << 16:
        return None
    x, a = w["x"], torch.sigmoid(w["gate"])
    keep = torch.sigmoid(-w["gate"])
    h = w["h0"].clone() if case["state"] else torch.zeros_like(w["h_last"])
    y, before = torch.empty_like(x), torch.empty_like(x)
    order = torch.argsort(length, descending=True, stable=True)
    sizes = torch.sort(length, descending=True).values.tolist()
    first, h = first[order], h[order]
    alive, steps = len(sizes), []
    for t in range(longest):
        while sizes[alive - 1] <= t:
            alive -= 1
        steps.append(alive)
        at = first[:alive] + t
        before[at] = h[:alive]
        h[:alive] = a[at] * h[:alive] + keep[at] * x[at]
        y[at] = h[:alive]
    h_last = torch.empty_like(h)
    h_last[order] = h
    out = {"y": y, "h_last": h_last}
    if case["op"] == "recur_train":
        d = w["d_last"][order] if case["state"] else torch.zeros_like(h)
        dx, dgate = torch.empty_like(x), torch.empty_like(x)
        for t in reversed(range(longest)):
            at = first[:steps[t]] + t
            g = d[:steps[t]] + w["dy"][at]
            dx[at] = g * keep[at]
            dgate[at] = g * (before[at] - x[at]) * a[at] * keep[at]
            d[:steps[t]] = g * a[at]
        out.update(dx=dx, dgate=dgate)
        if case["state"]:
            d_h0 = torch.empty_like(d)
            d_h0[order] = d
            out["d_h0"] = d_h0
    return out


# -------------------------------------------------------------------------------------- work
def _words_seen(case, count):
    """How many rows of the table a batch of count tokens meets."""
    return float(-np.expm1(count * np.log1p(-_frequencies(case["vocab"]))).sum())


def work(case):
    op, es = case["op"], BITS[case["dtype"]]
    if op == "embed":
        m, d = case["tokens"], case["dim"]
        seen = _words_seen(case, m)
        return {"bytes": int(m * (8 if case["wide"] else 4) + d * (seen * BITS[case["table"]]
                                                                   + m * es)), "flops": m * d}
    if op == "embed_grad":
        d = case["dim"]
        m = case["tokens"] - int(case["tokens"] * case["padded"])
        rows = 8 * _words_seen(case, m) if case["accumulate"] else 4 * case["vocab"]
        return {"bytes": int(case["tokens"] * (8 if case["wide"] else 4) + d * (m * es + rows)),
                "flops": 2 * m * d}
    n = case["rows"] * case["cols"]
    if op == "norm":  # x, y; the row's statistics; the weights
        return {"bytes": 2 * es * n + 8 * case["rows"] + 8 * case["cols"], "flops": 8 * n}
    if op == "norm_grad":
        return {"bytes": (3 + case["residual"]) * es * n + 8 * case["rows"] + 16 * case["cols"],
                "flops": 14 * n}
    if op == "dropout":
        return {"bytes": (2 + case["residual"]) * es * n, "flops": 2 * n}
    states = 4 * case["sequences"] * case["cols"]
    if op == "recur":  # x, gate, y
        return {"bytes": 3 * es * n + (2 if case["state"] else 1) * states, "flops": 8 * n}
    # and x, gate, dy, dx, dgate: the backward pass comes after the layers above, on its own read
    return {"bytes": 8 * es * n + (4 if case["state"] else 1) * states, "flops": 24 * n}
