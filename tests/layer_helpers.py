"""Buffers and 64-bit restatements for the operators around the feed-forward block.

Tolerances. u = half a step of the result's type, relative (binary32 2^-24, float16 2^-11, bfloat16
2^-8), with float16's and binary32's subnormal steps beside it; every result is rounded once. What
comes ahead of that rounding is binary32 arithmetic, bounded test by test in multiples of
E = 2^-24."""
from __future__ import annotations

import numpy as np
import torch

E = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -126, F16: 2.0 ** -25, BF16: 2.0 ** -126}


def buffer(rows, cols, dtype, pad=0, fill=float("nan")):
    """A view in a buffer filled with NaN. pad: a number of extra 8-entry steps from row to row, or
    "odd": an odd number of entries from row to row, the first row off every boundary, or "packed"."""
    if pad == "odd":
        ld = (cols + 1) | 1
        flat = torch.full((rows * ld + 2,), fill, dtype=dtype, device="cuda")
        return flat[1:1 + rows * ld].view(rows, ld)[:, :cols]
    if pad == "packed":
        return torch.full((rows, cols), fill, dtype=dtype, device="cuda")
    ld = -(-cols // 8) * 8 + 8 * pad
    return torch.full((max(rows, 1), max(ld, 8)), fill, dtype=dtype, device="cuda")[:rows, :cols]


def normal(gen, rows, cols, dtype, sigma=1.0, mean=0.0, pad=0):
    t = buffer(rows, cols, dtype, pad)
    t.copy_(torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float64) * sigma
            + mean)
    return t


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def workspace(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") if n else None


def whole(t):
    """Everything in the buffer that t is a view of."""
    return torch.empty(0, dtype=t.dtype, device=t.device).set_(t.untyped_storage())


def bits(t):
    return t.view({4: torch.int32, 2: torch.int16, 8: torch.int64}[t.element_size()])


def outside_is_untouched(t, fill=float("nan")):
    """What lies between and behind the rows still holds the fill."""
    flat = whole(t).clone()
    inside = flat.as_strided(t.shape, t.stride(), t.storage_offset())
    inside.fill_(fill)
    want = torch.full_like(flat, fill)
    assert torch.equal(bits(flat), bits(want))


def near(got, want, error=0.0):
    """got (rounded once to its type) against want in 64 bits; error: of the 32-bit arithmetic."""
    assert got.shape == want.shape, (got.shape, want.shape)
    want = want.to(got.device)
    error = error.to(got.device) if isinstance(error, torch.Tensor) else error
    tol = HALF[got.dtype] * want.abs() * (1 + 2.0 ** -10) + TINY[got.dtype] + 1.01 * error
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           got[bad][:4].tolist(), want[bad][:4].tolist())


# ------------------------------------------------------------------- the definitions, 64 bits
def dropout_kept(rows, cols, p, seed, step):
    """The generator by its definition, with numpy's 64-bit words."""
    g = 0x9E3779B97F4A7C15
    m = 2 ** 64 - 1

    def mix_int(z):
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        return z ^ (z >> 31)

    key = mix_int((seed + g * (1 + step)) & m)
    lanes = -(-cols // 4)
    z = (np.arange(1, rows * lanes + 1, dtype=np.uint64) * np.uint64(g) + np.uint64(key))
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    z = z ^ (z >> np.uint64(31))
    word = z.reshape(rows, lanes)
    col = np.arange(cols)
    draw = (word[:, col // 4] >> (16 * (col % 4)).astype(np.uint64)) & np.uint64(0xFFFF)
    return torch.from_numpy((draw >= np.uint64(int(p * 65536 + 0.5))))


def sigmoid(g):
    return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))),
                    np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def scan64(x, gate, ends, h0):
    """h of every row, h_{t-1} of every row, the last states; and the bound on a binary32 scan's
    error, as the same recurrence: a step's factor and summand are each off by at most 8 E (an
    exponential of 2 steps, a reciprocal and a division of 2, the additions and products), in
    whatever order they are joined; 64 E for the joints. x, gate, h0: numpy, binary64."""
    rows, cols = x.shape
    n = len(ends) - 1
    a, keep = sigmoid(gate), sigmoid(-gate)
    h, before, err = (np.full((rows, cols), np.nan) for _ in range(3))
    last, last_err = np.zeros((n, cols)), np.zeros((n, cols))
    for q in range(n):
        s = np.zeros(cols) if h0 is None else h0[q].copy()
        mag, e = np.abs(s), np.zeros(cols)
        for t in range(ends[q], ends[q + 1]):
            before[t] = s
            mag = a[t] * mag + keep[t] * np.abs(x[t])
            e = a[t] * e + 16 * E * mag
            s = a[t] * s + keep[t] * x[t]
            h[t], err[t] = s, e + 64 * E * mag
        last[q], last_err[q] = s, e + 64 * E * mag
    return h, before, err, last, last_err


def scan64_backward(x, gate, ends, h0, dy, d_last):
    """dx, dgate, d_h0, each with its bound."""
    rows, cols = x.shape
    n = len(ends) - 1
    a, keep = sigmoid(gate), sigmoid(-gate)
    _, before, h_err, _, _ = scan64(x, gate, ends, h0)
    dx, dgate, dx_err, dgate_err = (np.full((rows, cols), np.nan) for _ in range(4))
    d_h0, d_h0_err = np.zeros((n, cols)), np.zeros((n, cols))
    for q in range(n):
        u = np.zeros(cols) if d_last is None else d_last[q].copy()
        mag, e = np.abs(u), np.zeros(cols)
        for t in reversed(range(ends[q], ends[q + 1])):
            g = dy[t] + u
            mag = mag + np.abs(dy[t])
            e = e + 16 * E * mag
            ge = e + 64 * E * mag
            slope = (before[t] - x[t]) * a[t] * keep[t]
            size = (np.abs(before[t]) + np.abs(x[t])) * a[t] * keep[t]
            dx[t], dx_err[t] = g * keep[t], (ge + 16 * E * mag) * keep[t]
            dgate[t] = g * slope
            # the state ahead of the row: the error of the row before it
            prev = h_err[t - 1] if t > ends[q] else 0.0
            dgate_err[t] = (ge + 16 * E * mag) * size + (mag + ge) * prev * a[t] * keep[t]
            u, mag, e = a[t] * g, a[t] * mag, a[t] * e
        d_h0[q], d_h0_err[q] = u, e + 64 * E * mag
    return (dx, dx_err), (dgate, dgate_err), (d_h0, d_h0_err)
