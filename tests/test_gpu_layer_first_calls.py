"""First calls of the operators around the feed-forward block: captured with no call before, and from
threads that made no CUDA call before, each in a process of its own."""
import os
import subprocess
import sys

import pytest

import sparsified_gradient_compression_gb300 as dgc

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys
sys.path.insert(0, sys.argv[1])
import threading
import torch
import sparsified_gradient_compression_gb300 as dgc

dgc.lib()
m, d, vocab = 500, 72, 90
gen = torch.Generator(device="cuda").manual_seed(1)

def rand(*s, dtype=torch.bfloat16):
    return torch.randn(*s, generator=gen, device="cuda").to(dtype)

f32 = torch.float32
table, dy, x, gate = rand(vocab, d), rand(m, d), rand(m, d), rand(m, d)
tokens = torch.randint(0, vocab, (m,), generator=gen, device="cuda")
gamma, mean, rstd = rand(d, dtype=f32), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
off = torch.tensor([0, 100, m], device="cuda")
saved = torch.empty(dgc.dgc_recurrence_saved_rows(m), d, device="cuda")
outs = [torch.empty(m, d, dtype=torch.bfloat16, device="cuda") for _ in range(7)]
dgamma, dbeta, dtable = rand(d, dtype=f32), rand(d, dtype=f32), rand(vocab, d, dtype=f32)
st = torch.zeros(1, dtype=torch.int32, device="cuda")
ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()

calls = [
    lambda: dgc.dgc_embed(table, tokens, 2.0, outs[0], st),
    lambda: dgc.dgc_embed_backward(tokens, dy, 2.0, None, dtable, False, st, ws),
    lambda: dgc.dgc_layer_norm(x, gamma, None, 1e-5, outs[1], mean, rstd),
    lambda: dgc.dgc_layer_norm_backward(dy, x, gamma, mean, rstd, None, outs[2], dgamma, dbeta,
                                        False, ws),
    lambda: dgc.dgc_dropout(x, None, 0.5, 3, None, outs[3]),
    lambda: dgc.dgc_recurrence(x, gate, off, None, outs[4], None, saved, st, ws),
    lambda: dgc.dgc_recurrence_backward(dy, x, gate, off, None, saved, None, outs[5], outs[6], None,
                                        st, ws),
]
results = outs + [dgamma, dbeta, dtable, mean, rstd]
"""

CHECK = """
torch.cuda.synchronize()
got = [t.clone() for t in results]
for t in results:
    t.fill_(7.0)
for c in calls:
    c()
assert all(torch.equal(a, b) for a, b in zip(got, results))
assert dgc.dgc_read_status(st) == 0
"""

CAPTURE = SETUP + """
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for c in calls:
        c()
for t in results:
    t.fill_(7.0)
graph.replay()
""" + CHECK

THREADS = SETUP + """
errors = []

def one(c):
    try:
        c()
    except Exception as e:
        errors.append(e)

for c in calls:  # a new thread for every call, one behind the other
    t = threading.Thread(target=one, args=(c,))
    t.start()
    t.join()
assert not errors, errors
""" + CHECK


@pytest.mark.parametrize("code", [CAPTURE, THREADS], ids=["captured", "threads"])
def test_first_calls(code):
    dgc.build()
    r = subprocess.run([sys.executable, "-c", code, ROOT], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
