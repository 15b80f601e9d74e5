"""The feed-forward calls' first use of a device, each case in a process of its own."""
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
import torch
import sparsified_gradient_compression_gb300 as dgc

dgc.lib()
gen = torch.Generator(device="cuda").manual_seed(1)

def rand(r, c, s=1.0):
    return (torch.randn(r, c, generator=gen, device="cuda") * s).bfloat16()

def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")
"""

OTHER_THREAD = SETUP + """
import threading

def calls():
    st, out = status_word(), []
    for m in (1, 3, 300):
        x, dy = rand(m, 64), rand(m, 64)
        wg, wu, wd = rand(128, 64), rand(128, 64), rand(64, 128)
        hidden, gate, up, dg, du = (rand(m, 128) for _ in range(5))
        y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(128, 64, device="cuda")
        a = dict(gate=(dgc.dgc_ffn_gate, x, wg, wu, dgc.ACT_SILU, hidden, gate, up, st),
                 down=(dgc.dgc_ffn_down, hidden, wd, x, y, st),
                 down_backward=(dgc.dgc_ffn_down_backward, dy, wd, gate, up, dgc.ACT_SILU, dg, du,
                                st),
                 gate_backward=(dgc.dgc_ffn_gate_backward, dg, du, wg, wu, dy, dx, st),
                 weight_grad=(dgc.dgc_ffn_weight_grad, dg, x, dw, False, st, None))
        out += [(m, name, *call) for name, call in a.items()]
    return out, st

todo, st = calls()
if WARM:
    for _, _, f, *args in todo:
        f(*args)
torch.cuda.synchronize()
errors = []

def call(m, name, f, *args):
    try:
        f(*args)
    except Exception as e:
        errors.append((m, name, str(e)))

for t in todo:  # a new thread for every call
    thread = threading.Thread(target=call, args=t)
    thread.start()
    thread.join()
torch.cuda.synchronize()
assert not errors, errors
assert dgc.dgc_read_status(st) == 0
"""


THREADS = SETUP + """
import threading

# shapes that the cost model cuts into clusters by what the device holds of them
sets = []
for m, n, k in ((100, 1024, 4096), (40, 512, 8192), (700, 1024, 4096), (256, 2048, 2048)) * 3:
    sets.append((rand(m, k), rand(n, k, k ** -0.5), torch.empty(m, n, dtype=torch.bfloat16,
                                                                device="cuda"),
                 torch.cuda.Stream(), status_word()))
torch.cuda.synchronize()
gate = threading.Barrier(len(sets))
errors = []

def first_call(s):
    try:
        with torch.cuda.stream(s[3]):
            gate.wait()
            dgc.dgc_ffn_down(s[0], s[1], None, s[2], s[4])
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=first_call, args=(s,)) for s in sets]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
for h, w, y, _, st in sets:
    again = torch.empty_like(y)
    dgc.dgc_ffn_down(h, w, None, again, st)
    assert dgc.dgc_read_status(st) == 0
    assert torch.equal(y, again)
"""


CAPTURE = SETUP + """
st = status_word()
x, wg, wu, wd = rand(300, 64), rand(128, 64, 0.1), rand(128, 64, 0.1), rand(64, 128, 0.1)
hidden, gate, up, dg, du = (rand(300, 128) for _ in range(5))
y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(128, 64, device="cuda")
odd = torch.zeros(300, 65, device="cuda").bfloat16()[:, :64]
odd.copy_(x)
long = rand(65536, 32)
ws = torch.empty(dgc.dgc_ffn_weight_grad_workspace(32, 32, 65536), dtype=torch.uint8, device="cuda")
assert ws.numel() > 0
dw2, one = torch.empty(32, 32, device="cuda"), torch.empty(1, 128, device="cuda").bfloat16()
nothing = torch.empty(0, 128, device="cuda").bfloat16()
first = {
    "one token": lambda: dgc.dgc_ffn_gate(x[:1], wg, wu, 0, one, None, None, st),
    "odd rows": lambda: dgc.dgc_ffn_gate(odd, wg, wu, 0, hidden, None, None, st),
    "odd weight gradient": lambda: dgc.dgc_ffn_weight_grad(dg, odd, dw, False, st, None),
    "no tokens": lambda: dgc.dgc_ffn_weight_grad(nothing, x[:0], dw, False, st, None),
}[FIRST]
torch.cuda.synchronize()
first()
torch.cuda.synchronize()

def step():
    dgc.dgc_ffn_gate(x, wg, wu, dgc.ACT_GELU, hidden, gate, up, st)
    dgc.dgc_ffn_down(hidden, wd, x, y, st)
    dgc.dgc_ffn_down_backward(x, wd, gate, up, dgc.ACT_GELU, dg, du, st)
    dgc.dgc_ffn_gate_backward(dg, du, wg, wu, x, dx, st)
    dgc.dgc_ffn_weight_grad(dg, x, dw, False, st, None)
    dgc.dgc_ffn_weight_grad(long, long, dw2, False, st, ws)
    return hidden, gate, up, y, dg, du, dx, dw, dw2

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = step()
for t in outs:
    t.fill_(7.0)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
for t in outs:
    t.fill_(7.0)
step()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
assert dgc.dgc_read_status(st) == 0
"""


def run(code):
    dgc.build()
    r = subprocess.run([sys.executable, "-c", code, ROOT], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("warm", [False, True])
def test_calls_from_threads_that_made_no_cuda_call_before(warm):
    run(OTHER_THREAD.replace("WARM", str(warm)))


def test_first_calls_from_several_threads():
    """The same bits as from calls one after the other, later."""
    run(THREADS)


@pytest.mark.parametrize("first", ["one token", "odd rows", "odd weight gradient", "no tokens"])
def test_capture_after_one_call_of_another_form(first):
    run(CAPTURE.replace("FIRST", repr(first)))
