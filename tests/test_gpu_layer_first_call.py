"""The first calls of a process, captured into a graph without a call before them, and two
graphs replayed at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import block_sparse_attention_tsr_gb300 as tsr
tsr.lib()
BF = torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
x, w, b, dy, nw = rand(1, 300, 256), rand(512, 256), rand(512), rand(1, 4, 300, 128), torch.ones(128, device="cuda")
few, dfew = rand(1, 3, 256), rand(1, 3, 512)

def step():
    h, pre = tsr.tsr_linear(x, w, b, activation="silu", heads=4, pre=True)
    y = tsr.tsr_norm_rope(h, nw, (44, 42, 42), grid=(3, 10, 10))
    dh, dn = tsr.tsr_norm_rope_backward(dy, h, nw, (44, 42, 42), grid=(3, 10, 10))
    z = tsr.tsr_linear(few, w, b)
    return [h, y, dh, dn, z, *tsr.tsr_linear_backward(dh, x, w, activation="silu", pre=pre),
            *tsr.tsr_linear_backward(dfew, few, w)]

torch.cuda.synchronize()
graphs, got = [], []
for _ in range(2):
    graphs.append(torch.cuda.CUDAGraph())
    with torch.cuda.graph(graphs[-1]):
        got.append(step())
streams = [torch.cuda.Stream() for _ in range(2)]
for _ in range(20):
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
tsr.tsr_linear_device_status()
assert all(torch.equal(a, c) for outs in got for a, c in zip(outs, want))
assert all(torch.isfinite(t).all() for t in want)
print("same")
"""


def test_first_calls_captured_and_two_graphs_at_once():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


THREADS = """
import threading
import torch
import block_sparse_attention_tsr_gb300 as tsr
tsr.lib()
BF = torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
x, w, b, dy, nw = rand(1, 300, 256), rand(512, 256), rand(512), rand(1, 4, 300, 128), torch.ones(128, device="cuda")
few, dfew, wide, dwide = rand(1, 3, 256), rand(1, 3, 512), rand(1, 900, 264), rand(1, 900, 512)
ww = rand(512, 264)

def step():
    h, pre = tsr.tsr_linear(x, w, b, activation="silu", heads=4, pre=True)
    y = tsr.tsr_norm_rope(h, nw, (44, 42, 42), grid=(3, 10, 10))
    dh, dn = tsr.tsr_norm_rope_backward(dy, h, nw, (44, 42, 42), grid=(3, 10, 10))
    z = tsr.tsr_linear(few, w, b)
    return [h, y, dh, dn, z, tsr.tsr_linear(wide, ww), *tsr.tsr_linear_backward(dh, x, w, activation="silu", pre=pre),
            *tsr.tsr_linear_backward(dfew, few, w), *tsr.tsr_linear_backward(dwide, wide, ww)]

torch.cuda.synchronize()
start, got = threading.Barrier(4), [None] * 4

def run(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        got[i] = step()
        torch.cuda.current_stream().synchronize()

threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
for t in threads: t.start()
for t in threads: t.join()
want = step()
tsr.tsr_linear_device_status()
assert all(torch.isfinite(t).all() for t in want)
assert all(torch.equal(a, c) for outs in got for a, c in zip(outs, want))
print("same")
"""


def test_first_calls_of_four_threads():
    r = subprocess.run([sys.executable, "-c", THREADS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_first_call_is_the_status():
    """Before anything else has set up the device."""
    code = "import block_sparse_attention_tsr_gb300 as tsr; tsr.tsr_linear_device_status(); print('fine')"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]
