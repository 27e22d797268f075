"""The operators around the layer set the device up on their first call: a program
that never calls init() gets the results of one that does.  Each test runs a child
process, since the fixture of the other tests has initialised this one.  GPU only."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = '''
import torch
import moe_expert_layer_softmax_gb300 as m
torch.manual_seed(3)
B, F = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")
U = dict(dtype=torch.uint8, device="cuda")
x, w = torch.randn(4, 256, **F).bfloat16(), torch.ones(256, **F)
y, h, dx = torch.empty(4, 256, **B), torch.empty(4, 256, **B), torch.empty(4, 256, **B)
r, dw = torch.empty(4, **F), torch.empty(256, **F)
W = torch.randn(256, 256, **F).bfloat16()
q, s, full = torch.empty(256, 128, **U), torch.empty(256, 4, **B), torch.empty(256, 256, **F)
idx, g = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, **F)

def add_norm():
    m.add_norm(x, w, y, residual=x, h=h, rstd=r)
    return y
def add_norm_bwd():
    ws = torch.empty(m.add_norm_bwd_workspace(4, 256), **U)
    m.add_norm_bwd(x, x, torch.ones(4, **F), w, dx=dx, dw=dw, ws=ws)
    return torch.cat([dx.float(), dw[None]])
def dropout():
    m.dropout(x, y, 0.5, 7)
    return y
def quantize_w4():
    m.quantize_w4(W, q, s)
    return q
def dequantize_w4():
    m.dequantize_w4(torch.full((256, 128), 0x5B, **U), torch.ones(256, 4, **B), full)
    return full
def matvec_w4():
    m.matvec_w4(x, torch.full((256, 128), 0x5B, **U), torch.ones(256, 4, **B), y)
    return y
def experts_w4():
    e = {}
    for n in ("gate", "up", "down"):
        # columns of 4 and -3 in turn (of 3 and -3, the sum over equal activations is zero)
        e[n + "_q"], e[n + "_s"] = torch.full((1, 256, 128), 0x5C, **U), torch.full((1, 256, 4), 0.01, **B)
    m.experts_w4(x, idx, g, e, y, torch.zeros(m.experts_w4_workspace(4, 256, 1, 1, 256), **U))
    return y
'''


def child(tail):
    from moe_expert_layer_softmax_gb300 import _build
    _build.build()
    p = subprocess.run([sys.executable, "-c", CALLS + tail], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
    return p.stdout


@pytest.mark.parametrize("name", ["add_norm", "add_norm_bwd", "dropout", "quantize_w4", "dequantize_w4",
                                  "matvec_w4", "experts_w4"])
def test_first_call_without_init(name):
    child(f'''
first = {name}().clone()
m.init()
again = {name}()
torch.cuda.synchronize()
assert torch.equal(first, again) and first.float().abs().sum() > 0
''')


def test_first_call_within_a_capture_is_refused():
    """Setting a device up is no part of a graph: the call refuses as before, the
    capture goes on, and the next call outside one sets the device up."""
    child('''
graph, seen = torch.cuda.CUDAGraph(), []
with torch.cuda.graph(graph):
    y.zero_()
    try:
        dropout()
    except m.MoEError as e:
        seen.append(e.code)
assert seen == [-5], seen
graph.replay()
dropout()
torch.cuda.synchronize()
assert (y != 0).any()
''')


def test_first_call_on_a_capturing_stream_given_by_hand():
    child('''
side, graph, seen = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side):
    graph.capture_begin()
for stream in (side, side.cuda_stream):
    try:
        m.dropout(x, y, 0.5, 7, stream=stream)
    except m.MoEError as e:
        seen.append(e.code)
with torch.cuda.stream(side):
    y.zero_()
    graph.capture_end()
assert seen == [-5, -5], seen
dropout()
''')
