"""The layer norm, AdamW and the layer for a few tokens set the device up on their first
call, and a graph may hold the first one: each test runs a child process.  GPU only."""
import pytest

from test_gpu_first_call import child

pytestmark = pytest.mark.gpu
NAMES = ["add_layer_norm", "add_layer_norm_bwd", "adamw", "adamw_8", "few"]

CALLS = '''
b = torch.randn(256, **F)
mean, db = torch.empty(4, **F), torch.empty(256, **F)
lnws = torch.empty(m.add_layer_norm_bwd_workspace(4, 256), **U)
grad = torch.randn(1000, **F)
start = torch.randn(1000, **F)
param, states = start.clone(), {n: m.adamw_states([start], n) for n in (32, 8)}
lists = {n: m.adamw_list([param], [grad], *states[n]) for n in (32, 8)}
shape = m.shape(4, 256, 8, 2, 256)
wr, wg, wu, wd = (torch.randn(*s, **F).mul_(0.1).bfloat16() for s in ((8, 256),) + ((8, 256, 256),) * 3)
fws = torch.zeros(m.few_workspace(shape), **U)
rand = torch.randn(4, 256, **F).bfloat16()

def add_layer_norm():
    m.add_layer_norm(rand, w, b, y, residual=x, h=h, mean=mean, rstd=r)
    return y
def add_layer_norm_bwd():
    m.add_layer_norm_bwd(rand, x, torch.zeros(4, **F), torch.ones(4, **F), w, dx=dx, dw=dw, db=db, ws=lnws)
    return torch.cat([dx.float(), dw[None], db[None]])
def step(bits):
    param.copy_(start)
    for s in states[bits]:
        for t in (s[0] if bits == 8 else s):
            t.zero_()
    m.adamw(lists[bits], lr=0.01, step=3, seed=5)
    return param
def adamw():
    return step(32)
def adamw_8():
    return step(8)
def few():
    m.forward_few(shape, rand, wr, None, wg, wu, wd, y, fws)
    return y
'''


@pytest.mark.parametrize("name", NAMES)
def test_first_call_without_init(name):
    child(CALLS + f'''
first = {name}().clone()
m.init()
again = {name}()
torch.cuda.synchronize()
assert torch.equal(first, again) and first.float().abs().sum() > 0
''')


@pytest.mark.parametrize("name", NAMES)
def test_first_call_in_a_graph(name):
    child(CALLS + f'''
m.init()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = {name}()
graph.replay()
first = held.clone()
graph.replay()
again = held.clone()
other = {name}()
torch.cuda.synchronize()
assert torch.equal(first, other) and torch.equal(again, other) and first.float().abs().sum() > 0
''')


def test_first_call_within_a_capture_is_refused():
    child(CALLS + '''
graph, seen = torch.cuda.CUDAGraph(), []
with torch.cuda.graph(graph):
    dx.zero_()
    for call in (add_layer_norm, few, lambda: m.adamw(lists[32], lr=0.01, step=1)):
        try:
            call()
        except m.MoEError as e:
            seen.append(e.code)
assert seen == [-5] * 3, seen
graph.replay()
few()
torch.cuda.synchronize()
assert (y != 0).any() and (dx == 0).all()
''')
