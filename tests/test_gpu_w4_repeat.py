"""The same call of the 4-bit experts gives the same bits, whatever the order in
which a block's warps find an expert's routes: shapes whose experts have more routes
than a round serves, with rounds of sixteen and a shorter last one.  GPU only."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,E,k,f,group", [
    (64, 1536, 8, 2, 1024, 64),    # about sixteen routes an expert
    (64, 2048, 8, 4, 1408, 128),   # 32
    (22, 512, 1, 1, 512, 32),      # sixteen and six
    (40, 256, 2, 1, 256, 128),
], ids=str)
def test_repeated_calls_give_the_same_bits(moe_gpu, T, d, E, k, f, group):
    m, dev = moe_gpu
    rng = np.random.default_rng(T + f)
    w = {}
    for n, shape in (("gate", (E, f, d)), ("up", (E, f, d)), ("down", (E, d, f))):
        w[n + "_q"] = torch.from_numpy(B.w4_pack(rng.integers(0, 16, shape).astype(np.uint8))).to(dev)
        w[n + "_s"] = torch.from_numpy(rng.random((*shape[:-1], shape[-1] // group)) * 0.1 / np.sqrt(shape[-1])).bfloat16().to(dev)
    x = torch.from_numpy(rng.standard_normal((T, d))).bfloat16().to(dev)
    idx = torch.from_numpy(np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32).copy()).to(dev)
    gates = torch.from_numpy(rng.random((T, k))).float().to(dev)
    out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(m.experts_w4_workspace(T, d, E, k, f), dtype=torch.uint8, device=dev)
    first = None
    for _ in range(200):
        m.experts_w4(x, idx, gates, w, out, ws)
        now = (out.clone(), ws.clone())   # ws: the 32-bit sums of each route before they are joined
        if first is None:
            first = now
        assert torch.equal(now[0], first[0]) and torch.equal(now[1], first[1])
    assert m.read_error(ws) == 0
