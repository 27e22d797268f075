"""Pins of the block operators' oracle (oracle/block_oracle.py).  CPU only."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    """The known-answer vectors published with the generator."""
    got = B.philox4x32_10(np.array([counter], dtype=np.uint64), key)[0]
    assert tuple(int(v) for v in got) == want


def test_keep_mask_rate_and_independence():
    p, rows, cols = 0.3, 400, 1003
    m = B.keep_mask(rows, cols, p, seed=7, offset=5)
    n = rows * cols
    assert abs(m.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)
    other = B.keep_mask(rows, cols, p, seed=7, offset=6)
    # two masks agree where both keep or both drop: p^2 + (1-p)^2 of the places
    agree = p * p + (1 - p) ** 2
    assert abs((m == other).mean() - agree) < 5 * np.sqrt(agree * (1 - agree) / n)
    assert np.array_equal(m[:3, :17], B.keep_mask(3, 17, p, 7, 5))   # of the place alone


def test_dropout_edges():
    x = np.array([[np.nan, 1.0, -2.0, np.inf]])
    assert np.array_equal(B.dropout(x, 0.0, 1, 2), x, equal_nan=True)
    assert np.array_equal(B.dropout(x, 1.0, 1, 2), np.zeros_like(x))


@pytest.mark.parametrize("residual,p", [(True, 0.0), (False, 0.0), (True, 0.4)])
def test_norm_backward_is_the_gradient(residual, p):
    """Against torch float64 autograd and against central differences."""
    rng = np.random.default_rng(3)
    rows, d, eps = 5, 24, 1e-3
    x, res, w = rng.standard_normal((rows, d)), rng.standard_normal((rows, d)), rng.standard_normal(d)
    dy, dres = rng.standard_normal((rows, d)), rng.standard_normal((rows, d))
    r0 = res if residual else None

    def loss(x, res, w):
        h, y, _ = B.add_norm(x, res if residual else None, w, eps, p, 11, 1)
        return (y * dy).sum() + (h * dres).sum()

    h, _, rstd = B.add_norm(x, r0, w, eps, p, 11, 1)
    dh, dx, dw = B.add_norm_bwd(dy, h, rstd, w, dres, p, 11, 1)
    scale = torch.from_numpy(B.dropout(np.ones_like(x), p, 11, 1))
    tx, tr, tw = (torch.from_numpy(a).requires_grad_() for a in (x, res, w))
    th = tx * scale + (tr if residual else 0.0)
    ty = th * torch.rsqrt(th.square().mean(-1, keepdim=True) + eps) * tw
    ((ty * torch.from_numpy(dy)).sum() + (th * torch.from_numpy(dres)).sum()).backward()
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-11, atol=1e-12)
    if residual:
        np.testing.assert_allclose(dh, tr.grad.numpy(), rtol=1e-11, atol=1e-12)
    step = 1e-5
    for arr, grad, at in ((x, dx, (2, 7)), (x, dx, (4, 23)), (w, dw, (9,))):
        a, b = arr.copy(), arr.copy()
        a[at] += step
        b[at] -= step
        up, down = ((loss(v, res, w) if arr is x else loss(x, res, v)) for v in (a, b))
        assert abs((up - down) / (2 * step) - grad[at]) < 1e-7 * max(1, abs(grad[at]))


def test_w4_round_trip():
    rng = np.random.default_rng(4)
    w = rng.standard_normal((6, 128)) * 0.02
    w[2, 32:64] = 0
    codes, s = B.w4_quantize(w, 32, lambda v: v)
    v = B.w4_values(codes, s)
    assert np.abs(v - w).max() <= s.max() / 2 + 1e-15
    assert np.all(codes[2, 32:64] == 8) and s[2, 1] == 0 and np.all(v[2, 32:64] == 0)
    packed = B.w4_pack(codes)
    assert np.array_equal(packed & 15, codes[:, 0::2]) and np.array_equal(packed >> 4, codes[:, 1::2])


def test_experts_route_by_route():
    """Against a batched restatement; routes without an expert add nothing."""
    rng = np.random.default_rng(5)
    T, d, E, k, f = 7, 16, 4, 2, 8
    x, logits = rng.standard_normal((T, d)), rng.standard_normal((T, E))
    idx = np.argsort(-logits, 1)[:, :k]
    g = rng.random((T, k))
    wg, wu, wd = (rng.standard_normal(s) for s in ((E, f, d), (E, f, d), (E, d, f)))
    got = B.experts(x, idx, g, wg, wu, wd)
    want = np.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            a, b = x[t] @ wg[e].T, x[t] @ wu[e].T
            want[t] += g[t, j] * ((a / (1 + np.exp(-a)) * b) @ wd[e].T)
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-12)
    assert np.all(B.experts(x, np.full((T, k), -1), g, wg, wu, wd) == 0)
