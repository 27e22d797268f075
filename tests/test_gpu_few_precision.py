"""The few-token layer's activations keep both of their bf16 parts, on products that would
show the loss of the second.

a = silu(h) u is held as its bf16 rounding and the bf16 rounding of what that leaves: off by
2^-16 of a at most (half a step of each, 2^-8 2^-8).  Products of tensor-core sums and W_down
in which the first parts cancel leave an error of 2^-8 of a if the second part is lost.
GPU only."""
import pytest
import torch

from test_gpu_few import BF, HALF, call, sums

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 4), (3, 2), (4, 1), (5, 1), (8, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (64, 8), (40, 16)]


def routes(T, E, gen):
    """One expert a token, gate 1."""
    idx = torch.randint(0, E, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    return idx, torch.ones(T, 1, device="cuda")


@pytest.mark.parametrize("T,E", SHAPES, ids=str)
@pytest.mark.parametrize("f", [128, 384])
def test_second_parts_alone_are_left(moe_gpu, T, E, f):
    """h = 32 (silu(32) = 32 to 2^-40), u = 1 + p q 2^-14, so that a = 32 + p q 2^-9: p q of
    up to 225 are bits that its bf16 rounding (steps of 2^-2) does not have.  W_down takes an
    a of 32 away from each: out = p q 2^-9, a bf16 number.  All sums are exact.  The quotient
    of silu may be off by two last places, 2^-17 of each a; that the parts and the result
    are rounded by at most 2^-8 of themselves."""
    m, _ = moe_gpu
    d, half = 128, f // 2
    gen = torch.Generator(device="cuda").manual_seed(T * 100 + E + f)
    p = torch.randint(1, 16, (T,), generator=gen, device="cuda")
    q = torch.randint(1, 16, (E, half), generator=gen, device="cuda")
    x, wg, wu = torch.zeros(T, d, **BF), torch.zeros(E, f, d, **BF), torch.zeros(E, f, d, **BF)
    x[:, 0], x[:, 1] = 1.0, (p * 2.0 ** -7).to(torch.bfloat16)
    wg[:, :, 0], wu[:, :, 0] = 32.0, 1.0
    wu[:, :half, 1] = (q * 2.0 ** -7).to(torch.bfloat16)
    wd = torch.zeros(E, d, f, **BF)
    at = torch.arange(d, device="cuda")
    wd[:, at, at % half], wd[:, at, at % half + half] = 1.0, -1.0
    idx, gates = routes(T, E, gen)
    out, error = call(m, x, None, None, wg, wu, wd, 1, topk_idx=idx, gates=gates)
    want = p[:, None].double() * q[idx[:, 0].long()][:, at % half].double() * 2.0 ** -9
    assert error == 0
    assert ((out.double() - want).abs() <= 2 * 2.0 ** -17 + 2 * HALF * want).all()


@pytest.mark.parametrize("T,E", SHAPES, ids=str)
def test_differences_of_near_activations(moe_gpu, T, E):
    """Pairs of activations whose gate rows are equal and whose up rows nearly are, taken
    from one another by W_down, against 64 bits.  Each a is off by 2^-16 of itself (its
    parts), 2^-20 (silu: __expf is off by 2 + 1.2 |h| last places, |h| <= 4, the quotient by
    two) and what h and u are off by, the sums of test_gpu_few.  With the second part lost
    the error is about 2^-9.5 |a| sqrt(f) |w|, several times the bound."""
    m, _ = moe_gpu
    d, f = 128, 128
    half = f // 2
    gen = torch.Generator(device="cuda").manual_seed(T * 100 + E)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)
    x, wg, wu, wd = normal(T, d, scale=1.0), normal(E, f, d, scale=0.06), normal(E, f, d, scale=0.06), normal(E, d, f, scale=0.05)
    wg[:, half:] = wg[:, :half]
    wu[:, half:] = wu[:, :half]
    wu[:, half:, :4] *= 0.9375   # the difference of the pair, about 2^-7 of u
    wd[:, :, half:] = -wd[:, :, :half]
    idx, gates = routes(T, E, gen)
    out, error = call(m, x, None, None, wg, wu, wd, 1, topk_idx=idx, gates=gates)
    assert error == 0
    e = idx[:, 0].long()
    xd, g, u, w = x.double()[:, :, None], wg.double()[e], wu.double()[e], wd.double()[e]
    h, v = (g @ xd)[..., 0], (u @ xd)[..., 0]
    dh, dv = ((t.abs() @ xd.abs())[..., 0] * sums(d) for t in (g, u))
    assert h.abs().max() <= 4
    s = h * torch.sigmoid(h)
    a = s * v
    da = 1.1 * dh * (v.abs() + dv) + s.abs() * dv + (2.0 ** -16 + 2.0 ** -20) * a.abs()
    want = (w @ a[..., None])[..., 0]
    off = (w.abs() @ (da + (a.abs() + da) * sums(f))[..., None])[..., 0]
    assert ((out.double() - want).abs() <= off + HALF * (want.abs() + off)).all()
    # the first parts alone would not do
    first = (w @ a.to(torch.bfloat16).double()[..., None])[..., 0]
    assert ((first - want).abs() > off + HALF * (want.abs() + off)).any()
