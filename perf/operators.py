"""Cases of the operators that stand around the MoE expert layer in a transformer block.

Four operators: the residual addition with the root-mean-square norm (and its
backward), dropout from a counter-based generator, matrix-vector products with
4-bit weights, and the SwiGLU experts on 4-bit weights for a few tokens.  Each
case runs in a plain form (elementary torch operations in 32 bits, rounded once
at the end) or, with `own` set, through the library's entry points.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
M32 = 0xFFFFFFFF
WIDTHS = [128, 256, 384, 512, 640, 768, 896, 1024, 1408, 1536, 2048, 2816, 4096, 5632, 8192]   # whole 128-column blocks


def listed():
    return [
        # decode step of four sequences: the norm before the layer, latency counts
        dict(name="norm decode 4x4096", op="norm", rows=4, d=4096, dtype="bf16", res="bf16", p=0.0, out="y"),
        # training forward of the 8192-token layer: bf16 stream
        dict(name="norm 8192x2048", op="norm", rows=8192, d=2048, dtype="bf16", res="bf16", p=0.0, out="y"),
        # training forward of the MXFP8 layer's block: residual dropout, 8-bit output
        # with its dequantised copy for the weight gradients
        dict(name="norm mxfp8 32768x4096", op="norm", rows=32768, d=4096, dtype="bf16", res="bf16", p=0.1, out="mx"),
        # a width that no vector divides, fp16 activations on an fp32 stream
        dict(name="norm odd 777x1001", op="norm", rows=777, d=1001, dtype="f16", res="f32", p=0.1, out="y"),
        # training backward of the 8192-token layer
        dict(name="norm bwd 8192x2048", op="norm_bwd", rows=8192, d=2048, dtype="bf16", res="bf16", p=0.0),
        # training backward of the largest block: fp32 stream, residual dropout
        dict(name="norm bwd 32768x4096", op="norm_bwd", rows=32768, d=4096, dtype="bf16", res="f32", p=0.1),
        # dropout of the layer's output (forward, and the same call on the gradient)
        dict(name="dropout 16384x2048", op="dropout", rows=16384, d=2048, dtype="bf16", p=0.1),
        # an odd fp32 matrix
        dict(name="dropout odd 1000x1407", op="dropout", rows=1000, d=1407, dtype="f32", p=0.25),
        # one token through a square projection
        dict(name="matvec 1 4096x4096", op="matvec", m=1, n=4096, k=4096, group=128, dtype="bf16"),
        # eight sequences through an output projection with a ragged row count, small groups, fp16
        dict(name="matvec 8 20011x2048", op="matvec", m=8, n=20011, k=2048, group=32, dtype="f16"),
        # one token through the experts of the largest layer
        dict(name="experts 1 of 64x8", op="experts", t=1, d=4096, f=2048, e=64, top=8, group=128, dtype="bf16"),
        # a batch of 64 sequences through the layer with d_ff 1408: every expert is read
        dict(name="experts 64 of 64x4", op="experts", t=64, d=2048, f=1408, e=64, top=4, group=64, dtype="bf16"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "dropout", "matvec", "experts"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    p = rng.choice([0.0, rng.randint(1, 50) / 100])
    if op in ("norm", "norm_bwd", "dropout"):
        rows = log_int(rng, 1, 32768)
        d = log_int(rng, 64, 8192)
        out = "y"
        if rng.random() < 0.6:
            d = rng.choice(WIDTHS)
            if dtype == "bf16" and rng.random() < 0.5:
                out = "mx"
        while rows * d > 16384 * 4096:   # wide types stay below the largest listed case
            rows = max(1, rows // 2)
        if op == "norm":
            return dict(op=op, rows=rows, d=d, dtype=dtype, res=rng.choice([dtype, "f32"]), p=p, out=out)
        if op == "norm_bwd":
            return dict(op=op, rows=rows, d=d, dtype=dtype, res=rng.choice([dtype, "f32"]), p=p)
        return dict(op=op, rows=rows, d=d, dtype=dtype, p=max(p, 0.01))
    dtype = rng.choice(["bf16", "f16"])
    group = rng.choice([32, 64, 128])
    if op == "matvec":
        return dict(op=op, m=log_int(rng, 1, 64), n=log_int(rng, 64, 32768),
                    k=rng.choice(WIDTHS), group=group, dtype=dtype)
    e = rng.choice([8, 32, 64])
    return dict(op=op, t=log_int(rng, 1, 64), d=128 * rng.randint(4, 16), f=128 * rng.randint(2, 11), e=e,
                top=rng.choice([1, 2, 4, 8]), group=group, dtype=dtype)


# ------------------------------------------------------------------ inputs
def w4(gen, shape, group, dtype):
    """4-bit weights of N(0, 0.02^2) values: codes (value + 8, two a byte, low
    nibble first) and one scale a group of columns."""
    w = torch.randn(shape, generator=gen, device="cuda").mul_(0.02).unflatten(-1, (-1, group))
    s = (w.abs().amax(-1) / 7).to(dtype)
    c = torch.round(w / s.float().unsqueeze(-1)).clamp_(-8, 7).add_(8).to(torch.uint8).flatten(-2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    st = dict(op=op, case=case, seed=(int(seed) * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF, offset=int(seed) % 1000)
    if op in ("norm", "norm_bwd", "dropout"):
        rows, d = case["rows"], case["d"]
        st["p"] = case["p"]
        if op == "dropout":
            st["x"] = normal(rows, d)
            st["y"] = torch.empty_like(st["x"])
            return st
        rt = DT[case["res"]]
        st["weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
        if op == "norm":
            st["x"] = normal(rows, d)
            st["residual"] = normal(rows, d, scale=2.0, dtype=rt)
            st["h"] = torch.empty_like(st["residual"])
            st["rstd"] = torch.empty(rows, device="cuda")
            if case["out"] == "mx":   # buffers of whole 128-row tiles, as the MXFP8 GEMMs read them
                pad = (rows + 127) // 128 * 128
                st["y_q"] = torch.empty(pad, d, dtype=torch.uint8, device="cuda")
                st["y_scales"] = torch.empty(pad * d // 32, dtype=torch.uint8, device="cuda")
                st["y_dq"] = torch.empty(pad, d, dtype=dt, device="cuda")
            else:
                st["y"] = torch.empty_like(st["x"])
            return st
        st["dy"] = normal(rows, d)
        st["h"] = normal(rows, d, scale=2.0, dtype=rt)
        st["dres"] = normal(rows, d, dtype=rt)
        st["rstd"] = (st["h"].double().square().mean(-1) + EPS).rsqrt().float()
        st["dh"] = torch.empty_like(st["h"])
        st["dx"] = torch.empty_like(st["dy"])
        st["dw"] = torch.empty(d, device="cuda")
        st["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        return st
    g = case["group"]
    if op == "matvec":
        st["x"] = normal(case["m"], case["k"])
        st["q"], st["scales"] = w4(gen, (case["n"], case["k"]), g, dt)
        st["y"] = torch.empty(case["m"], case["n"], dtype=dt, device="cuda")
        return st
    t, d, f, e, top = (case[n] for n in ("t", "d", "f", "e", "top"))
    st["x"] = normal(t, d)
    logits, idx = torch.randn(t, e, generator=gen, device="cuda").topk(top, -1)
    st["topk_idx"] = idx.to(torch.int32)
    st["gates"] = torch.softmax(logits, -1)
    st["w"] = {}
    for name, shape in (("gate", (e, f, d)), ("up", (e, f, d)), ("down", (e, d, f))):
        st["w"][name + "_q"], st["w"][name + "_s"] = w4(gen, shape, g, dt)
    st["out"] = torch.empty(t, d, dtype=dt, device="cuda")
    st["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def keep_mask(rows, cols, p, seed, offset):
    """Philox4x32-10: eight 16-bit numbers for each eight neighbouring columns of a row."""
    c = [torch.arange((cols + 7) // 8, device="cuda")[None, :], torch.arange(rows, device="cuda")[:, None],
         torch.tensor(offset & M32, device="cuda"), torch.tensor(offset >> 32, device="cuda")]
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & M32) ^ c[1] ^ k0, b & M32, (a >> 32 & M32) ^ c[3] ^ k1, a & M32]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    u = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], -1).flatten(1)[:, :cols]
    return u >= threshold(p)


def threshold(p):
    """The keep probability is a multiple of 2^-16."""
    return int(math.floor(p * 65536 + 0.5))


def keep_scale(p):
    return 65536 / (65536 - threshold(p))


def drop(v, p, seed, offset):
    """v (32 bits) with dropped places at zero and the others scaled up."""
    if p == 0:
        return v
    return torch.where(keep_mask(*v.shape, p, seed, offset), v * keep_scale(p), 0.0)


def mx_values(v):
    """The values that E4M3 codes with one power-of-two scale a 32 columns stand for."""
    b = v.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    s = (e - torch.where(m <= 0.875, 9, 8)).clamp(-127, 127) * (m > 0)
    q = torch.ldexp(b, -s).clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.ldexp(q.float(), s).flatten(-2)


def w4_values(q, s):
    """Codes and group scales to fp32 weights."""
    c = torch.stack([q & 15, q >> 4], -1).flatten(-2).float() - 8
    return (c.unflatten(-1, (s.shape[-1], -1)) * s.float().unsqueeze(-1)).flatten(-2)


def plain(st):
    op, case = st["op"], st["case"]
    if op == "dropout":
        return {"y": drop(st["x"].float(), st["p"], st["seed"], st["offset"]).to(st["x"].dtype)}
    if op == "norm":
        h = (st["residual"].float() + drop(st["x"].float(), st["p"], st["seed"], st["offset"])).to(st["residual"].dtype)
        v = h.float()
        rstd = torch.rsqrt(v.square().mean(-1) + EPS)
        y = v * rstd[:, None] * st["weight"].float()
        y = mx_values(y) if case["out"] == "mx" else y
        return {"h": h, "y": y.to(st["x"].dtype), "rstd": rstd}
    if op == "norm_bwd":
        h, dy, r = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
        g = dy * st["weight"].float()
        dh = st["dres"].float() + r * (g - h * (r * r * (g * h).mean(-1, keepdim=True)))
        dx = drop(dh, st["p"], st["seed"], st["offset"])
        return {"dh": dh.to(st["dh"].dtype), "dx": dx.to(st["dx"].dtype), "dw": (dy * (h * r)).sum(0)}
    if op == "matvec":
        return {"y": (st["x"].float() @ w4_values(st["q"], st["scales"]).T).to(st["x"].dtype)}
    x, idx, w = st["x"].float(), st["topk_idx"].long(), st["w"]
    n = {k: v for k, v in w.items()}
    t, top = idx.shape
    if t * top < case["e"]:   # fewer routes than experts: only the routed experts' weights
        n = {k: v[idx.flatten()] for k, v in w.items()}
        x = x.repeat_interleave(top, 0)[:, :, None]
        h, u = (w4_values(n[a + "_q"], n[a + "_s"]) @ x for a in ("gate", "up"))
        y = (w4_values(n["down_q"], n["down_s"]) @ (h / (1 + torch.exp(-h)) * u))[..., 0]
        return {"out": (y.unflatten(0, (t, top)) * st["gates"][..., None]).sum(1).to(st["x"].dtype)}
    gate = torch.zeros(t, case["e"], device="cuda").scatter_(1, idx, st["gates"])
    h, u = (x @ w4_values(n[a + "_q"], n[a + "_s"]).transpose(1, 2) for a in ("gate", "up"))
    a = h / (1 + torch.exp(-h)) * u * gate.T[:, :, None]
    return {"out": (a @ w4_values(n["down_q"], n["down_s"]).transpose(1, 2)).sum(0).to(st["x"].dtype)}


def run(st):
    if not own:
        return plain(st)
    import moe_expert_layer_softmax_gb300 as moe
    op = st["op"]
    if op == "dropout":
        moe.dropout(st["x"], st["y"], st["p"], st["seed"], st["offset"])
        return {"y": st["y"]}
    if op == "norm":
        if "y_q" in st:
            moe.add_norm(st["x"], st["weight"], None, residual=st["residual"], h=st["h"], rstd=st["rstd"], eps=EPS,
                         p=st["p"], seed=st["seed"], offset=st["offset"], y_q=st["y_q"], y_scales=st["y_scales"],
                         y_dq=st["y_dq"])
            return {"h": st["h"], "y": st["y_dq"][:st["x"].shape[0]], "rstd": st["rstd"]}
        moe.add_norm(st["x"], st["weight"], st["y"], residual=st["residual"], h=st["h"], rstd=st["rstd"], eps=EPS,
                     p=st["p"], seed=st["seed"], offset=st["offset"])
        return {"h": st["h"], "y": st["y"], "rstd": st["rstd"]}
    if op == "norm_bwd":
        moe.add_norm_bwd(st["dy"], st["h"], st["rstd"], st["weight"], dres=st["dres"], dh=st["dh"], dx=st["dx"],
                         dw=st["dw"], ws=st["ws"], p=st["p"], seed=st["seed"], offset=st["offset"])
        return {"dh": st["dh"], "dx": st["dx"], "dw": st["dw"]}
    if op == "matvec":
        moe.matvec_w4(st["x"], st["q"], st["scales"], st["y"])
        return {"y": st["y"]}
    moe.experts_w4(st["x"], st["topk_idx"], st["gates"], st["w"], st["out"], st["ws"])
    return {"out": st["out"]}


# ------------------------------------------------------------------ work
def work(case):
    op, s = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "norm_bwd", "dropout"):
        n, d, rows = case["rows"] * case["d"], case["d"], case["rows"]
        if op == "dropout":
            return {"bytes": 2 * n * s, "flops": 2 * n}
        r = SIZE[case["res"]]
        if op == "norm":   # x, residual in; h, y (or codes, scales and the dequantised copy), rstd out
            y = n * s + (n + n // 32 if case["out"] == "mx" else 0)
            return {"bytes": n * (s + 2 * r) + y + 4 * rows + d * s, "flops": 8 * n}
        return {"bytes": n * (2 * s + 3 * r) + 4 * rows + d * (s + 4), "flops": 14 * n}
    per = 0.5 + s / case["group"]
    if op == "matvec":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * per + s * m * (n + k), "flops": 2 * m * n * k}
    t, d, f, e, top = (case[n] for n in ("t", "d", "f", "e", "top"))
    active = e * (1 - (1 - top / e) ** t)   # experts that at least one token takes, on average
    return {"bytes": active * 3 * d * f * per + 2 * s * t * d + 8 * t * top, "flops": 6 * t * top * d * f}


# ------------------------------------------------------------------ 64 bits
def exact_mask(rows, cols, p, seed, offset):
    """The same generator on the host, in numpy's unsigned 64-bit integers."""
    import numpy as np
    lo = np.uint64(M32)
    sh = np.uint64(32)
    nb = (cols + 7) // 8
    x0 = np.broadcast_to(np.arange(nb, dtype=np.uint64), (rows, nb))
    x1 = np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, nb))
    x2, x3 = np.uint64(offset) & lo, np.uint64(offset) >> sh
    for i in range(10):
        ka = np.uint64(((seed & M32) + i * 0x9E3779B9) & M32)
        kb = np.uint64(((seed >> 32) + i * 0xBB67AE85) & M32)
        pa, pb = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (pb >> sh) ^ x1 ^ ka, pb & lo, (pa >> sh) ^ x3 ^ kb, pa & lo
    words = np.stack([x0, x1, x2, x3], -1).astype("<u4").view("<u2").reshape(rows, nb * 8)[:, :cols]
    return torch.from_numpy(np.ascontiguousarray(words >= int(p * 65536 + 0.5))).cuda()


def exact_drop(v, case, seed, offset):
    if case["p"] == 0:
        return v
    mask = exact_mask(case["rows"], case["d"], case["p"], seed, offset)
    return torch.where(mask, v / (1 - int(case["p"] * 65536 + 0.5) / 65536), torch.zeros_like(v))


def exact_mx(v):
    """Round each 32 columns to E4M3 steps of a common power of two, by the step sizes."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    s = torch.ceil(torch.log2(top / 448))   # smallest s with top <= 448 * 2^s, mended where log2 rounds
    s = torch.where(top > 448 * torch.exp2(s), s + 1, s)
    s = torch.where(top <= 448 * torch.exp2(s - 1), s - 1, s)
    s = torch.where(top > 0, s.clamp(-127, 127), torch.zeros_like(s))
    z = b / torch.exp2(s)
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(z / step) * step * torch.exp2(s)).reshape(v.shape)


def exact_w(q, s, group):
    """4-bit codes of one matrix to 64-bit weights."""
    out = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    out[:, 0::2] = (q % 16).double() - 8
    out[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double() - 8
    return out * s.double().repeat_interleave(group, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        return {"y": exact_drop(st["x"].double(), case, st["seed"], st["offset"])}
    if op == "norm":
        # the stream is stored in its own type, and the norm is that of what is stored
        h = st["residual"].double() + exact_drop(st["x"].double(), case, st["seed"], st["offset"])
        v = h.to(st["h"].dtype).double()
        rstd = 1 / torch.sqrt((v * v).sum(-1) / case["d"] + EPS)
        y = v * st["weight"].double() * rstd[:, None]
        return {"h": h, "y": exact_mx(y) if case["out"] == "mx" else y, "rstd": rstd}
    if op == "norm_bwd":
        h, dy, r = st["h"].double(), st["dy"].double(), st["rstd"].double()[:, None]
        g = dy * st["weight"].double()
        dh = st["dres"].double() + r * g - r ** 3 * h * ((g * h).sum(-1, keepdim=True) / case["d"])
        return {"dh": dh, "dx": exact_drop(dh, case, st["seed"], st["offset"]), "dw": torch.einsum("td,td,t->d", dy, h, r[:, 0])}
    if op == "matvec":
        return {"y": st["x"].double() @ exact_w(st["q"], st["scales"], case["group"]).T}
    out = torch.zeros(case["t"], case["d"], dtype=torch.float64, device="cuda")
    x, w, g = st["x"].double(), st["w"], case["group"]
    for e in range(case["e"]):
        t, j = (st["topk_idx"] == e).nonzero(as_tuple=True)
        if len(t):
            h, u = (x[t] @ exact_w(w[a + "_q"][e], w[a + "_s"][e], g).T for a in ("gate", "up"))
            a = h * torch.sigmoid(h) * u
            out.index_add_(0, t, (a @ exact_w(w["down_q"][e], w["down_s"][e], g).T) * st["gates"][t, j].double()[:, None])
    return {"out": out}
