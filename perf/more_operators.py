"""Cases of the operators with which a block that holds the MoE layer trains and is used
between two updates.

Residual addition with layer norm (forward and backward), an AdamW step over many
tensors with states in 32 or in 8 bits, and the whole MoE layer for a few tokens on
its bf16 weights.  Each case runs in a plain form (elementary torch operations in 32
bits, rounded once at the end) or, with `own` set, through the library's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
M32 = 0xFFFFFFFF
BLOCK = 128   # values that share a scale of the 8-bit states
LR, STEP, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 10, 0.9, 0.999, 1e-8, 0.01
WIDTHS = [128, 256, 384, 512, 640, 768, 896, 1024, 1408, 1536, 2048, 2816, 4096, 5632, 8192]   # whole 128-column blocks


def listed():
    return [
        # decode step of four sequences: the norm before the layer, latency counts
        dict(name="layer norm decode 4x4096", op="ln", rows=4, d=4096, dtype="bf16", res="bf16", p=0.0, out="y"),
        # training forward of the 8192-token layer: bf16 stream
        dict(name="layer norm 8192x2048", op="ln", rows=8192, d=2048, dtype="bf16", res="bf16", p=0.0, out="y"),
        # a width that no vector divides, fp16 activations on an fp32 stream
        dict(name="layer norm odd 777x1001", op="ln", rows=777, d=1001, dtype="f16", res="f32", p=0.1, out="y"),
        # training backward of the 8192-token layer
        dict(name="layer norm bwd 8192x2048", op="ln_bwd", rows=8192, d=2048, dtype="bf16", res="bf16", p=0.0),
        # training backward of the largest block: fp32 stream, residual dropout
        dict(name="layer norm bwd 32768x4096", op="ln_bwd", rows=32768, d=4096, dtype="bf16", res="f32", p=0.1),
        # weights and biases of two norms and the router of the 8192-token layer: fp32
        # parameters and states, latency counts
        dict(name="adamw norms and router", op="adamw", kind="block", e=32, d=2048, f=0, param="f32", grad="f32",
             master=False, bits=32),
        # router and experts of the 8192-token layer: bf16 weights with an fp32 copy, the
        # fp32 gradients of the layer's backward, states in 32 bits
        dict(name="adamw layer 32 bits", op="adamw", kind="layer", e=32, d=2048, f=1024, param="bf16", grad="f32",
             master=True, bits=32),
        # the same weights without the copy (stochastic rounding), states in 8 bits
        dict(name="adamw layer 8 bits", op="adamw", kind="layer", e=32, d=2048, f=1024, param="bf16", grad="f32",
             master=False, bits=8),
        # many tensors of odd sizes, one element among them, bf16 gradients
        dict(name="adamw ragged 8 bits", op="adamw", kind="ragged", tensors=131, most=100003, param="bf16", grad="bf16",
             master=False, bits=8),
        # one token through the largest layer
        dict(name="few 1 of 64x8", op="few", t=1, d=4096, f=2048, e=64, top=8),
        # sixteen sequences through the 8192-token layer
        dict(name="few 16 of 32x4", op="few", t=16, d=2048, f=1024, e=32, top=4),
        # 64 sequences through the layer with d_ff 1408: every expert is read
        dict(name="few 64 of 64x4", op="few", t=64, d=2048, f=1408, e=64, top=4),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln_bwd", "adamw", "adamw", "few", "few"])
    if op in ("ln", "ln_bwd"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        p = rng.choice([0.0, rng.randint(1, 50) / 100])
        rows, d, out = log_int(rng, 1, 32768), log_int(rng, 64, 8192), "y"
        if rng.random() < 0.6:
            d = rng.choice(WIDTHS)
            if dtype == "bf16" and rng.random() < 0.3:
                out = "mx"
        while rows * d > 16384 * 4096:   # wide types stay below the largest listed case
            rows = max(1, rows // 2)
        case = dict(op=op, rows=rows, d=d, dtype=dtype, res=rng.choice([dtype, "f32"]), p=p)
        return dict(case, out=out) if op == "ln" else case
    if op == "adamw":
        param, master = rng.choice([("bf16", True), ("bf16", False), ("f32", False), ("f16", True)])
        case = dict(op=op, param=param, grad=rng.choice(["f32", param]), master=master, bits=rng.choice([8, 32]))
        if rng.random() < 0.5:
            return dict(case, kind="ragged", tensors=log_int(rng, 1, 300), most=log_int(rng, 10, 300000))
        return dict(case, kind="layer", e=rng.choice([4, 8, 16, 32]), d=128 * rng.randint(1, 16), f=128 * rng.randint(1, 8))
    e = rng.choice([8, 32, 64, 128])
    return dict(op=op, t=log_int(rng, 1, 64), d=128 * rng.randint(4, 20), f=128 * rng.randint(1, 11), e=e,
                top=rng.choice([1, 2, 4, 8]))


# ------------------------------------------------------------------ inputs
def sizes_of(case):
    """Elements of each tensor of an AdamW case."""
    if case["kind"] == "ragged":
        rng = random.Random(case["tensors"] * 7919 + case["most"])
        return [1] + [log_int(rng, 1, case["most"]) for _ in range(case["tensors"] - 1)]
    e, d, f = case["e"], case["d"], case["f"]
    if case["kind"] == "block":
        return [d, d, d, d, e * d]
    return [e * d, e * f * d, e * f * d, e * d * f]


def states_8(v):
    """Codes and scales of 128 values each (rounded to nearest): a state some steps in."""
    b = v.unflatten(0, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, b * (448 / top), torch.zeros_like(b)).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).flatten(), (top / 448).flatten()


def prepare_adamw(case, seed, gen):
    """All tensors of a kind lie in one buffer, each from a 128-element boundary, with
    zeros between them; what the optimiser keeps is a list of the tensors."""
    sizes = sizes_of(case)
    starts, n = [], 0
    for s in sizes:
        starts.append(n)
        n += (s + BLOCK - 1) // BLOCK * BLOCK
    inside = torch.ones(n, dtype=torch.bool, device="cuda")
    for at, s in zip(starts, sizes):
        inside[at + s:(at + s + BLOCK - 1) // BLOCK * BLOCK] = False
    pt, gt = DT[case["param"]], DT[case["grad"]]

    def normal(scale):
        return (torch.randn(n, generator=gen, device="cuda") * scale).mul_(inside)

    st = dict(op="adamw", case=case, sizes=sizes, starts=starts, n=n,
              seed=(int(seed) * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF, offset=int(seed) % 1000)
    master = normal(0.02)
    st["param"] = master.to(pt)
    if case["master"]:
        st["master"] = master
    # gradients and states of places whose gradients differ in size by a factor of ten
    size = 1e-3 * torch.exp(1.2 * normal(1.0)).mul_(inside)
    st["grad"] = normal(1.0).mul_(size).to(gt)
    m, root = normal(0.3).mul_(size), size * 0.7
    if case["bits"] == 8:
        st["m"], st["m_scale"] = states_8(m)
        st["v"], st["v_scale"] = states_8(root)
        # a second moment is only zero where every gradient has been zero
        st["v"].clamp_(min=1).mul_(inside)
    else:
        st["m"], st["v"] = m, root.square()
    if own:
        import moe_expert_layer_softmax_gb300 as moe

        def cut(name, per=1):
            return [st[name][at // per:at // per + (s + per - 1) // per] for at, s in zip(starts, sizes)]
        states = [cut(k) if case["bits"] == 32 else list(zip(cut(k), cut(k + "_scale", BLOCK))) for k in ("m", "v")]
        st["list"] = moe.adamw_list(cut("param"), cut("grad"), *states, master=cut("master") if case["master"] else None)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "adamw":
        return prepare_adamw(case, seed, gen)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    st = dict(op=op, case=case, seed=(int(seed) * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF, offset=int(seed) % 1000)
    if op == "few":
        t, d, f, e, top = (case[n] for n in ("t", "d", "f", "e", "top"))
        st["x"] = normal(t, d)
        st["w_router"] = normal(e, d, scale=0.02)
        st["w_gate"], st["w_up"], st["w_down"] = (normal(*s, scale=0.02) for s in ((e, f, d), (e, f, d), (e, d, f)))
        st["out"] = torch.empty_like(st["x"])
        st["gates"] = torch.empty(t, top, device="cuda")
        st["topk_idx"] = torch.empty(t, top, dtype=torch.int32, device="cuda")
        if own:
            import moe_expert_layer_softmax_gb300 as moe
            st["shape"] = moe.shape(t, d, e, top, f)
            st["ws"] = torch.zeros(moe.few_workspace(st["shape"]), dtype=torch.uint8, device="cuda")
        return st
    dt, rt = DT[case["dtype"]], DT[case["res"]]
    rows, d = case["rows"], case["d"]
    st["p"] = case["p"]
    st["weight"] = normal(d, scale=0.1).add_(1).to(dt)
    if op == "ln":
        st["bias"] = normal(d, scale=0.1, dtype=dt)
        st["x"] = normal(rows, d, dtype=dt)
        # the stream of a row has a mean of its own
        st["residual"] = (normal(rows, d, scale=2.0, dtype=torch.float32) + normal(rows, 1, dtype=torch.float32)).to(rt)
        st["h"] = torch.empty_like(st["residual"])
        st["mean"], st["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if case["out"] == "mx":   # buffers of whole 128-row tiles, as the MXFP8 GEMMs read them
            pad = (rows + 127) // 128 * 128
            st["y_q"] = torch.empty(pad, d, dtype=torch.uint8, device="cuda")
            st["y_scales"] = torch.empty(pad * d // 32, dtype=torch.uint8, device="cuda")
            st["y_dq"] = torch.empty(pad, d, dtype=dt, device="cuda")
        else:
            st["y"] = torch.empty_like(st["x"])
        return st
    st["dy"] = normal(rows, d, dtype=dt)
    st["h"] = (normal(rows, d, scale=2.0, dtype=torch.float32) + normal(rows, 1, dtype=torch.float32)).to(rt)
    st["dres"] = normal(rows, d, dtype=rt)
    v = st["h"].double()
    st["mean"] = v.mean(-1).float()
    st["rstd"] = (v.var(-1, correction=0) + EPS).rsqrt().float()
    st["dh"] = torch.empty_like(st["h"])
    st["dx"] = torch.empty_like(st["dy"])
    st["dw"], st["db"] = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    if own:
        import moe_expert_layer_softmax_gb300 as moe
        st["ws"] = torch.empty(moe.add_layer_norm_bwd_workspace(rows, d), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def philox(c0, c1, offset, seed):
    """Philox4x32-10 of the counters (c0, c1, offset): eight 16-bit numbers each, in the last axis."""
    c = [c0, c1, torch.tensor(offset & M32, device="cuda"), torch.tensor(offset >> 32, device="cuda")]
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & M32) ^ c[1] ^ k0, b & M32, (a >> 32 & M32) ^ c[3] ^ k1, a & M32]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([h.to(torch.int32) for w in c for h in (w & 0xFFFF, w >> 16)], -1)


def drop(v, p, seed, offset):
    """v (32 bits) with dropped places at zero and the others scaled up; the keep
    probability is a multiple of 2^-16."""
    thr = int(math.floor(p * 65536 + 0.5))
    if thr == 0:
        return v
    rows, cols = v.shape
    r = philox(torch.arange((cols + 7) // 8, device="cuda")[None, :], torch.arange(rows, device="cuda")[:, None], offset, seed)
    return torch.where(r.flatten(1)[:, :cols] >= thr, v * (65536 / (65536 - thr)), 0.0)


def mx_values(v):
    """The values that E4M3 codes with one power-of-two scale a 32 columns stand for."""
    b = v.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    s = (e - torch.where(m <= 0.875, 9, 8)).clamp(-127, 127) * (m > 0)
    q = torch.ldexp(b, -s).clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.ldexp(q.float(), s).flatten(-2)


def numbers(st, what):
    """16-bit numbers of every place: the counter is (index / 8, 4 tensor + what)."""
    counts = torch.tensor([(s + BLOCK - 1) // BLOCK * (BLOCK // 8) for s in st["sizes"]], device="cuda")
    tensor = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), counts, output_size=st["n"] // 8)
    index = torch.arange(st["n"] // 8, device="cuda") - (counts.cumsum(0) - counts)[tensor]
    return philox(index, 4 * tensor + what, st["offset"], st["seed"]).flatten()


def to_e4m3(v, r, least):
    """E4M3 codes and scales of 128 values each, the magnitude rounded up where its
    remainder is at least 1 - r / 2^16; with `least` no value above zero becomes zero."""
    b = v.unflatten(0, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    some = top >= 2.0 ** -100   # smaller ones have no inverse in 32 bits
    z = torch.where(some, (b.abs() * (448 * torch.reciprocal(top))).clamp(max=448), torch.zeros_like(b))
    step = (torch.frexp(z)[1].clamp(min=-5) + 123 << 23).view(torch.float32)   # a power of two
    q = z / step
    low = q.floor()
    q = (low + ((q - low) * 65536 >= 65536 - r.view_as(b))) * step
    q = torch.where((z > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q) if least else q
    return torch.copysign(q, b).to(torch.float8_e4m3fn).view(torch.uint8).flatten(), torch.where(some, top * (1 / 448), torch.zeros_like(top)).flatten()


def from_e4m3(q, scale):
    return (q.view(torch.float8_e4m3fn).float().unflatten(0, (-1, BLOCK)) * scale[:, None]).flatten()


def plain_adamw(st):
    """Every operation rounded to 32 bits."""
    case, small = st["case"], st["case"]["bits"] == 8
    g = st["grad"].float()
    m = from_e4m3(st["m"], st["m_scale"]) if small else st["m"]
    v = from_e4m3(st["v"], st["v_scale"]).square() if small else st["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    p = st["master"] if case["master"] else st["param"].float()
    p = p * (1 - LR * DECAY) - m / (root * (1 - BETA2 ** STEP) ** -0.5 + ADAM_EPS) * (LR / (1 - BETA1 ** STEP))
    if small:
        for name, x, what in (("m", m, 0), ("v", root, 1)):
            q, s = to_e4m3(x, numbers(st, what), what == 1)
            st[name].copy_(q)
            st[name + "_scale"].copy_(s)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    if case["master"]:
        st["master"].copy_(p)
    if case["param"] == "bf16" and not case["master"]:   # stochastic rounding: 16 bits are cut off
        st["param"].copy_((p.view(torch.int32) + numbers(st, 2) & -65536).view(torch.float32))
    else:
        st["param"].copy_(p)
    return adamw_outputs(st)


def adamw_outputs(st):
    out = {k: st[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if k in st}
    if st["case"]["bits"] == 8:   # as the values that they stand for, in units of their scales
        out.update(m=st["m"].view(torch.float8_e4m3fn), v=st["v"].view(torch.float8_e4m3fn))
    return out


def plain_few(st):
    x, top = st["x"].float(), st["case"]["top"]
    logits, idx = torch.sort(x @ st["w_router"].float().T, stable=True, dim=-1, descending=True)
    gates, idx = torch.softmax(logits[:, :top], -1), idx[:, :top]
    t, e = x.shape[0], st["case"]["e"]
    w = [st["w_" + n] for n in ("gate", "up", "down")]
    if t * top < e:   # fewer routes than experts: only the routed experts' weights
        w_gate, w_up, w_down = (v[idx.flatten()].float() for v in w)
        x = x.repeat_interleave(top, 0)[:, :, None]
        h = w_gate @ x
        y = (w_down @ (h / (1 + torch.exp(-h)) * (w_up @ x)))[..., 0]
        out = (y.unflatten(0, (t, top)) * gates[..., None]).sum(1)
    else:
        gate = torch.zeros(t, e, device="cuda").scatter_(1, idx, gates)
        h = x @ w[0].float().transpose(1, 2)
        a = h / (1 + torch.exp(-h)) * (x @ w[1].float().transpose(1, 2)) * gate.T[:, :, None]
        out = (a @ w[2].float().transpose(1, 2)).sum(0)
    return {"out": out.to(st["x"].dtype), "gates": gates}


def plain(st):
    op, case = st["op"], st["case"]
    if op == "adamw":
        return plain_adamw(st)
    if op == "few":
        return plain_few(st)
    if op == "ln":
        h = (st["residual"].float() + drop(st["x"].float(), st["p"], st["seed"], st["offset"])).to(st["residual"].dtype)
        v = h.float()
        mean = v.mean(-1)
        c = v - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(-1) + EPS)
        y = c * rstd[:, None] * st["weight"].float() + st["bias"].float()
        y = mx_values(y) if case["out"] == "mx" else y
        return {"h": h, "y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}
    dy, r = st["dy"].float(), st["rstd"][:, None]
    xh = (st["h"].float() - st["mean"][:, None]) * r
    g = dy * st["weight"].float()
    dh = st["dres"].float() + r * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    dx = drop(dh, st["p"], st["seed"], st["offset"])
    return {"dh": dh.to(st["dh"].dtype), "dx": dx.to(st["dx"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def run(st):
    if not own:
        return plain(st)
    import moe_expert_layer_softmax_gb300 as moe
    op = st["op"]
    if op == "adamw":
        moe.adamw(st["list"], lr=LR, step=STEP, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY,
                  seed=st["seed"], offset=st["offset"])
        return adamw_outputs(st)
    if op == "few":
        moe.forward_few(st["shape"], st["x"], st["w_router"], None, st["w_gate"], st["w_up"], st["w_down"], st["out"],
                        st["ws"], topk_idx=st["topk_idx"], gates=st["gates"])
        return {"out": st["out"], "gates": st["gates"]}
    if op == "ln":
        kw = dict(residual=st["residual"], h=st["h"], mean=st["mean"], rstd=st["rstd"], eps=EPS, p=st["p"],
                  seed=st["seed"], offset=st["offset"])
        if "y_q" in st:
            moe.add_layer_norm(st["x"], st["weight"], st["bias"], None, y_q=st["y_q"], y_scales=st["y_scales"],
                               y_dq=st["y_dq"], **kw)
            y = st["y_dq"][:st["x"].shape[0]]
        else:
            moe.add_layer_norm(st["x"], st["weight"], st["bias"], st["y"], **kw)
            y = st["y"]
        return {"h": st["h"], "y": y, "mean": st["mean"], "rstd": st["rstd"]}
    moe.add_layer_norm_bwd(st["dy"], st["h"], st["mean"], st["rstd"], st["weight"], dres=st["dres"], dh=st["dh"],
                           dx=st["dx"], dw=st["dw"], db=st["db"], ws=st["ws"], p=st["p"], seed=st["seed"],
                           offset=st["offset"])
    return {"dh": st["dh"], "dx": st["dx"], "dw": st["dw"], "db": st["db"]}


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(sizes_of(case))
        param = SIZE[case["param"]] * (1 if case["master"] else 2) + (8 if case["master"] else 0)
        states = 4 * (1 + 4 / BLOCK) if case["bits"] == 8 else 16
        return {"bytes": n * (SIZE[case["grad"]] + param + states), "flops": 16 * n}
    if op == "few":
        t, d, f, e, top = (case[n] for n in ("t", "d", "f", "e", "top"))
        active = e * (1 - (1 - top / e) ** t)   # experts that at least one token takes, on average
        return {"bytes": active * 3 * d * f * 2 + 2 * e * d + 4 * t * d + 4 * t * top, "flops": 6 * t * top * d * f + 2 * t * d * e}
    s, r = SIZE[case["dtype"]], SIZE[case["res"]]
    n, d, rows = case["rows"] * case["d"], case["d"], case["rows"]
    if op == "ln":   # x, residual in; h, y (or codes, scales and the dequantised copy), mean, rstd out
        y = n * s + (n + n // 32 if case["out"] == "mx" else 0)
        return {"bytes": n * (s + 2 * r) + y + 8 * rows + 2 * d * s, "flops": 10 * n}
    return {"bytes": n * (2 * s + 3 * r) + 8 * rows + d * (s + 8), "flops": 18 * n}


# ------------------------------------------------------------------ 64 bits
def exact_words(low, high, offset, seed):
    """The generator from its definition, products in two halves: four 32-bit words a counter."""
    def mulhilo(a, b):
        p0, p1 = (a & 0xFFFF) * b, (a >> 16) * b
        low = p0 + ((p1 & 0xFFFF) << 16)
        return (p1 >> 16) + (low >> 32), low & M32
    x0, x1 = torch.broadcast_tensors(low, high)
    x2, x3 = torch.full_like(x0, offset % (1 << 32)), torch.full_like(x0, offset // (1 << 32))
    for i in range(10):
        ka, kb = ((seed & M32) + i * 0x9E3779B9) & M32, ((seed >> 32) + i * 0xBB67AE85) & M32
        (ha, la), (hb, lb) = mulhilo(x0, 0xD2511F53), mulhilo(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = hb ^ x1 ^ ka, lb, ha ^ x3 ^ kb, la
    return x0, x1, x2, x3


def exact_drop(v, case, st):
    thr = int(case["p"] * 65536 + 0.5)
    if thr == 0:
        return v
    rows, cols = v.shape
    w = exact_words(torch.arange((cols + 7) // 8, device="cuda")[None, :], torch.arange(rows, device="cuda")[:, None],
                    st["offset"], st["seed"])
    keep = torch.empty(rows, (cols + 7) // 8, 8, dtype=torch.bool, device="cuda")
    for i in range(4):
        keep[:, :, 2 * i] = w[i] % 65536 >= thr
        keep[:, :, 2 * i + 1] = w[i] // 65536 >= thr
    return torch.where(keep.reshape(rows, -1)[:, :cols], v / (1 - thr / 65536), torch.zeros_like(v))


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


def exact_numbers(st, tensor, what, size):
    """16-bit numbers of one tensor's places."""
    w = exact_words(torch.arange((size + 7) // 8, device="cuda"), torch.tensor(4 * tensor + what, device="cuda"),
                    st["offset"], st["seed"])
    r = torch.empty((size + 7) // 8, 8, dtype=torch.float64, device="cuda")
    for i in range(4):
        r[:, 2 * i] = w[i] % 65536
        r[:, 2 * i + 1] = w[i] // 65536
    return r.reshape(-1)[:size]


def exact_state(x, r, least):
    """(values in units of their scale, scales) of one tensor's 8-bit state."""
    n = x.numel()
    blocks = (n + BLOCK - 1) // BLOCK
    pad = torch.zeros(blocks * BLOCK, dtype=torch.float64, device="cuda")
    pad[:n] = x
    scale = pad.reshape(blocks, BLOCK).abs().amax(1) / 448
    z = (x / scale.clamp_min(1e-300).repeat_interleave(BLOCK)[:n]).abs()
    step = torch.exp2(torch.floor(torch.log2(z.clamp_min(2.0 ** -6))) - 3)
    down = torch.floor(z / step)
    q = (down + (z / step - down >= 1 - r / 65536).double()) * step
    if least:
        q = torch.where(z > 0, q.clamp_min(2.0 ** -9), q)
    return q * torch.sign(x), scale


def exact_adamw(st):
    case = st["case"]
    out = {k: torch.zeros(v.numel(), dtype=torch.float64, device="cuda") for k, v in adamw_outputs(st).items()}
    for i, (at, n) in enumerate(zip(st["starts"], st["sizes"])):
        def part(name):
            v = st[name][at:at + n]
            if case["bits"] == 32:
                return v.double()
            scales = st[name + "_scale"].double()[at // BLOCK:(at + n + BLOCK - 1) // BLOCK]
            return v.view(torch.float8_e4m3fn).double() * scales.repeat_interleave(BLOCK)[:n]
        g = st["grad"][at:at + n].double()
        m = BETA1 * part("m") + (1 - BETA1) * g
        v = part("v")
        v = BETA2 * (v * v if case["bits"] == 8 else v) + (1 - BETA2) * g * g
        p = (st["master"] if case["master"] else st["param"])[at:at + n].double()
        p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + ADAM_EPS)
        if case["bits"] == 32:
            out["m"][at:at + n], out["v"][at:at + n] = m, v
        else:
            for name, x, what in (("m", m, 0), ("v", torch.sqrt(v), 1)):
                q, s = exact_state(x, exact_numbers(st, i, what, n), what == 1)
                out[name][at:at + n], out[name + "_scale"][at // BLOCK:at // BLOCK + len(s)] = q, s
        if case["master"]:
            out["master"][at:at + n] = p
        elif case["param"] == "bf16":   # to a neighbour, by the number of the place
            a = p.abs()
            step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -126))) - 7)
            down = torch.floor(a / step)
            up = a / step - down >= 1 - exact_numbers(st, i, 2, n) / 65536
            p = torch.sign(p) * (down + up.double()) * step
        out["param"][at:at + n] = p
    return out


def exact_few(st):
    case = st["case"]
    logits = st["x"].double() @ st["w_router"].double().T
    order = torch.sort(-logits, stable=True, dim=-1).indices[:, :case["top"]]
    z = logits.gather(1, order)
    z = torch.exp(z - z.amax(-1, keepdim=True))
    gates = z / z.sum(-1, keepdim=True)
    out = torch.zeros(case["t"], case["d"], dtype=torch.float64, device="cuda")
    x = st["x"].double()
    for e in range(case["e"]):
        t, j = (order == e).nonzero(as_tuple=True)
        if len(t):
            h, u = x[t] @ st["w_gate"][e].double().T, x[t] @ st["w_up"][e].double().T
            out.index_add_(0, t, ((h * torch.sigmoid(h) * u) @ st["w_down"][e].double().T) * gates[t, j][:, None])
    return {"out": out, "gates": gates}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return exact_adamw(st)
    if op == "few":
        return exact_few(st)
    if op == "ln":
        # the stream is stored in its own type, and the norm is that of what is stored
        h = st["residual"].double() + exact_drop(st["x"].double(), case, st)
        v = h.to(st["h"].dtype).double()
        mean = v.sum(-1) / case["d"]
        rstd = 1 / torch.sqrt(((v - mean[:, None]) ** 2).sum(-1) / case["d"] + EPS)
        y = (v - mean[:, None]) * (st["weight"].double() * rstd[:, None]) + st["bias"].double()
        return {"h": h, "y": exact_mx(y) if case["out"] == "mx" else y, "mean": mean, "rstd": rstd}
    h, dy, r, mu = st["h"].double(), st["dy"].double(), st["rstd"].double()[:, None], st["mean"].double()[:, None]
    g = dy * st["weight"].double()
    d = case["d"]
    dh = st["dres"].double() + r * g - r * g.sum(-1, keepdim=True) / d - r ** 3 * (h - mu) * ((g * (h - mu)).sum(-1, keepdim=True) / d)
    return {"dh": dh, "dx": exact_drop(dh, case, st), "dw": torch.einsum("td,td,t->d", dy, h - mu, r[:, 0]), "db": dy.sum(0)}
