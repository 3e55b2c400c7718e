"""Cases of the operators of a memory-lean MLP block: the root-mean-square norm
with its residual, products with bias, activation and residual, activation
checkpoints in 8 bits, and the gradients that read those checkpoints.

A checkpoint of t [rows, C] holds groups of 128 channels of one row: a power of
two 2^k, the smallest with max|t| / 2^k <= 127 (k in -120..121), and the codes
q = round(t / 2^k), ties to even.  Codes are int8 [rows, C rounded up to 16],
exponents uint8 k + 127 [groups, rows].

Each case names its operator in "op":
  norm       h = x + res, y = rms_norm(h) * gamma, checkpoint of the normalised h
  norm_back  gradients of x (with the residual's added) and gamma, from the checkpoint
  linear     y = act(x w^T + bias) + res, with or without checkpoints of the
             pre-activation and of y
  back       gradient through a product and the activation before it,
             (gy w) * act'(z) + res, z from its checkpoint
  pack       the checkpoint of a tensor that comes from elsewhere
  grad_w     weight and bias gradient of a product, its input from a checkpoint
"""

import math

import torch

own = False

GROUP = 128
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token of generation through the norm of a 4096-wide block: latency
        dict(name="norm_token", op="norm", dtype="bf16", rows=1, C=4096, res=True),
        # a training batch of 4 x 2048 tokens through the same norm
        dict(name="norm_long", op="norm", dtype="bf16", rows=8192, C=4096, res=True),
        # gradient of a 448-wide norm in fp32: 256 images of 49 tokens
        dict(name="norm_back_vit_f32", op="norm_back", dtype="f32", rows=12544, C=448, res=True),
        # gradient of the long batch's norm
        dict(name="norm_back_long", op="norm_back", dtype="bf16", rows=8192, C=4096, res=True),
        # one token of generation through the widening product: reads the weights once
        dict(name="linear_token", op="linear", dtype="bf16", rows=1, Cx=4096, Cy=11008, act="gelu",
             res=False, ckpt=False),
        # the vision block's widening product in training, both checkpoints kept
        dict(name="linear_vit", op="linear", dtype="bf16", rows=12544, Cx=448, Cy=1792, act="gelu",
             res=False, ckpt=True),
        # the long batch's narrowing product with the block's residual
        dict(name="linear_long", op="linear", dtype="bf16", rows=8192, Cx=11008, Cy=4096, act="none",
             res=True, ckpt=False),
        # a small fp32 layer's gradient through its activation, odd token count
        dict(name="back_f32", op="back", dtype="f32", rows=333, Cx=1792, Cy=448, act="silu", res=False),
        # the long batch's gradient through the narrowing product and the activation
        dict(name="back_long", op="back", dtype="bf16", rows=8192, Cx=11008, Cy=4096, act="gelu",
             res=False),
        # an activation that no operator here made: packed by itself, odd token count
        dict(name="pack_wide", op="pack", dtype="bf16", rows=8191, C=11008),
        # weight gradient of a BERT-width layer over a ragged batch, last group short
        dict(name="grad_w_ragged", op="grad_w", dtype="bf16", rows=1571, Cx=776, Cy=768, scale=False),
        # the long batch's weight gradient of the widening product, input kept by the norm
        dict(name="grad_w_long", op="grad_w", dtype="bf16", rows=8192, Cx=4096, Cy=11008, scale=True),
    ]


def draw(rng):
    """One more case: tokens from one to 8192, widths of 64 to 11008 in steps of
    8, small sizes in fp32, every activation, with and without residual."""
    op = rng.choice(["norm", "norm_back", "linear", "linear", "back", "pack", "grad_w"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(hi):
        while True:
            c = 8 * log(8, hi // 8)
            if c != 3072:
                return c

    rows = log(1, 8192)
    if op in ("norm", "norm_back", "pack"):
        c = dict(op=op, dtype=dtype, rows=rows, C=width(11008))
        if op != "pack":
            c["res"] = rng.random() < 0.5
        return c
    small = dtype == "f32"
    if small:
        rows = log(1, 1024)
    c = dict(op=op, dtype=dtype, rows=rows, Cx=width(2048 if small else 11008),
             Cy=width(2048 if small else 11008))
    most = 8192 * 4096 * 11008
    if rows * c["Cx"] * c["Cy"] > most:
        c["rows"] = most // (c["Cx"] * c["Cy"])
    if op == "grad_w":
        c["scale"] = rng.random() < 0.5
    else:
        c["act"] = rng.choice(["none", "relu", "gelu", "silu"])
        c["res"] = rng.random() < 0.5
    if op == "linear":
        c["ckpt"] = rng.random() < 0.5
    return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["rows"]
    op = case["op"]
    if op in ("norm", "norm_back", "pack"):
        C = case["C"]
        code = n * C + n * -(-C // GROUP)
        if op == "pack":  # reads t, writes the codes, and the values they stand for (2 bytes each)
            return {"bytes": n * C * e + code + 2 * n * C, "flops": 3 * n * C}
        res = n * C * e if case["res"] else 0
        if op == "norm":
            # x, res -> h, y, codes, r and the codes' values
            return {"bytes": n * C * e + res + (n * C * e if case["res"] else 0) + n * C * e + code
                    + 2 * n * C + 4 * n + C * e, "flops": 8 * n * C}
        return {"bytes": 2 * n * C * e + res + code + 4 * n + C * e + 4 * C, "flops": 10 * n * C}
    Cx, Cy = case["Cx"], case["Cy"]
    flops = 2 * n * Cx * Cy
    if op == "linear":
        b = (n * Cx + Cx * Cy + Cy + n * Cy) * e
        if case["res"]:
            b += n * Cy * e
        if case["ckpt"]:
            b += 2 * (n * Cy + n * -(-Cy // GROUP) + 2 * n * Cy)
        return {"bytes": b, "flops": flops}
    if op == "back":
        b = (n * Cy + Cx * Cy + n * Cx) * e
        if case["res"]:
            b += n * Cx * e
        if case["act"] != "none":
            b += n * Cx + n * -(-Cx // GROUP)
        return {"bytes": b, "flops": flops}
    b = n * Cy * e + n * Cx + n * -(-Cx // GROUP) + 4 * Cx * Cy + 4 * Cy + (Cx * e if case["scale"] else 0)
    return {"bytes": b, "flops": flops + n * Cy}


# --------------------------------------------------------------------------
# the checkpoint in elementary operations
# --------------------------------------------------------------------------
def grouped(t):
    """t [rows, C] padded with zeros to whole groups: [rows, groups, 128]."""
    rows, C = t.shape
    return torch.nn.functional.pad(t, (0, -C % GROUP)).view(rows, -1, GROUP)


def pack(t):
    """(codes int8 [rows, C to 16], exponents uint8 [groups, rows]) of an fp32 t."""
    rows, C = t.shape
    g = grouped(t)
    m, e = torch.frexp(g.abs().amax(-1))
    k = (e - 7 + (m > 127 / 128)).clamp(-120, 121)
    q = torch.ldexp(g, -k.unsqueeze(-1)).round().clamp(-127, 127)
    q = q.view(rows, -1)[:, :C].to(torch.int8)
    q = torch.nn.functional.pad(q, (0, -C % 16)).contiguous()
    return q, (k + 127).to(torch.uint8).t().contiguous()


def values(q, s, C):
    """What the codes stand for, fp32 [rows, C]."""
    rows = q.shape[0]
    k = (s.t().to(torch.int32) - 127).unsqueeze(-1)
    return torch.ldexp(grouped(q[:, :C].float()), k).reshape(rows, -1)[:, :C]


def activated(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def inputs(case, seed):
    """The tensors of a case, from the seed alone.  Activations are normal with a
    few channels twenty times larger, as in trained transformers; gradients are
    small; weights have variance 1 / width."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed * 1_000_003 + 17)
    dt = TYPES[case["dtype"]]
    n, op = case["rows"], case["op"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std)

    def activation(rows, C):
        big = torch.ones(C, device=dev)
        big[torch.randint(0, C, (max(1, C // 256),), generator=gen, device=dev)] = 20.0
        return normal(rows, C) * big

    d = {}
    if op in ("norm", "norm_back", "pack"):
        C = case["C"]
        if op == "pack":
            return {"x": activation(n, C).to(dt)}
        d["gamma"] = (1 + normal(C, std=0.1)).to(dt)
        if op == "norm":
            d["x"] = activation(n, C).to(dt)
            if case["res"]:
                d["res"] = activation(n, C).to(dt)
            return d
        h = activation(n, C)
        r = torch.rsqrt(h.square().mean(-1) + EPS)
        d["q"], d["s"] = pack(h * r[:, None])
        d["r"] = r
        d["gy"] = normal(n, C, std=1e-2).to(dt)
        if case["res"]:
            d["res"] = normal(n, C, std=1e-2).to(dt)
        return d
    Cx, Cy = case["Cx"], case["Cy"]
    if op == "linear":
        d["x"] = activation(n, Cx).to(dt)
        d["w"] = normal(Cy, Cx, std=Cx ** -0.5).to(dt)
        d["bias"] = normal(Cy, std=0.1).to(dt)
        if case["res"]:
            d["res"] = activation(n, Cy).to(dt)
        return d
    if op == "back":
        d["gy"] = normal(n, Cy, std=1e-2).to(dt)
        d["w"] = normal(Cy, Cx, std=Cx ** -0.5).to(dt)
        if case["act"] != "none":
            d["q"], d["s"] = pack(normal(n, Cx, std=1.5))
        if case["res"]:
            d["res"] = normal(n, Cx, std=1e-2).to(dt)
        return d
    d["gy"] = normal(n, Cy, std=1e-2).to(dt)
    d["q"], d["s"] = pack(activation(n, Cx))
    if case["scale"]:
        d["scale"] = (1 + normal(Cx, std=0.1)).to(dt)
    return d


def prepare(case, seed):
    """The inputs, and the output buffers that a training program keeps."""
    d = inputs(case, seed)
    n, op, dt = case["rows"], case["op"], TYPES[case["dtype"]]
    dev = next(iter(d.values())).device

    def buf(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev)

    def ckpt(name, C):
        d[name + "q"] = buf(n, C + -C % 16, dtype=torch.int8)
        d[name + "s"] = buf(-(-C // GROUP), n, dtype=torch.uint8)
        d[name + "v"] = buf(n, C, dtype=torch.bfloat16)

    if op == "norm":
        C = case["C"]
        d["y"], d["r"] = buf(n, C), buf(n, dtype=torch.float32)
        if case["res"]:
            d["h"] = buf(n, C)
        ckpt("u", C)
    elif op == "norm_back":
        d["gx"], d["ggamma"] = buf(n, case["C"]), buf(case["C"], dtype=torch.float32)
    elif op == "pack":
        ckpt("x", case["C"])
    elif op == "linear":
        d["y"] = buf(n, case["Cy"])
        if case["ckpt"]:
            ckpt("z", case["Cy"])
            ckpt("y", case["Cy"])
    elif op == "back":
        d["gx"] = buf(n, case["Cx"])
    else:
        d["gw"] = buf(case["Cy"], case["Cx"], dtype=torch.float32)
        d["gb"] = buf(case["Cy"], dtype=torch.float32)
    return case, d


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    case, d = state
    return (run_own if own else run_plain)(case, d)


def run_plain(case, d):
    op, dt = case["op"], TYPES[case["dtype"]]

    def held(t):  # a checkpoint's values
        return values(*pack(t), t.shape[1]).to(torch.bfloat16)

    if op == "pack":
        return {"values": held(d["x"].float())}
    if op == "norm":
        h = d["x"].float()
        if case["res"]:
            h = h + d["res"].float()
        r = torch.rsqrt(h.square().mean(-1) + EPS)
        u = h * r[:, None]
        out = {"y": (u * d["gamma"].float()).to(dt), "r": r, "values": held(u)}
        if case["res"]:
            out["h"] = h.to(dt)
        return out
    if op == "norm_back":
        u = values(d["q"], d["s"], case["C"])
        gy = d["gy"].float()
        dn = gy * d["gamma"].float()
        c = (dn * u).mean(-1, keepdim=True)
        gx = d["r"][:, None] * (dn - u * c)
        if case["res"]:
            gx = gx + d["res"].float()
        return {"gx": gx.to(dt), "ggamma": (gy * u).sum(0)}
    if op == "linear":
        z = d["x"].float() @ d["w"].float().t() + d["bias"].float()
        y = activated(z, case["act"])
        if case["res"]:
            y = y + d["res"].float()
        out = {"y": y.to(dt)}
        if case["ckpt"]:
            out["z_values"], out["y_values"] = held(z), held(y)
        return out
    if op == "back":
        g = d["gy"].float() @ d["w"].float()
        if case["act"] != "none":
            g = g * slope(values(d["q"], d["s"], case["Cx"]), case["act"])
        if case["res"]:
            g = g + d["res"].float()
        return {"gx": g.to(dt)}
    gy = d["gy"].float()
    gw = gy.t() @ values(d["q"], d["s"], case["Cx"])
    if case["scale"]:
        gw = gw * d["scale"].float()
    return {"gw": gw, "gb": gy.sum(0)}


def run_own(case, d):
    from rank_compressed_backprop_gb300 import api

    op = case["op"]
    if op == "pack":
        api.ckpt_pack(d["x"], d["xq"], d["xs"])
        return {"values": api.ckpt_unpack(d["xq"], d["xs"], d["xv"])}
    if op == "norm":
        api.rms_norm(d["x"], d["gamma"], d["y"], residual=d.get("res"), h=d.get("h"), q=d["uq"], s=d["us"],
                     r=d["r"], eps=EPS)
        out = {"y": d["y"], "r": d["r"], "values": api.ckpt_unpack(d["uq"], d["us"], d["uv"])}
        if case["res"]:
            out["h"] = d["h"]
        return out
    if op == "norm_back":
        ws = api.rms_norm_backward_workspace(case["rows"], case["C"], d["gy"].device)
        api.rms_norm_backward(d["gy"], d["q"], d["s"], d["r"], d["gamma"], d["gx"], d["ggamma"], ws,
                              residual=d.get("res"))
        return {"gx": d["gx"], "ggamma": d["ggamma"]}
    if op == "linear":
        api.linear_act(d["x"], d["w"], d["y"], bias=d["bias"], act=case["act"], residual=d.get("res"),
                       zq=d.get("zq"), zs=d.get("zs"), yq=d.get("yq"), ys=d.get("ys"))
        out = {"y": d["y"]}
        if case["ckpt"]:
            out["z_values"] = api.ckpt_unpack(d["zq"], d["zs"], d["zv"])
            out["y_values"] = api.ckpt_unpack(d["yq"], d["ys"], d["yv"])
        return out
    if op == "back":
        api.linear_act_grad(d["gy"], d["w"], d["gx"], act=case["act"], zq=d.get("q"), zs=d.get("s"),
                            residual=d.get("res"))
        return {"gx": d["gx"]}
    ws = api.ckpt_grad_w_workspace(case["rows"], case["Cx"], case["Cy"], d["gy"].device)
    api.ckpt_grad_w(d["gy"], d["q"], d["s"], d["gw"], ws, gb=d["gb"], col_scale=d.get("scale"))
    return {"gw": d["gw"], "gb": d["gb"]}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    d = inputs(case, seed)
    op = case["op"]
    a = {k: v.double() for k, v in d.items() if v.dtype in (torch.bfloat16, torch.float32)}

    def rounded(t):  # to 8 bits and back: the power of two from the logarithm
        out = torch.empty_like(t)
        for j in range(0, t.shape[1], GROUP):
            g = t[:, j:j + GROUP]
            top = g.abs().max(1, keepdim=True).values
            # 1e-9: a logarithm that should be whole may come out an ulp above it
            step = torch.exp2(torch.ceil(torch.log2(top / 127) - 1e-9).clamp(-120, 121))
            out[:, j:j + GROUP] = (g / step).round().clamp(-127, 127) * step
        return out

    def decoded(C):  # the codes' values
        step = torch.exp2(d["s"].double() - 127).t().repeat_interleave(GROUP, 1)[:, :C]
        return d["q"][:, :C].double() * step

    if op == "pack":
        return {"values": rounded(a["x"])}
    if op == "norm":
        h = a["x"] + a["res"] if case["res"] else a["x"]
        r = 1 / torch.sqrt((h * h).sum(1) / case["C"] + EPS)
        u = torch.einsum("nc,n->nc", h, r)
        out = {"y": u * a["gamma"], "r": r, "values": rounded(u)}
        if case["res"]:
            out["h"] = h
        return out
    if op == "norm_back":
        u = decoded(case["C"])
        dot = torch.einsum("nc,nc,c->n", a["gy"], u, a["gamma"]) / case["C"]
        gx = (a["gy"] * a["gamma"] - dot[:, None] * u) * a["r"][:, None]
        return {"gx": gx + a["res"] if case["res"] else gx, "ggamma": torch.einsum("nc,nc->c", a["gy"], u)}
    if op == "linear":
        z = torch.addmm(a["bias"], a["x"], a["w"].t())
        y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0),
             "gelu": lambda: z * torch.special.ndtr(z), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        if case["res"]:
            y = y + a["res"]
        out = {"y": y}
        if case["ckpt"]:
            out["z_values"], out["y_values"] = rounded(z), rounded(y)
        return out
    if op == "back":
        g = torch.mm(a["gy"], a["w"])
        if case["act"] != "none":
            z = decoded(case["Cx"])
            if case["act"] == "relu":
                g = torch.where(z > 0, g, 0.0)
            elif case["act"] == "gelu":
                g = g * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5)
            else:
                g = g * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
        return {"gx": g + a["res"] if case["res"] else g}
    gw = torch.mm(a["gy"].t(), decoded(case["Cx"]))
    return {"gw": gw * a["scale"] if case["scale"] else gw, "gb": a["gy"].sum(0)}
