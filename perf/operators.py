"""Measured cases of the operators that stand around the expert layer.

  dispatch / dispatch_grad   tokens to rows sorted by expert, and the gradient back to the tokens
  combine / combine_grad     rows back to tokens with the routing weights, and the gradients of both
  block / block_grad         post-norm, gate, scaled residual and the next pre-norm, in one pass
  linear / linear_grad       (grouped) product with a frozen quantized weight; bias, activation and
                             residual in the epilogue; input and bias gradient

``run`` computes them in plain torch operations (fp32, rounded once) or, with ``own``, through
the library's entry points.
"""
import math

import torch

own = False

# The storage formats' code values (index = code).
NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
       -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
       0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
WEIGHT_BYTES = {"nf4": 0.5 + 4 / 64, "fp4": 0.5 + 4 / 64, "mxfp4": 0.5 + 1 / 32, "bf16": 2.0}
EPS = 1e-6


def listed():
    return [
        # One decode step of 8 sequences into 128 experts: only latency counts.
        dict(name="dispatch_decode", op="dispatch", T=8, k=8, E=128, H=2048, dtype="bf16", pad=0),
        # A prefill batch, 64 experts, top-8: eight copies of every token are written.
        dict(name="dispatch_prefill", op="dispatch", T=4096, k=8, E=64, H=2048, dtype="bf16", pad=0),
        # Training in fp32 on a padded batch of odd length: the input gradient of the dispatch.
        dict(name="dispatch_grad_padded", op="dispatch_grad", T=2047, k=4, E=32, H=2880, dtype="fp32", pad=128),
        # Rows back to tokens after the experts of a prefill with 128 experts, padding at the end.
        dict(name="combine_prefill", op="combine", T=8192, k=8, E=128, H=2048, dtype="bf16", pad=37),
        # Training, the largest batch: gradients of the rows and of the routing weights.
        dict(name="combine_grad_large", op="combine_grad", T=16384, k=2, E=8, H=4096, dtype="bf16", pad=0),
        # One decode token between two layers: combine of 8 rows, post-norm, token gate, residual, next pre-norm.
        dict(name="block_decode", op="block", T=1, k=8, H=2048, dtype="bf16", gate="token", post=True, pre=True),
        # The same stretch over a training batch, dense branch, gate per channel.
        dict(name="block_train", op="block", T=16384, k=0, H=4096, dtype="bf16", gate="channel", post=True, pre=True),
        # Its backward on an odd number of tokens, gate per element.
        dict(name="block_grad_train", op="block_grad", T=8191, k=0, H=2880, dtype="bf16", gate="element", post=True,
             pre=True),
        # One decode token through a projection: the weight stream counts.
        dict(name="linear_decode", op="linear", P=1, E=1, n_in=4096, n_out=14336, fmt="nf4", act="silu", bias=True,
             res=False, save=False),
        # A short batch of 96 rows onto the residual stream: too few rows to fill the GPU with output tiles.
        dict(name="linear_short", op="linear", P=96, E=1, n_in=2880, n_out=2880, fmt="mxfp4", act="none", bias=True,
             res=True, save=False),
        # Non-gated experts of a training batch: 64 experts over the dispatched rows, derivative saved.
        dict(name="linear_experts", op="linear", P=32768, E=64, n_in=2048, n_out=1024, fmt="nf4", act="gelu_tanh",
             bias=True, res=False, save=True),
        # Input and bias gradient of a wide projection over the largest batch.
        dict(name="linear_grad_large", op="linear_grad", P=16384, E=1, n_in=4096, n_out=14336, fmt="nf4", act="silu"),
    ]


def draw(rng):
    """One more case of the same ranges (sizes uniform in their logarithm)."""
    def size(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "block", "block", "block_grad",
                     "block_grad", "linear", "linear", "linear_grad"])
    if op.startswith(("dispatch", "combine")):
        E = rng.choice([4, 8, 32, 60, 64, 128, 256])
        k = rng.choice([1, 2, 4, min(E, 6), min(E, 8)])
        H = rng.choice([size(64, 4096), 64 * size(1, 64)])
        T = min(size(1, 16384), 16384 * 2 * 4096 // (k * H))
        return dict(op=op, T=T, k=k, E=E, H=H, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    pad=rng.choice([0, T // 7]))
    if op.startswith("block"):
        H = rng.choice([size(64, 8192), 64 * size(1, 64)])
        T = min(size(1, 16384), 16384 * 4096 // H)
        post, pre = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op=op, T=T, k=rng.choice([0, 0, 2, 8]) if op == "block" and T <= 4096 else 0, H=H,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    gate=rng.choice(["none", "token", "channel", "element"]), post=post, pre=pre)
    E = rng.choice([1, 1, 1, 8, 64])
    n_in, n_out = 64 * size(2, 96), 64 * size(2, 96)
    P = size(1, 16384)
    if E > 1:
        n_in, n_out = min(n_in, 2048), min(n_out, 2048)
    act = rng.choice(["none", "relu", "silu", "gelu_tanh"])
    fmt = rng.choice(["nf4", "nf4", "fp4", "mxfp4", "bf16"])
    if op == "linear":
        return dict(op=op, P=P, E=E, n_in=n_in, n_out=n_out, fmt=fmt, act=act, bias=rng.random() < 0.5,
                    res=rng.random() < 0.5, save=act != "none" and rng.random() < 0.5)
    return dict(op=op, P=P, E=E, n_in=n_in, n_out=n_out, fmt=fmt, act=act)


def work(c):
    if c["op"].startswith(("dispatch", "combine")):
        T, n, s = c["T"], (c["T"] - c["pad"]) * c["k"], SIZE[c["dtype"]]
        pairs, tok, rows = 4 * T * c["k"], T * c["H"] * s, n * c["H"] * s
        if c["op"] == "dispatch":
            return {"bytes": 2 * pairs + 4 * n + 4 * (c["E"] + 1) + (T - c["pad"]) * c["H"] * s + rows, "flops": 0}
        if c["op"] == "dispatch_grad":
            return {"bytes": pairs + rows + tok, "flops": n * c["H"]}
        if c["op"] == "combine":
            return {"bytes": 2 * pairs + rows + tok, "flops": 2 * n * c["H"]}
        return {"bytes": 3 * pairs + 2 * rows + (T - c["pad"]) * c["H"] * s, "flops": 3 * n * c["H"]}
    if c["op"].startswith("block"):
        T, H, s = c["T"], c["H"], SIZE[c["dtype"]]
        tok = T * H * s
        gate = {"none": 0, "token": 4 * T, "channel": 4 * H, "element": tok}[c["gate"]]
        vec = 4 * H * (c["post"] + c["pre"])
        if c["op"] == "block":
            branch = tok if c["k"] == 0 else c["k"] * (tok + 8 * T)
            return {"bytes": branch + gate + vec + tok * (2 + c["pre"]), "flops": T * H * (12 + 2 * c["k"])}
        return {"bytes": 2 * gate + 2 * vec + tok * (5 + c["pre"]), "flops": 30 * T * H}
    P, E, a, b = c["P"], c["E"], c["n_in"], c["n_out"]
    weights = min(E, P) * a * b * WEIGHT_BYTES[c["fmt"]]
    if c["op"] == "linear":
        rows = 2 * P * (a + b * (1 + c["res"] + c["save"]))
        return {"bytes": weights + rows + 4 * min(E, P) * b * c["bias"], "flops": 2 * P * a * b}
    return {"bytes": weights + 2 * P * (a + b * (1 + (c["act"] != "none"))) + 4 * E * b, "flops": 2 * P * a * b}


# ---------------------------------------------------------------------- inputs

def _quantize(w, fmt):
    """Codes (two a byte, first element high) and block scales of w [E, out, in]; the layouts of include/e4b.h."""
    E, o, i = w.shape
    if fmt == "bf16":
        return w.to(torch.bfloat16).view(torch.uint8).reshape(E, -1), None
    if fmt == "mxfp4":
        blocks = w.view(E, o, i // 32, 32)
        top = blocks.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top.clamp_min(1e-30))) - 2
        mids = torch.tensor([(p + q) / 2 for p, q in zip(E2M1, E2M1[1:])], device=w.device)
        v = blocks / torch.exp2(e)
        code = torch.bucketize(v.abs().contiguous(), mids).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        stride = -(-(i // 32) // 16) * 16
        scales = torch.zeros(E, o, stride, dtype=torch.uint8, device=w.device)
        scales[..., : i // 32] = (e.squeeze(-1) + 127).to(torch.uint8)
    else:
        blocks = w.view(E, o, i // 64, 64)
        top = blocks.abs().amax(-1, keepdim=True)
        if fmt == "nf4":
            mids = torch.tensor([(p + q) / 2 for p, q in zip(NF4, NF4[1:])], device=w.device)
            code = torch.bucketize((blocks / top).contiguous(), mids).to(torch.uint8)
        else:
            mids = torch.tensor([(p + q) / 12 for p, q in zip(E2M1, E2M1[1:])], device=w.device)
            v = blocks / top
            code = torch.bucketize(v.abs().contiguous(), mids).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        scales = top.reshape(E, -1).contiguous()
    code = code.reshape(E, -1, 2)
    return (code[..., 0] << 4 | code[..., 1]).contiguous(), scales


def _routing(c, g):
    """top-k experts (uneven popularity), weights, and the sorted order's maps; padding tokens at the end are routed nowhere."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    top, idx = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, dim=1).contiguous()
    idx = idx.to(torch.int32)
    if c["pad"]:
        idx[T - c["pad"]:] = -1
    return idx.contiguous(), w


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)

    op, s = c["op"], {"case": c}
    if op.startswith(("dispatch", "combine")):
        T, k, H, dt = c["T"], c["k"], c["H"], DTYPES[c["dtype"]]
        s["idx"], s["w"] = _routing(c, g)
        if op == "dispatch":
            s["x"] = randn(T, H, dtype=dt)
            s["rows"] = torch.zeros(T * k, H, dtype=dt, device="cuda")   # rows behind the last expert stay as they are
        else:
            s["inv_perm"] = _sort_pairs(s["idx"], c["E"])[2]
            s["rows"] = randn(T * k, H, dtype=dt)
            s["grad_rows"] = torch.zeros(T * k, H, dtype=dt, device="cuda")
            s["grad_y"] = randn(T, H, dtype=dt)
    elif op.startswith("block"):
        T, H, dt = c["T"], c["H"], DTYPES[c["dtype"]]
        k = c["k"]
        s["scale"] = 0.7
        s["h"] = randn(T, H, dtype=dt, scale=2.0)
        s["post_w"] = randn(H, scale=0.1, shift=1.0) if c["post"] else None
        s["pre_w"] = randn(H, scale=0.1, shift=1.0) if c["pre"] else None
        s["gate"] = {"none": lambda: None, "token": lambda: randn(T), "channel": lambda: randn(H),
                     "element": lambda: randn(T, H, dtype=dt)}[c["gate"]]()
        if k:
            s["rows"] = randn(T * k, H, dtype=dt)
            s["inv_perm"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
            s["w"] = torch.softmax(randn(T, k), dim=1)
        else:
            s["f"] = randn(T, H, dtype=dt)
        if op == "block_grad":   # h holds the stream after the residual sum
            s["grad_o"] = randn(T, H, dtype=dt)
            s["grad_n"] = randn(T, H, dtype=dt) if c["pre"] else None
    else:
        P, E, a, b = c["P"], c["E"], c["n_in"], c["n_out"]
        s["packed"], s["scales"] = _quantize(randn(E, b, a, scale=0.02), c["fmt"])
        s["bias"] = randn(E, b, scale=0.1) if c.get("bias") else None
        s["offsets"] = None
        if E > 1:
            e = torch.randint(0, E, (P,), generator=g, device="cuda")
            n = torch.bincount(e, minlength=E)
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        if op == "linear":
            s["x"] = randn(P, a, dtype=torch.bfloat16)
            s["residual"] = randn(P, b, dtype=torch.bfloat16) if c["res"] else None
        else:
            s["grad_y"] = randn(P, b, dtype=torch.bfloat16)
            s["saved"] = None
            if c["act"] != "none":
                s["saved"] = _act(randn(P, b), c["act"])[1].to(torch.bfloat16)
    if own:
        s["plan"] = _plan(s)
    return s


# ----------------------------------------------------------------- plain forms

def _sort_pairs(idx, E):
    """offsets [E+1], perm [P] (zero behind the last row) and inv_perm [T, k] of the pairs, stable by expert."""
    e = idx.reshape(-1).long()
    e = torch.where((e < 0) | (e >= E), torch.full_like(e, E), e)
    order = torch.argsort(e, stable=True)
    offsets = torch.searchsorted(e[order], torch.arange(E + 1, device=e.device)).to(torch.int32)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(e.numel(), device=e.device)
    inv = torch.where(e == E, torch.full_like(inv, -1), inv)
    perm = torch.where(torch.arange(e.numel(), device=e.device) < offsets[E], order, torch.zeros_like(order))
    return offsets, perm.to(torch.int32), inv.to(torch.int32).view(idx.shape)


def _gathered(rows, inv):
    """rows of every pair [T, k, H] in fp32, zeros for pairs routed nowhere."""
    r = rows[inv.clamp_min(0).long()].float()
    return torch.where((inv < 0)[..., None], torch.zeros_like(r), r)


def _act(z, name):
    """act(z) and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if name == "silu":
        g = torch.sigmoid(z)
        return z * g, g * (1 + z * (1 - g))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _dequantize(s):
    c = s["case"]
    E, o, i = c["E"], c["n_out"], c["n_in"]
    if c["fmt"] == "bf16":
        return s["packed"].view(torch.bfloat16).view(E, o, i).float()
    code = torch.stack([s["packed"] >> 4, s["packed"] & 15], dim=-1).long()
    if c["fmt"] == "nf4":
        table = torch.tensor(NF4, device="cuda")
    else:
        half = torch.tensor(E2M1, device="cuda") / (6 if c["fmt"] == "fp4" else 1)
        table = torch.cat([half, -half])
    v = table[code.reshape(-1)]
    if c["fmt"] == "mxfp4":
        sc = torch.exp2(s["scales"][..., : i // 32].float() - 127)
        w = v.view(E, o, i // 32, 32) * sc[..., None]
    else:
        w = v.view(E, -1, 64) * s["scales"][..., None]
    return w.reshape(E, o, i).to(torch.bfloat16).float()   # the format's values are bf16


def _product(x, w, offsets):
    """x [P, K] times each expert's w [E, K, N] over the expert's rows."""
    if offsets is None:
        return x @ w[0]
    n = (offsets[1:] - offsets[:-1]).long()
    e = torch.repeat_interleave(torch.arange(n.numel(), device=x.device), n)
    at = torch.arange(x.shape[0], device=x.device) - offsets[:-1].long()[e]
    padded = x.new_zeros(n.numel(), int(n.max()), x.shape[1])
    padded[e, at] = x
    return torch.bmm(padded, w)[e, at]


def _expert_rows(s):
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    return torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "dispatch":
        offsets, perm, inv = _sort_pairs(s["idx"], c["E"])
        n = (c["T"] - c["pad"]) * c["k"]
        s["rows"][:n] = s["x"][perm[:n].long() // c["k"]]
        return {"rows": s["rows"], "offsets": offsets, "perm": perm[:n], "inv_perm": inv}
    if op == "dispatch_grad":
        return {"grad_x": _gathered(s["rows"], s["inv_perm"]).sum(1).to(s["rows"].dtype)}
    if op == "combine":
        return {"y": (_gathered(s["rows"], s["inv_perm"]) * s["w"][..., None]).sum(1).to(s["rows"].dtype)}
    if op == "combine_grad":
        inv = s["inv_perm"]
        n = (c["T"] - c["pad"]) * c["k"]
        go = s["grad_y"].float()
        grad_w = (_gathered(s["rows"], inv) * go[:, None]).sum(2)
        live = inv[: c["T"] - c["pad"]].reshape(-1).long()
        pairs = (go[:, None] * s["w"][..., None]).reshape(-1, c["H"])[:n]
        s["grad_rows"][live] = pairs.to(s["rows"].dtype)
        return {"grad_rows": s["grad_rows"], "grad_w": grad_w}
    if op.startswith("block"):
        return _plain_block(s) if op == "block" else _plain_block_grad(s)
    w = _dequantize(s)
    if op == "linear":
        z = _product(s["x"].float(), w.transpose(1, 2), s["offsets"])
        if s["bias"] is not None:
            z = z + (s["bias"][0] if s["offsets"] is None else s["bias"][_expert_rows(s)])
        y, d = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(torch.bfloat16)}
        if c["save"]:
            out["saved"] = d.to(torch.bfloat16)
        return out
    dz = s["grad_y"].float()
    if s["saved"] is not None:
        dz = dz * s["saved"].float()
    if s["offsets"] is None:
        gb = dz.sum(0, keepdim=True)
    else:
        gb = torch.zeros(c["E"], c["n_out"], device="cuda").index_add_(0, _expert_rows(s), dz)
    return {"grad_x": _product(dz, w, s["offsets"]).to(torch.bfloat16), "grad_bias": gb}


def _gate(s):
    g = s["gate"]
    if g is None:
        return None
    g = torch.sigmoid(g.float())
    return g[:, None] if s["case"]["gate"] == "token" else g


def _plain_block(s):
    dt = s["h"].dtype
    f = (_gathered(s["rows"], s["inv_perm"]) * s["w"][..., None]).sum(1) if s["case"]["k"] else s["f"].float()
    if s["post_w"] is not None:
        f = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * s["post_w"]
    g = _gate(s)
    o = s["h"].float() + s["scale"] * (f if g is None else g * f)
    out = {"o": o.to(dt)}
    if s["pre_w"] is not None:
        out["n"] = (o * torch.rsqrt(o.square().mean(1, keepdim=True) + EPS) * s["pre_w"]).to(dt)
    return out


def _plain_block_grad(s):
    dt, out = s["h"].dtype, {}
    o, f, do = s["h"].float(), s["f"].float(), s["grad_o"].float()
    if s["pre_w"] is not None:
        r = torch.rsqrt(o.square().mean(1, keepdim=True) + EPS)
        gn = s["grad_n"].float()
        out["grad_pre_w"] = (gn * o * r).sum(0)
        gn = gn * s["pre_w"]
        do = do + r * (gn - o * r * r * (gn * o).mean(1, keepdim=True))
    out["grad_h"] = do.to(dt)
    b, r = f, None
    if s["post_w"] is not None:
        r = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
        b = f * r * s["post_w"]
    g = _gate(s)
    db = s["scale"] * do
    if g is not None:
        dg = db * b * g * (1 - g)
        out["grad_gate"] = {"token": lambda: dg.sum(1), "channel": lambda: dg.sum(0),
                            "element": lambda: dg.to(dt)}[s["case"]["gate"]]()
        db = db * g
    if r is not None:
        out["grad_post_w"] = (db * f * r).sum(0)
        db = db * s["post_w"]
        db = r * (db - f * r * r * (db * f).mean(1, keepdim=True))
    out["grad_f"] = db.to(dt)
    return out


# ------------------------------------------------------- the library's own calls

def _plan(s):
    """What a program keeps between calls: descriptors, weight handles, workspaces and output buffers."""
    import bit_quantized_mixture_nf4_b200 as e4b
    c, p = s["case"], {"lib": e4b}
    if c["op"] == "dispatch":
        p["ws"] = e4b.dispatch_workspace(c["E"], c["k"], c["T"])
        p["maps"] = (torch.empty(c["E"] + 1, dtype=torch.int32, device="cuda"),
                     torch.zeros(c["T"] * c["k"], dtype=torch.int32, device="cuda"),
                     torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda"))
    elif c["op"].startswith("block"):
        gate = {"none": e4b.GATE_NONE, "token": e4b.GATE_TOKEN, "channel": e4b.GATE_CHANNEL,
                "element": e4b.GATE_ELEMENT}[c["gate"]]
        p["desc"] = e4b.make_block_desc(c["H"], s["h"].dtype, eps=EPS, gate=gate, gate_sigmoid=True,
                                        residual_scale=s["scale"])
        if c["op"] == "block_grad":
            p["ws"] = e4b.block_norm_workspace(p["desc"], c["T"])
    elif c["op"].startswith("linear"):
        fmt = {"nf4": e4b.NF4, "fp4": e4b.FP4, "mxfp4": e4b.MXFP4, "bf16": e4b.BF16_WEIGHTS}[c["fmt"]]
        act = {"none": e4b.LINEAR_ACT_NONE, "relu": e4b.LINEAR_ACT_RELU, "silu": e4b.LINEAR_ACT_SILU,
               "gelu_tanh": e4b.LINEAR_ACT_GELU_TANH}[c["act"]]
        p["desc"] = e4b.make_linear_desc(c["n_in"], c["n_out"], E=c["E"], codebook=fmt, activation=act)
        p["weights"] = e4b.make_linear_weights(s["packed"], s["scales"], s["bias"])
        p["ws"] = e4b.linear_workspace(p["desc"], c["P"])
        if c.get("save"):
            p["saved"] = torch.empty(c["P"], c["n_out"], dtype=torch.bfloat16, device="cuda")
    return p


def _own(s):
    c, p = s["case"], s["plan"]
    op, e4b = c["op"], p["lib"]
    if op == "dispatch":
        offsets, perm, inv = p["maps"]
        e4b.e4b_moe_dispatch(c["E"], s["idx"], s["x"], rows=s["rows"], offsets=offsets, perm=perm, inv_perm=inv,
                             ws=p["ws"])
        return {"rows": s["rows"], "offsets": offsets, "perm": perm[: (c["T"] - c["pad"]) * c["k"]], "inv_perm": inv}
    if op == "dispatch_grad":
        return {"grad_x": e4b.e4b_moe_dispatch_backward(s["rows"], s["inv_perm"])}
    if op == "combine":
        return {"y": e4b.e4b_moe_combine(s["rows"], s["inv_perm"], s["w"])}
    if op == "combine_grad":
        grad_rows, grad_w = e4b.e4b_moe_combine_backward(s["rows"], s["inv_perm"], s["w"], s["grad_y"],
                                                         grad_rows=s["grad_rows"])
        return {"grad_rows": grad_rows, "grad_w": grad_w}
    if op == "block":
        branch = dict(rows=s["rows"], inv_perm=s["inv_perm"], topk_w=s["w"]) if c["k"] else dict(f=s["f"])
        o, n = e4b.e4b_block_norm_forward(p["desc"], s["h"], post_w=s["post_w"], gate=s["gate"], pre_w=s["pre_w"],
                                          **branch)
        return {"o": o} if n is None else {"o": o, "n": n}
    if op == "block_grad":
        got = e4b.e4b_block_norm_backward(p["desc"], s["h"], f=s["f"], post_w=s["post_w"], gate=s["gate"],
                                          pre_w=s["pre_w"], grad_o=s["grad_o"], grad_n=s["grad_n"], ws=p["ws"])
        return {k: v for k, v in got.items() if v is not None}
    if op == "linear":
        y = e4b.e4b_linear_forward(p["desc"], p["weights"], s["x"], offsets=s["offsets"], residual=s["residual"],
                                   saved_d=p.get("saved"), ws=p["ws"])
        return {"y": y, "saved": p["saved"]} if c["save"] else {"y": y}
    grad_x, grad_bias = e4b.e4b_linear_backward(p["desc"], p["weights"], s["grad_y"], offsets=s["offsets"],
                                                saved_d=s["saved"], ws=p["ws"])
    return {"grad_x": grad_x, "grad_bias": grad_bias}


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------- values in 64 bits

def _exact_rms(v, w):
    """v / sqrt(mean v^2 + eps) * w, row by row."""
    return v / (v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * w


def _exact_weight(s, e):
    """Expert e's weight [out, in] in fp64, from the stored bytes."""
    c = s["case"]
    o, i = c["n_out"], c["n_in"]
    raw = s["packed"][e]
    if c["fmt"] == "bf16":
        return raw.view(torch.bfloat16).view(o, i).double()
    v = torch.empty(o * i, dtype=torch.float64, device="cuda")
    pos = [float(x) for x in E2M1]
    codes = list(NF4) if c["fmt"] == "nf4" else [x / (6 if c["fmt"] == "fp4" else 1) for x in pos + [-x for x in pos]]
    table = torch.tensor(codes, dtype=torch.float64, device="cuda").float().double()
    v[0::2] = table[(raw // 16).long()]
    v[1::2] = table[(raw % 16).long()]
    if c["fmt"] == "mxfp4":
        scale = 2.0 ** (s["scales"][e][:, : i // 32].double() - 127)
        return (v.view(o, i // 32, 32) * scale[..., None]).view(o, i)   # exact in bf16
    w = v.view(-1, 64) * s["scales"][e].double()[:, None]
    # the format defines one fp32 product, then bf16
    return w.float().to(torch.bfloat16).double().view(o, i)


def _exact_act(z, name):
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, z * 0), torch.where(z > 0, 1.0, 0.0).double()
    u = z if name == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
    du = torch.ones_like(z) if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z.pow(2))
    p = 1 / (1 + torch.exp(-u))   # gelu_tanh(z) = z * logistic(2 u), silu(z) = z * logistic(z)
    return z * p, p + z * p * (1 - p) * du


def exact(c, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    op = c["op"]
    if op.startswith("linear"):
        return _exact_linear(c, s)
    if op == "block":
        return _exact_block(c, s)
    if op == "block_grad":
        return _exact_block_grad(c, s)
    T, k, H = c["T"], c["k"], c["H"]
    if op == "dispatch":
        idx = s["idx"].reshape(-1)
        hit = (idx[:, None] == torch.arange(c["E"], device="cuda")).int()
        first = hit.sum(0).cumsum(0) - hit.sum(0)
        place = ((hit.cumsum(0) - 1 + first) * hit).sum(1)
        live = idx >= 0
        rows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        token = torch.arange(T, device="cuda").repeat_interleave(k)
        rows[place[live].long()] = s["x"][token[live]].double()
        return {"rows": rows, "offsets": None, "perm": None, "inv_perm": None}
    inv, rows = s["inv_perm"], s["rows"]
    acc = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    grad_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    grad_rows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        live = inv[:, j] >= 0
        at = inv[live, j].long()
        if op == "dispatch_grad":
            acc[live] += rows[at].double()
        elif op == "combine":
            acc[live] += s["w"][live, j].double()[:, None] * rows[at].double()
        else:
            grad_rows[at] = s["w"][live, j].double()[:, None] * s["grad_y"][live].double()
            grad_w[live, j] = torch.einsum("th,th->t", s["grad_y"][live].double(), rows[at].double())
    return {"dispatch_grad": {"grad_x": acc}, "combine": {"y": acc},
            "combine_grad": {"grad_rows": grad_rows, "grad_w": grad_w}}[op]


def _exact_block(c, s):
    h = s["h"].double()
    if c["k"]:
        f = torch.zeros_like(h)
        for j in range(c["k"]):
            f += s["rows"][s["inv_perm"][:, j].long()].double() * s["w"][:, j].double()[:, None]
    else:
        f = s["f"].double()
    if c["post"]:
        f = _exact_rms(f, s["post_w"].double())
    if c["gate"] != "none":
        g = 1 / (1 + torch.exp(-s["gate"].double()))
        f = f * (g.view(-1, 1) if c["gate"] == "token" else g)
    o = h + s["scale"] * f
    return {"o": o, "n": _exact_rms(o, s["pre_w"].double())} if c["pre"] else {"o": o}


def _exact_block_grad(c, s):
    """Through autograd in fp64, from the stored stream: o = (o - s g b) + s g b."""
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    o0, f = s["h"].double(), leaf(s["f"])
    post = leaf(s["post_w"]) if c["post"] else None
    pre = leaf(s["pre_w"]) if c["pre"] else None
    gate = leaf(s["gate"]) if c["gate"] != "none" else None
    b = f if post is None else _exact_rms(f, post)
    if gate is not None:
        g = 1 / (1 + torch.exp(-gate))
        b = b * (g.view(-1, 1) if c["gate"] == "token" else g)
    b = s["scale"] * b
    h = (o0 - b.detach()).requires_grad_()
    o = h + b
    total = (o * s["grad_o"].double()).sum()
    if pre is not None:
        total = total + (_exact_rms(o, pre) * s["grad_n"].double()).sum()
    total.backward()
    out = {"grad_h": h.grad, "grad_f": f.grad}
    for name, t in (("grad_post_w", post), ("grad_pre_w", pre), ("grad_gate", gate)):
        if t is not None:
            out[name] = t.grad
    return out


def _exact_linear(c, s):
    P, E, a, b = c["P"], c["E"], c["n_in"], c["n_out"]
    ends = [0, P] if E == 1 else s["offsets"].tolist()
    if c["op"] == "linear":
        y = torch.zeros(P, b, dtype=torch.float64, device="cuda")
        d = torch.zeros(P, b, dtype=torch.float64, device="cuda") if c["save"] else None
        for e in range(E):
            r = slice(ends[e], ends[e + 1])
            if r.stop > r.start:
                z = s["x"][r].double() @ _exact_weight(s, e).t()
                if c["bias"]:
                    z += s["bias"][e].double()
                y[r], der = _exact_act(z, c["act"])
                if d is not None:
                    d[r] = der
        if c["res"]:
            y += s["residual"].double()
        return {"y": y, "saved": d} if c["save"] else {"y": y}
    gx = torch.zeros(P, a, dtype=torch.float64, device="cuda")
    gb = torch.zeros(E, b, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        if r.stop > r.start:
            dz = s["grad_y"][r].double()
            if c["act"] != "none":
                dz = dz * s["saved"][r].double()
            gx[r] = dz @ _exact_weight(s, e)
            gb[e] = dz.sum(0)
    return {"grad_x": gx, "grad_bias": gb}
