"""Plain 64-bit statements of the operators around the expert layer, with the magnitudes
that their rounding errors are measured by.

Tolerances: an fp32 result computed with about c roundings from terms whose absolute values
sum to m is off by at most c 2^-24 m; an output of type t adds half a step of its own,
u(t) = eps(t) / 2 relative (2^-8 for bf16, 2^-24 for fp32)."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U24 = 2.0 ** -24


def unit(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_near(got, ref, mag, c, what=""):
    """|got - ref| <= c 2^-24 mag + u |ref| (+ u of the first term), element by element."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    got64, u = got.to(F64), unit(got.dtype)
    err = c * U24 * mag
    tol = err + u * (ref.abs() + err) + 1e-37
    bad = ~((got64 - ref).abs() <= tol)
    if bool(bad.any()):
        i = int(((got64 - ref).abs() / tol).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: "
                             f"{got64.flatten()[i].item()} against {ref.flatten()[i].item()}, "
                             f"allowed {tol.flatten()[i].item():.3e}")


# --------------------------------------------------------------- dispatch / combine

def sort_pairs(idx, E):
    """offsets, perm (rows only) and inv_perm of topk_idx [T, k], by a plain loop."""
    T, k = idx.shape
    flat = idx.flatten().tolist()
    order = sorted((p for p in range(T * k) if 0 <= flat[p] < E), key=lambda p: flat[p])   # sorted() is stable
    offsets = [0] * (E + 1)
    for p in order:
        offsets[flat[p] + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    inv = [-1] * (T * k)
    for r, p in enumerate(order):
        inv[p] = r
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(order), i32(inv).view(T, k)


def combine(rows, inv, w):
    """(sum, sum of absolute values) of the weighted rows."""
    T, k = inv.shape
    ok = (inv >= 0) & (inv < rows.shape[0])
    r = rows.to(F64)[inv.clamp(0, rows.shape[0] - 1).long()] * ok[..., None]
    r = torch.where(ok[..., None], r, torch.zeros_like(r))
    if w is not None:
        r = torch.where(ok[..., None], r * w.to(F64)[..., None], r)
    return r.sum(1), r.abs().sum(1)


# ----------------------------------------------------------------------- block norm

def block_forward(h, f, post_w, gate, kind, sig, pre_w, eps, off, scale, fmag=None):
    """o, n and their magnitudes; kind: 0 none, 1 token, 2 channel, 3 element."""
    h, f = h.to(F64), None if f is None else f.to(F64)
    o, om = h, h.abs()
    if f is not None:
        fm = f.abs() if fmag is None else fmag
        b, bm = f, fm
        if post_w is not None:
            w = post_w.to(F64) + off
            r = 1 / torch.sqrt(f.pow(2).mean(1, keepdim=True) + eps)
            b, bm = f * r * w, fm * r * w.abs()
        g = 1.0
        if kind:
            g = gate.to(F64)
            g = 1 / (1 + torch.exp(-g)) if sig else g
            g = g[:, None] if kind == 1 else g
        o = h + scale * g * b
        om = h.abs() + (scale * g * bm).abs() if kind else h.abs() + abs(scale) * bm
    n = nm = None
    if pre_w is not None:
        r = 1 / torch.sqrt(o.pow(2).mean(1, keepdim=True) + eps)
        w = pre_w.to(F64) + off
        n, nm = o * r * w, om * r * w.abs()
    return o, om, n, nm


def block_backward(o, f, post_w, gate, kind, sig, pre_w, eps, off, scale, go, gn):
    """{name: (gradient, magnitude)} by the closed formulas."""
    out = {}
    d = torch.zeros_like(gn, dtype=F64) if go is None else go.to(F64)
    dm = d.abs()
    if pre_w is not None:
        o, u0 = o.to(F64), gn.to(F64)
        w = pre_w.to(F64) + off
        r = 1 / torch.sqrt(o.pow(2).mean(1, keepdim=True) + eps)
        u = u0 * w
        d = d + r * (u - o * r * r * (u * o).mean(1, keepdim=True))
        dm = dm + r * (u.abs() + o.abs() * r * r * (u * o).abs().mean(1, keepdim=True))
        out["grad_pre_w"] = ((u0 * o * r).sum(0), (u0 * o * r).abs().sum(0))
    out["grad_h"] = (d, dm)
    if f is None:
        return out
    f = f.to(F64)
    r, w = 1.0, 1.0
    if post_w is not None:
        r = 1 / torch.sqrt(f.pow(2).mean(1, keepdim=True) + eps)
        w = post_w.to(F64) + off
    b = f * r * w
    g, gd = 1.0, 1.0
    if kind:
        g = gate.to(F64)
        if sig:
            g = 1 / (1 + torch.exp(-g))
            gd = g * (1 - g)
        if kind == 1:
            g, gd = g[:, None], gd[:, None] if sig else gd
    db, dbm = scale * d, abs(scale) * dm
    if kind:
        dg, dgm = db * b * gd, dbm * (b * gd).abs()
        red = {1: lambda t: t.sum(1), 2: lambda t: t.sum(0), 3: lambda t: t}[kind]
        out["grad_gate"] = (red(dg), red(dgm))
    db, dbm = db * g, dbm * (abs(g) if not torch.is_tensor(g) else g.abs())
    if post_w is not None:
        out["grad_post_w"] = ((db * f * r).sum(0), (dbm * (f * r).abs()).sum(0))
        v, vm = db * w, dbm * w.abs()
        db = r * (v - f * r * r * (v * f).mean(1, keepdim=True))
        dbm = r * (vm + f.abs() * r * r * (vm * f.abs()).mean(1, keepdim=True))
    out["grad_f"] = (db, dbm)
    return out


# --------------------------------------------------------------------------- linear

def act(z, kind):
    """act(z), act'(z) for NONE, RELU, SILU, GELU_TANH (0..3)."""
    if kind == 0:
        return z, torch.ones_like(z)
    if kind == 1:
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if kind == 2:
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def expert_rows(offsets, E, P):
    """[(begin, end)] of every expert."""
    if offsets is None:
        return [(0, P)]
    o = offsets.tolist()
    return [(o[e], o[e + 1]) for e in range(E)]
