"""e4b_linear_forward / backward against a plain product in 64 bits of the storage format's
own bf16 values (from the oracle's dequantization), in every format, dense and grouped."""
import numpy as np
import pytest
import torch

import oracle
from tests import _ops

pytestmark = pytest.mark.gpu

NONE, RELU, SILU, GELU = range(4)
FORMATS = {"nf4": 0, "fp4": 1, "mxfp4": 2, "int8": 3, "fp8": 4, "bf16": 5}


@pytest.fixture(scope="module")
def e4b():
    import bit_quantized_mixture_nf4_b200 as m
    m.lib
    return m


def _weights(e4b, E, o, i, fmt, bias, seed):
    """(handle, W fp64 [E, o, i], bias fp64 or None); codes and values by the oracle."""
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((E, o, i)) * 0.05).astype(np.float32)
    cb = FORMATS[fmt]
    if fmt == "bf16":
        t = torch.from_numpy(w).to(torch.bfloat16)
        packed, scale, val = t.contiguous(), None, t.double()
    elif fmt == "mxfp4":
        p, s = oracle.quantize_mxfp4(w)
        packed, scale, val = torch.from_numpy(p), torch.from_numpy(s), oracle.dequantize_mxfp4(p, s, (E, o, i))
    elif fmt in ("int8", "fp8"):
        p, s = oracle.quantize8(w, cb)
        packed, scale, val = torch.from_numpy(p), torch.from_numpy(s), oracle.dequantize8(p, s, (E, o, i), cb)
    else:
        p, s = oracle.quantize(w, cb)
        packed, scale, val = torch.from_numpy(p), torch.from_numpy(s), oracle.dequantize(p, s, (E, o, i), cb)
    if not torch.is_tensor(val):
        val = torch.from_numpy(np.asarray(val, np.float64)).reshape(E, o, i)
    b = torch.from_numpy(rng.standard_normal((E, o)).astype(np.float32) * 0.3) if bias else None
    h = e4b.make_linear_weights(packed.cuda(), None if scale is None else scale.cuda(), None if b is None else b.cuda())
    return h, val, None if b is None else b.double()


def _offsets(E, P, seed, lo=0, hi=None):
    """Uneven expert ranges inside [lo, hi), some of them empty."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(lo, (P if hi is None else hi) + 1, (E - 1,), generator=g).sort().values.tolist()
    return torch.tensor([lo] + cuts + [P if hi is None else hi], dtype=torch.int32)


def _reference(x, W, b, offs, kind, P, E):
    """y, act', and their error bounds' magnitudes over the experts' rows (zeros elsewhere)."""
    o = W.shape[1]
    z, zm = torch.zeros(P, o, dtype=torch.float64), torch.zeros(P, o, dtype=torch.float64)
    live = torch.zeros(P, dtype=torch.bool)
    for e, (r0, r1) in enumerate(_ops.expert_rows(offs, E, P)):
        z[r0:r1] = x[r0:r1].double() @ W[e].t()
        zm[r0:r1] = x[r0:r1].double().abs() @ W[e].abs().t()
        if b is not None:
            z[r0:r1] += b[e]
            zm[r0:r1] += b[e].abs()
        live[r0:r1] = True
    y, d = _ops.act(z, kind)
    return z, zm, y, d, live


def _bounds(K, z, zm, kind):
    """Errors of act(z) and act'(z) before their rounding.  z: the tensor cores add K products in
    fp32 without rounding each sum to nearest, at most a step 2^-23 of the magnitude per addition.
    act: slope at most 1.13, act' : slope at most 1; the logistic function by __expf and a fast
    quotient is off by a few 2^-22 (2 + |u|), times |z| s (1 - s) <= 0.3 there."""
    ze = (K + 8) * 2.0 ** -23 * zm
    extra = 0.0 if kind in (NONE, RELU) else 2.0 ** -18 * (1 + z.abs().clamp_max(10))
    return ze, 1.13 * ze + extra, (1.0 if kind != RELU else 0.0) * ze + extra


def _near(got, ref, err, u, what):
    tol = err + u * (ref.abs() + err) + 1e-37
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), ((got.double() - ref).abs() / tol).nan_to_num(9e9).max().item())


def _check(e4b, P, E, i, o, fmt, kind, bias, res, save, seed, offs=None, backward=True):
    W, val, b = _weights(e4b, E, o, i, fmt, bias, seed)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(P, i, generator=g).to(torch.bfloat16)
    r = torch.randn(P, o, generator=g).to(torch.bfloat16) if res else None
    gy = torch.randn(P, o, generator=g).to(torch.bfloat16)
    if offs is None and E > 1:
        offs = _offsets(E, P, seed)
    od = None if offs is None else offs.cuda()
    desc = e4b.make_linear_desc(i, o, E=E, codebook=FORMATS[fmt], activation=kind)
    y = torch.full((P, o), 3.0, dtype=torch.bfloat16, device="cuda")
    saved = torch.full((P, o), 3.0, dtype=torch.bfloat16, device="cuda") if save else None
    e4b.e4b_linear_forward(desc, W, x.cuda(), offsets=od, residual=None if r is None else r.cuda(), y=y, saved_d=saved)
    z, zm, ry, rd, live = _reference(x, val, b, offs, kind, P, E)
    ze, ye, de = _bounds(i, z, zm, kind)
    u = 2.0 ** -8
    full = ry if r is None else ry + r.double()
    extra = 0.0 if r is None else 2.0 ** -24 * (ry.abs() + r.double().abs())
    _near(y.cpu()[live], full[live], (ye + extra)[live], u, "y")
    assert bool((y.cpu()[~live] == 3).all())
    if save:
        ok = saved.cpu()
        if kind == RELU:   # the step lies anywhere within the error of z
            near = (z.abs() <= ze)
            assert bool(((ok == 0) | (ok == 1))[live].all())
            assert torch.equal(ok.double()[live & ~near.any(1)], rd[live & ~near.any(1)])
        else:
            _near(ok[live], rd[live], de[live], u, "saved")
        assert bool((ok[~live] == 3).all())
    if not backward:
        return
    # the backward takes the derivative as stored, so its reference does too
    sd = saved if save else None
    if kind != NONE and sd is None:
        sd = torch.zeros(P, o, dtype=torch.bfloat16, device="cuda")
        e4b.e4b_linear_forward(desc, W, x.cuda(), offsets=od, saved_d=sd)
    gx = torch.full((P, i), 3.0, dtype=torch.bfloat16, device="cuda")
    gx, gb = e4b.e4b_linear_backward(desc, W, gy.cuda(), x=x.cuda(), offsets=od, saved_d=saved, grad_x=gx)
    dz = gy.double() if kind == NONE else gy.double() * sd.cpu().double()
    dzb = dz.to(torch.bfloat16).double()   # the products of two bf16 are exact in fp32, so this rounding is known
    rx, xm = torch.zeros(P, i, dtype=torch.float64), torch.zeros(P, i, dtype=torch.float64)
    rb, bm = torch.zeros(E, o, dtype=torch.float64), torch.zeros(E, o, dtype=torch.float64)
    for e, (r0, r1) in enumerate(_ops.expert_rows(offs, E, P)):
        rx[r0:r1] = dzb[r0:r1] @ val[e]
        xm[r0:r1] = dzb[r0:r1].abs() @ val[e].abs()
        rb[e] = dz[r0:r1].sum(0)
        bm[e] = dz[r0:r1].abs().sum(0)
    _near(gx.cpu()[live], rx[live], ((o + 8) * 2.0 ** -23 * xm)[live], u, "grad_x")
    assert bool((gx.cpu()[~live] == 3).all())
    _near(gb.cpu(), rb, (P + 8) * 2.0 ** -24 * bm, 2.0 ** -24, "grad_bias")
    if save:   # the derivative recomputed from x gives the same bits
        gx2, gb2 = e4b.e4b_linear_backward(desc, W, gy.cuda(), x=x.cuda(), offsets=od)
        assert torch.equal(gx2.cpu()[live], gx.cpu()[live]) and torch.equal(gb2, gb)
    assert e4b.e4b_device_status() == 0


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("P", [1, 8, 9, 16, 17, 33, 300])
def test_formats_and_row_counts(e4b, fmt, P):
    _check(e4b, P, 1, 320, 192, fmt, SILU, True, True, True, seed=P)


@pytest.mark.parametrize("kind", [NONE, RELU, SILU, GELU])
@pytest.mark.parametrize("bias,res,save", [(False, False, False), (True, False, True), (False, True, False),
                                           (True, True, True)])
@pytest.mark.parametrize("P", [5, 260])
def test_epilogues(e4b, kind, bias, res, save, P):
    _check(e4b, P, 1, 256, 320, "nf4", kind, bias, res, save, seed=40 + kind)


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4", "bf16", "int8"])
@pytest.mark.parametrize("P,E", [(1, 8), (7, 256), (12, 3), (13, 3), (200, 5), (900, 17), (40, 64), (256, 64), (257, 64), (1024, 256)])
def test_grouped(e4b, fmt, P, E):
    _check(e4b, P, E, 128, 192, fmt, GELU, True, True, True, seed=P + E)


@pytest.mark.parametrize("P", [20, 700])
def test_rows_outside_the_experts_are_left(e4b, P):
    _check(e4b, P, 4, 192, 128, "nf4", SILU, True, True, True, seed=3, offs=_offsets(4, P, 5, 3, P - 4))
    _check(e4b, P, 1, 192, 128, "nf4", SILU, True, True, True, seed=3, offs=torch.tensor([2, P - 3], dtype=torch.int32))
    _check(e4b, P, 3, 192, 128, "nf4", NONE, False, False, False, seed=3, offs=torch.tensor([4] * 4, dtype=torch.int32))


def test_offsets_out_of_range_are_clamped(e4b):
    """Descending or out-of-range offsets are read as their running maximum inside [0, P]."""
    for P in (30, 600):
        W, val, b = _weights(e4b, 4, 128, 64, "nf4", True, 9)
        x = torch.randn(P, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        gy = torch.randn(P, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
        desc = e4b.make_linear_desc(64, 128, E=4)
        outs = []
        for o in ([-5, 10, 4, 2 ** 31 - 1, 7], [0, 10, 10, P, P]):
            offs = torch.tensor(o, dtype=torch.int32).cuda()
            outs.append((e4b.e4b_linear_forward(desc, W, x, offsets=offs),
                         *e4b.e4b_linear_backward(desc, W, gy, offsets=offs)))
        assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("P,i,o", [(1, 64, 64), (2, 2880, 64), (17, 64, 2880), (64, 2880, 2880), (96, 4096, 256),
                                   (513, 64, 128), (1030, 128, 64), (257, 1024, 576)])
def test_sizes(e4b, P, i, o):
    """Single blocks, ragged tiles, split sums (few tiles, long K) in both directions."""
    _check(e4b, P, 1, i, o, "nf4", NONE, True, True, False, seed=P)
    _check(e4b, P, 1, i, o, "fp4", SILU, True, False, True, seed=P + 1)


@pytest.mark.parametrize("fmt", ["nf4", "bf16"])
@pytest.mark.parametrize("P,i", [(3, 64), (8, 192), (16, 320), (40, 192)])
def test_infinities_stay_in_their_rows_and_columns(e4b, fmt, P, i):
    """An infinity in one row of x (at the end of a K that fills no step) spoils that row alone."""
    W, val, _ = _weights(e4b, 1, 128, i, fmt, False, 12)
    x = torch.randn(P, i, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    desc = e4b.make_linear_desc(i, 128, codebook=FORMATS[fmt])
    y = e4b.e4b_linear_forward(desc, W, x)
    for col in (0, i - 1):
        x2 = x.clone()
        x2[P - 1, col] = float("inf")
        y2 = e4b.e4b_linear_forward(desc, W, x2)
        assert torch.equal(y2[:-1], y[:-1])
        w = val[0, :, col]
        want = torch.where(w > 0, float("inf"), torch.where(w < 0, -float("inf"), float("nan"))).to(torch.bfloat16)
        assert torch.equal(y2[-1].cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_residual_in_place_and_repeat(e4b):
    for P in (6, 500, 3000):
        W, _, _ = _weights(e4b, 1, 256, 192, "nf4", True, 4)
        x = torch.randn(P, 192, device="cuda").to(torch.bfloat16)
        r = torch.randn(P, 256, device="cuda").to(torch.bfloat16)
        desc = e4b.make_linear_desc(192, 256, activation=SILU)
        y = e4b.e4b_linear_forward(desc, W, x, residual=r)
        r2 = r.clone()
        e4b.e4b_linear_forward(desc, W, x, residual=r2, y=r2)
        assert torch.equal(y, r2)
        assert torch.equal(y, e4b.e4b_linear_forward(desc, W, x, residual=r))


def test_activations_at_the_ends_of_the_range(e4b):
    """Large, tiny, infinite and NaN pre-activations (by the bias of a zero weight)."""
    zs = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 50.0, -50.0, 87.5, -87.5, 200.0, -200.0, 1e20, -1e20, 3e38, -3e38,
                       float("inf"), float("nan")])
    bias = torch.zeros(1, 64)
    bias[0, :16] = zs
    W = e4b.make_linear_weights(torch.zeros(1, 64, 64, dtype=torch.bfloat16, device="cuda"), None, bias.cuda())
    for P in (2, 40):
        x = torch.ones(P, 64, dtype=torch.bfloat16, device="cuda")
        for kind in (RELU, SILU, GELU):
            saved = torch.empty(P, 64, dtype=torch.bfloat16, device="cuda")
            y = e4b.e4b_linear_forward(e4b.make_linear_desc(64, 64, codebook=5, activation=kind), W, x, saved_d=saved)
            y, d = y[0, :16].cpu().double(), saved[0, :16].cpu().double()
            # beyond |z| = 50: y is z (to bf16) or 0, the derivative 1 or 0
            big = torch.tensor([4, 6, 8, 10, 12])
            want = zs[big].to(torch.bfloat16).double()
            assert torch.equal(y[big], want) and bool((d[big] == 1).all())
            assert bool((y[big + 1].abs() < 1e-19).all()) and bool((d[big + 1].abs() < 1e-18).all())
            assert y[14] == float("inf") and bool(y[15].isnan())
            assert bool((y[:4].abs() < 1e-29).all())


def test_gradient_against_differences(e4b):
    """The derivative saved by the forward against a central difference of y over the bias."""
    P, i, o = 40, 64, 64
    W, val, _ = _weights(e4b, 1, o, i, "nf4", False, 6)
    x = torch.randn(P, i, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    packed, scale, _ = W._tensors
    for kind in (SILU, GELU):
        desc = e4b.make_linear_desc(i, o, activation=kind)
        saved = torch.empty(P, o, dtype=torch.bfloat16, device="cuda")
        e4b.e4b_linear_forward(desc, W, x, saved_d=saved)
        h = 0.5   # bf16 outputs: a wide step, and the exact difference quotient by the formula beside it
        ys = [e4b.e4b_linear_forward(desc, e4b.make_linear_weights(packed, scale, torch.full((1, o), s, device="cuda")), x)
              .cpu().double() for s in (h, -h)]
        z = x.cpu().double() @ val[0].t()
        want = (_ops.act(z + h, kind)[0] - _ops.act(z - h, kind)[0]) / (2 * h)
        got = (ys[0] - ys[1]) / (2 * h)
        # two roundings of y over the step
        tol = 2.0 ** -8 * (ys[0].abs() + ys[1].abs()) / (2 * h) + 1e-3
        assert bool(((got - want).abs() <= tol).all())
        # the derivative is the quotient up to the third derivative (at most 1.5) times h^2 / 6
        assert bool(((saved.cpu().double() - got).abs() <= tol + 1.5 * h * h / 6 + 2.0 ** -8).all())


def test_empty_and_graph(e4b):
    W, _, _ = _weights(e4b, 3, 192, 128, "nf4", True, 8)
    desc = e4b.make_linear_desc(128, 192, E=3, activation=SILU)
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert e4b.e4b_linear_forward(desc, W, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), offsets=offs).shape == (0, 192)
    gx, gb = e4b.e4b_linear_backward(desc, W, torch.empty(0, 192, dtype=torch.bfloat16, device="cuda"), offsets=offs,
                                     saved_d=torch.empty(0, 192, dtype=torch.bfloat16, device="cuda"))
    assert gx.shape == (0, 128) and not bool(gb.any())
    for P in (16, 700):
        x = torch.randn(P, 128, device="cuda").to(torch.bfloat16)
        gy = torch.randn(P, 192, device="cuda").to(torch.bfloat16)
        offs = _offsets(3, P, 1).cuda()

        def step():
            saved = torch.empty(P, 192, dtype=torch.bfloat16, device="cuda")
            y = e4b.e4b_linear_forward(desc, W, x, offsets=offs, saved_d=saved)
            return [y, saved, *e4b.e4b_linear_backward(desc, W, gy, offsets=offs, saved_d=saved)]

        step()
        torch.cuda.synchronize()
        graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        with torch.cuda.graph(other):   # a second graph with its own workspaces
            out2 = step()
        offs.copy_(_offsets(3, P, 2))
        x.neg_()
        eager = step()
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(eager, out, out2):
            assert torch.equal(a, b) and torch.equal(a, c)
    assert e4b.e4b_device_status() == 0


@pytest.mark.parametrize("P,E,fmt", [(40, 1, "nf4"), (600, 1, "bf16"), (900, 5, "mxfp4")])
def test_input_gradient_stays_within_the_rounding_of_dz(e4b, P, E, fmt):
    """grad_x against the product of the unrounded dz.  Each dz is off by at most half a bf16 step,
    2^-8 of it, so an element of grad_x is off by 2^-8 sum |dz| |W| next to its own rounding.  In the
    2-norm the roundings are independent and spread over +-2^-8: 2^-8 / sqrt(3) from dz and as much
    from the result, sqrt(2) times that together; twice that is allowed."""
    i, o = 320, 1024
    W, val, _ = _weights(e4b, E, o, i, fmt, False, 50 + P)
    g = torch.Generator().manual_seed(P)
    gy, sd = torch.randn(P, o, generator=g).to(torch.bfloat16), torch.rand(P, o, generator=g).to(torch.bfloat16)
    offs = None if E == 1 else _offsets(E, P, P)
    desc = e4b.make_linear_desc(i, o, E=E, codebook=FORMATS[fmt], activation=SILU)
    gx, _ = e4b.e4b_linear_backward(desc, W, gy.cuda(), offsets=None if offs is None else offs.cuda(), saved_d=sd.cuda())
    dz = gy.double() * sd.double()
    rx, xm = torch.zeros(P, i, dtype=torch.float64), torch.zeros(P, i, dtype=torch.float64)
    for e, (r0, r1) in enumerate(_ops.expert_rows(offs, E, P)):
        rx[r0:r1], xm[r0:r1] = dz[r0:r1] @ val[e], dz[r0:r1].abs() @ val[e].abs()
    _near(gx.cpu(), rx, (2.0 ** -8 + (o + 8) * 2.0 ** -23) * xm, 2.0 ** -8, "grad_x")
    off = ((gx.cpu().double() - rx).norm() / rx.norm()).item()
    assert off <= 2 * (2 / 3) ** 0.5 * 2.0 ** -8, off


@pytest.mark.parametrize("P,E", [(300, 1), (700, 1), (900, 3)])
def test_more_column_tiles_than_a_group(e4b, P, E):
    """Over 16 column tiles of 256 (a group, a remainder and a ragged last tile), in both directions."""
    _check(e4b, P, E, 64, 4416, "nf4", SILU, True, True, True, seed=P)
    _check(e4b, P, E, 4416, 64, "mxfp4", NONE, True, False, False, seed=P + 1)
    _check(e4b, P, E, 320, 8256, "bf16", GELU, False, True, True, seed=P + 2, backward=False)


@pytest.mark.parametrize("i,o,E", [(2880, 576, 1), (1024, 256, 1), (192, 128, 3)])
def test_short_calls_in_the_largest_batchs_workspace(e4b, i, o, E):
    """One workspace, sized for 4096 rows and no larger, for calls of every kind of size."""
    W, _, _ = _weights(e4b, E, o, i, "nf4", True, 31)
    desc = e4b.make_linear_desc(i, o, E=E)
    ws = torch.full((e4b.e4b_linear_workspace_size(desc, 4096),), 0xFF, dtype=torch.uint8, device="cuda")
    for P in (1, 16, 17, 96, 256, 257, 512, 1024, 4096):
        g = torch.Generator().manual_seed(P)
        x, gy = (torch.randn(P, n, generator=g).to(torch.bfloat16).cuda() for n in (i, o))
        offs = None if E == 1 else _offsets(E, P, 3).cuda()
        want = [e4b.e4b_linear_forward(desc, W, x, offsets=offs), *e4b.e4b_linear_backward(desc, W, gy, offsets=offs)]
        got = [e4b.e4b_linear_forward(desc, W, x, offsets=offs, ws=ws),
               *e4b.e4b_linear_backward(desc, W, gy, offsets=offs, ws=ws)]
        assert all(torch.equal(a, b) for a, b in zip(want, got)), P


@pytest.mark.parametrize("P,E,fmt", [(3, 1, "nf4"), (3, 1, "fp8"), (96, 1, "mxfp4"), (700, 1, "nf4"), (900, 5, "int8")])
def test_forward_in_a_workspace_of_its_own_size(e4b, P, E, fmt):
    """What lies behind the forward's workspace is not touched, and too small a one is refused."""
    i, o = 1024, 320
    W, _, _ = _weights(e4b, E, o, i, fmt, True, 33)
    desc = e4b.make_linear_desc(i, o, E=E, codebook=FORMATS[fmt], activation=SILU)
    x = torch.randn(P, i, generator=torch.Generator().manual_seed(P)).to(torch.bfloat16).cuda()
    offs = None if E == 1 else _offsets(E, P, 3).cuda()
    n = e4b.e4b_linear_forward_workspace_size(desc, P)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    saved = torch.empty(P, o, dtype=torch.bfloat16, device="cuda")
    y = e4b.e4b_linear_forward(desc, W, x, offsets=offs, saved_d=saved, ws=buf[:n])
    assert bool((buf[n:] == 0xA5).all())
    full = torch.empty_like(saved)
    ws = e4b.linear_workspace(desc, P)
    assert torch.equal(y, e4b.e4b_linear_forward(desc, W, x, offsets=offs, saved_d=full, ws=ws)) and torch.equal(saved, full)
    with pytest.raises(e4b.E4BError):
        e4b.e4b_linear_forward(desc, W, x, offsets=offs, ws=buf[:256])
