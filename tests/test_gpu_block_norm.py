"""e4b_block_norm_forward / backward against the formulas in 64 bits."""
import pytest
import torch

from tests import _ops

pytestmark = pytest.mark.gpu

# roundings between load and store: a row sum of squares over 8 serial terms and two trees of
# 5 levels (18), its mean, rsqrt (2 ulp = 4 half steps) and the products, each counted against
# the row's magnitudes; expf of the gate (2 ulp) and its quotient
C_FWD, C_BWD = 64, 128


@pytest.fixture(scope="module")
def e4b():
    import bit_quantized_mixture_nf4_b200 as m
    m.lib
    return m


def _inputs(T, H, dtype, kind, seed, post=True, pre=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gate = {0: lambda: None, 1: lambda: r(T), 2: lambda: r(H), 3: lambda: r(T, H).to(dtype)}[kind]()
    return dict(h=(2 * r(T, H)).to(dtype), f=r(T, H).to(dtype), post_w=r(H) * 0.2 + 1 if post else None,
                pre_w=r(H) * 0.2 + 1 if pre else None, gate=gate, go=r(T, H).to(dtype), gn=r(T, H).to(dtype))


def _dev(t):
    return None if t is None else t.cuda()


SHAPES = [(1, 64), (1, 2048), (3, 1), (5, 7), (33, 256), (40, 257), (300, 320), (17, 1000), (64, 2880), (9, 4096),
          (4, 4098), (3, 8192), (2, 8191), (2500, 72),
          # runs of rows long enough for the shared-memory rings, by block size and rows per block
          (20001, 72), (9999, 256), (5000, 512), (1301, 2880), (1203, 4096), (601, 8192),
          # the same with rows that start anywhere
          (3001, 1003), (2401, 2050), (20011, 65), (12345, 130), (333, 8191)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_and_backward_shapes(e4b, T, H, dtype):
    for kind, sig in ((1, True), (3, False)):
        _check(e4b, T, H, dtype, kind, sig, True, True, 0.0, 0.7, seed=T + H + kind)


@pytest.mark.parametrize("kind,sig", [(0, False), (1, False), (1, True), (2, False), (2, True), (3, False), (3, True)])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_gates_and_norms(e4b, kind, sig, post, pre):
    for dtype in (torch.bfloat16, torch.float32):
        _check(e4b, 70, 640, dtype, kind, sig, post, pre, 1.0, -1.3, seed=5 + kind)
        _check(e4b, 1400, 2056, dtype, kind, sig, post, pre, 1.0, -1.3, seed=6 + kind)   # rings


def _check(e4b, T, H, dtype, kind, sig, post, pre, off, scale, seed):
    v = _inputs(T, H, dtype, kind, seed, post, pre)
    eps = 1e-5
    desc = e4b.make_block_desc(H, dtype, eps=eps, weight_offset=off, gate=kind, gate_sigmoid=sig, residual_scale=scale)
    eps, off, scale = desc.eps, desc.weight_offset, desc.residual_scale   # as fp32
    o, n = e4b.e4b_block_norm_forward(desc, _dev(v["h"]), f=_dev(v["f"]), post_w=_dev(v["post_w"]), gate=_dev(v["gate"]),
                                      pre_w=_dev(v["pre_w"]))
    ro, om, rn, nm = _ops.block_forward(v["h"], v["f"], v["post_w"], v["gate"], kind, sig, v["pre_w"], eps, off, scale)
    _ops.assert_near(o.cpu(), ro, om, C_FWD, "o")
    if pre:
        _ops.assert_near(n.cpu(), rn, nm + rn.abs(), C_FWD, "n")
    else:
        assert n is None
    got = e4b.e4b_block_norm_backward(desc, o, f=_dev(v["f"]), post_w=_dev(v["post_w"]), gate=_dev(v["gate"]),
                                      pre_w=_dev(v["pre_w"]), grad_o=_dev(v["go"]), grad_n=_dev(v["gn"]) if pre else None)
    ref = _ops.block_backward(o.cpu(), v["f"], v["post_w"], v["gate"], kind, sig, v["pre_w"], eps, off, scale, v["go"],
                              v["gn"] if pre else None)
    assert {k for k, t in got.items() if t is not None} == set(ref)
    for name, (r, m) in ref.items():
        # sums over the tokens: a term more per token, at most
        c = C_BWD + (T if name in ("grad_post_w", "grad_pre_w") or (name == "grad_gate" and kind == 2) else 0)
        _ops.assert_near(got[name].cpu(), r, m, c, f"{name} kind {kind}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 2048), (50, 257), (9, 8192), (3000, 1024), (12001, 200)])
def test_norm_alone(e4b, T, H, dtype):
    """No branch: n is the norm of h, and its backward with and without the stream's own gradient."""
    v = _inputs(T, H, dtype, 0, 77)
    desc = e4b.make_block_desc(H, dtype, eps=1e-6)
    o, n = e4b.e4b_block_norm_forward(desc, _dev(v["h"]), pre_w=_dev(v["pre_w"]))
    assert o is None
    _, _, rn, nm = _ops.block_forward(v["h"], None, None, None, 0, False, v["pre_w"], desc.eps, 0.0, 1.0)
    _ops.assert_near(n.cpu(), rn, nm, C_FWD, "n")
    for go in (None, v["go"]):
        got = e4b.e4b_block_norm_backward(desc, _dev(v["h"]), pre_w=_dev(v["pre_w"]), grad_o=_dev(go), grad_n=_dev(v["gn"]))
        ref = _ops.block_backward(v["h"], None, None, None, 0, False, v["pre_w"], desc.eps, 0.0, 1.0, go, v["gn"])
        for name, (r, m) in ref.items():
            _ops.assert_near(got[name].cpu(), r, m, C_BWD + (T if name == "grad_pre_w" else 0), name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H", [(1, 8, 2048), (37, 3, 130), (65, 1, 2880), (11, 8, 8192)])
def test_branch_from_grouped_rows(e4b, T, k, H, dtype):
    """The branch as the combine of k rows; pairs without a row add nothing."""
    v = _inputs(T, H, dtype, 1, 13)
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(T * k, H, generator=g).to(dtype)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    if T > 1:
        inv[1] = -1
        inv[2, 0] = T * k
    w = torch.randn(T, k, generator=g)
    desc = e4b.make_block_desc(H, dtype, gate=1, gate_sigmoid=True, residual_scale=0.5)
    f_out = torch.empty(T, H, dtype=dtype, device="cuda")
    o, n = e4b.e4b_block_norm_forward(desc, _dev(v["h"]), rows=rows.cuda(), inv_perm=inv.cuda(), topk_w=w.cuda(),
                                      post_w=_dev(v["post_w"]), gate=_dev(v["gate"]), pre_w=_dev(v["pre_w"]), f_out=f_out)
    f, fm = _ops.combine(rows, inv, w)
    assert torch.equal(f_out, e4b.e4b_moe_combine(rows.cuda(), inv.cuda(), w.cuda()))
    # the row's rms carries the combine's error too: |d rms| <= rms of the magnitudes' error
    fm = fm + f.abs() * (fm.pow(2).mean(1, keepdim=True) / (f.pow(2).mean(1, keepdim=True) + 1e-30)).sqrt()
    ro, om, rn, nm = _ops.block_forward(v["h"], f, v["post_w"], v["gate"], 1, True, v["pre_w"], desc.eps, 0.0, 0.5, fm)
    _ops.assert_near(o.cpu(), ro, om, C_FWD, "o")
    nm = nm + rn.abs() * (om.pow(2).mean(1, keepdim=True) / ro.pow(2).mean(1, keepdim=True)).sqrt()
    _ops.assert_near(n.cpu(), rn, nm, C_FWD, "n")


def test_gradients_against_differences(e4b):
    """fp32: a central difference of the forward along random directions against the backward."""
    T, H = 6, 96
    v = {k: _dev(t) for k, t in _inputs(T, H, torch.float32, 3, 21).items()}
    desc = e4b.make_block_desc(H, torch.float32, gate=3, gate_sigmoid=True, residual_scale=0.9)

    def loss(h, f, post_w, gate, pre_w):
        o, n = e4b.e4b_block_norm_forward(desc, h, f=f, post_w=post_w, gate=gate, pre_w=pre_w)
        return (o.double() * v["go"].double()).sum() + (n.double() * v["gn"].double()).sum()

    at = dict(h=v["h"], f=v["f"], post_w=v["post_w"], gate=v["gate"], pre_w=v["pre_w"])
    o, _ = e4b.e4b_block_norm_forward(desc, **{k: at[k] for k in ("h", "f", "post_w", "gate", "pre_w")})
    got = e4b.e4b_block_norm_backward(desc, o, f=v["f"], post_w=v["post_w"], gate=v["gate"], pre_w=v["pre_w"],
                                      grad_o=v["go"], grad_n=v["gn"])
    step = 1e-2   # truncation ~ step^2; rounding ~ 2^-24 |terms| / step per value, both well under 1e-3 of the scale
    for name, t in at.items():
        d = torch.randn(t.shape, generator=torch.Generator().manual_seed(1)).cuda()
        up = loss(**{**at, name: t + step * d})
        dn = loss(**{**at, name: t - step * d})
        want = ((up - dn) / (2 * step)).item()
        have = (got["grad_" + name].double() * d.double()).sum().item()
        scale = (got["grad_" + name].double() * d.double()).abs().sum().item()
        assert abs(want - have) <= 2e-3 * scale, (name, want, have, scale)


@pytest.mark.parametrize("T,H", [(700, 512), (1500, 2048), (12000, 128)])
def test_in_place_stream_and_repeat(e4b, T, H):
    """o may be h; the same call twice gives the same bits."""
    v = {k: _dev(t) for k, t in _inputs(T, H, torch.bfloat16, 2, 31).items()}
    desc = e4b.make_block_desc(H, gate=2, residual_scale=0.3)
    kw = dict(f=v["f"], post_w=v["post_w"], gate=v["gate"], pre_w=v["pre_w"])
    o, n = e4b.e4b_block_norm_forward(desc, v["h"], **kw)
    h2 = v["h"].clone()
    o2, n2 = e4b.e4b_block_norm_forward(desc, h2, o=h2, **kw)
    assert o2 is h2 and torch.equal(o, o2) and torch.equal(n, n2)
    a = e4b.e4b_block_norm_backward(desc, o, grad_o=v["go"], grad_n=v["gn"], **kw)
    b = e4b.e4b_block_norm_backward(desc, o, grad_o=v["go"], grad_n=v["gn"], **kw)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("T,H", [(300, 384), (2000, 2304), (15000, 64)])
def test_nan_rows_stay_in_their_rows(e4b, T, H):
    v = {k: _dev(t) for k, t in _inputs(T, H, torch.float32, 1, 41).items()}
    desc = e4b.make_block_desc(H, torch.float32, gate=1)
    kw = dict(post_w=v["post_w"], gate=v["gate"], pre_w=v["pre_w"])
    o, n = e4b.e4b_block_norm_forward(desc, v["h"], f=v["f"], **kw)
    f = v["f"].clone()
    f[17] = float("nan")
    o2, n2 = e4b.e4b_block_norm_forward(desc, v["h"], f=f, **kw)
    keep = torch.arange(T, device="cuda") != 17
    assert torch.equal(o[keep], o2[keep]) and torch.equal(n[keep], n2[keep]) and bool(n2[17].isnan().all())


def test_zero_rows(e4b):
    """All-zero rows: the norms give zeros (eps > 0), no NaN anywhere."""
    H = 256
    z = torch.zeros(3, H, device="cuda")
    w = torch.ones(H, device="cuda")
    desc = e4b.make_block_desc(H, torch.float32)
    o, n = e4b.e4b_block_norm_forward(desc, z, f=z, post_w=w, pre_w=w)
    assert not bool(o.any()) and not bool(n.any())
    got = e4b.e4b_block_norm_backward(desc, z, f=z, post_w=w, pre_w=w, grad_o=z, grad_n=z)
    assert all(t is None or not bool(t.any()) for t in got.values())


def test_empty_batch(e4b):
    H = 128
    e = torch.empty(0, H, device="cuda")
    w = torch.ones(H, device="cuda")
    desc = e4b.make_block_desc(H, torch.float32, gate=2)
    o, n = e4b.e4b_block_norm_forward(desc, e, f=e, post_w=w, gate=w, pre_w=w)
    assert o.shape == n.shape == (0, H)
    got = e4b.e4b_block_norm_backward(desc, e, f=e, post_w=w, gate=w, pre_w=w, grad_o=e, grad_n=e)
    for k in ("grad_post_w", "grad_gate", "grad_pre_w"):
        assert not bool(got[k].any())


@pytest.mark.parametrize("T,H", [(129, 2880), (1500, 2880)])
def test_graph_replay(e4b, T, H):
    v = {k: _dev(t) for k, t in _inputs(T, H, torch.bfloat16, 3, 51).items()}
    desc = e4b.make_block_desc(H, gate=3, gate_sigmoid=True)

    def step():
        kw = dict(f=v["f"], post_w=v["post_w"], gate=v["gate"], pre_w=v["pre_w"])
        o, n = e4b.e4b_block_norm_forward(desc, v["h"], **kw)
        return [o, n] + list(e4b.e4b_block_norm_backward(desc, o, grad_o=v["go"], grad_n=v["gn"], **kw).values())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    v["h"].mul_(0.5)
    v["f"].neg_()
    eager = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, out))


@pytest.mark.parametrize("T,H", [(40, 640), (1400, 2056), (1400, 1003)])
@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_backward_outputs_one_at_a_time(e4b, T, H, kind):
    """Every output alone, through the C entry point, has the bits it has with the others; so has
    each without the stream's gradient."""
    v = {k: _dev(t) for k, t in _inputs(T, H, torch.bfloat16, kind, 61).items()}
    desc = e4b.make_block_desc(H, gate=kind, gate_sigmoid=True, residual_scale=0.6)
    kw = dict(f=v["f"], post_w=v["post_w"], gate=v["gate"], pre_w=v["pre_w"])
    o, _ = e4b.e4b_block_norm_forward(desc, v["h"], **kw)
    ws = e4b.block_norm_workspace(desc, T)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    for go in (v["go"], None):
        full = e4b.e4b_block_norm_backward(desc, o, grad_o=go, grad_n=v["gn"], **kw)
        for name in ("grad_h", "grad_f", "grad_post_w", "grad_gate", "grad_pre_w"):
            if full[name] is None:
                continue
            out = torch.full_like(full[name], 3.0)
            p = [out.data_ptr() if name == n else None for n in ("grad_h", "grad_f", "grad_post_w", "grad_gate", "grad_pre_w")]
            st = e4b.lib.e4b_block_norm_backward(desc, ptr(o), ptr(v["f"]), T, ptr(v["post_w"]), ptr(v["gate"]),
                                                 ptr(v["pre_w"]), ptr(go), ptr(v["gn"]), *p, ws.data_ptr(), ws.numel(),
                                                 torch.cuda.current_stream().cuda_stream)
            assert st == 0
            assert torch.equal(out, full[name]), (name, go is None)


def test_views_that_start_off_a_16_byte_boundary(e4b):
    for T, H in ((50, 64), (3000, 256)):
        v = {k: _dev(t) for k, t in _inputs(T, H, torch.bfloat16, 3, 71).items()}
        desc = e4b.make_block_desc(H, gate=3)
        kw = dict(post_w=v["post_w"], pre_w=v["pre_w"])
        o, n = e4b.e4b_block_norm_forward(desc, v["h"], f=v["f"], gate=v["gate"], **kw)

        def off(t):
            buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            buf[1:] = t.flatten()
            return buf[1:].view(t.shape)
        o2, n2 = e4b.e4b_block_norm_forward(desc, off(v["h"]), f=off(v["f"]), gate=off(v["gate"]), o=off(o), n=off(n), **kw)
        assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
        ref = e4b.e4b_block_norm_backward(desc, o, f=v["f"], gate=v["gate"], grad_o=v["go"], grad_n=v["gn"], **kw)
        got = e4b.e4b_block_norm_backward(desc, off(o), f=off(v["f"]), gate=off(v["gate"]), grad_o=off(v["go"]),
                                          grad_n=off(v["gn"]), **kw)
        for k in ref:
            m = ref[k].float().abs().max()
            assert (got[k].float() - ref[k].float()).abs().max() <= 2.0 ** -7 * m, k


ENDS = (20.0, -20.0, 60.0, -60.0, 87.5, -87.5, 100.0, -100.0, 200.0, -200.0)


@pytest.mark.parametrize("kind", [1, 2, 3])
@pytest.mark.parametrize("T,H", [(20, 70), (4000, 256), (1500, 2050)])
def test_sigmoid_gates_at_the_ends_of_the_range(e4b, T, H, kind):
    """fp32, no norms and h = 0, so that o = s g f and the gradients show the gate's own relative
    error; f of 1e10 keeps them normal numbers.  Below 2^-126 a gate is a multiple of 2^-149: the
    exponential (2 units there), its quotient and the product with s add up to 4 units of f.  A
    product that is itself below 2^-126 is rounded to a multiple of 2^-149, half a unit whatever its
    factors: grad_f = g s grad_o passes up to four of them (by s, g and two weights of 1): 2 units."""
    g = torch.Generator().manual_seed(9)
    n = {1: T, 2: H, 3: T * H}[kind]
    gate = torch.tensor(ENDS).repeat(-(-n // len(ENDS)))[:n].view(T, H) if kind == 3 else \
        torch.tensor(ENDS).repeat(-(-n // len(ENDS)))[:n]
    h, f, go = torch.zeros(T, H), 1e10 * torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    desc = e4b.make_block_desc(H, torch.float32, gate=kind, gate_sigmoid=True, residual_scale=0.7)
    s = desc.residual_scale
    kw = dict(f=f.cuda(), gate=gate.cuda())
    o, _ = e4b.e4b_block_norm_forward(desc, h.cuda(), **kw)
    x = gate.double()
    e = torch.exp(-x.abs())
    sg, dg = torch.where(x < 0, e, torch.ones_like(e)) / (1 + e), e / (1 + e).pow(2)
    if kind == 1:
        sg, dg = sg[:, None], dg[:, None]

    def near(got, ref, terms, c, what):
        tol = c * _ops.U24 * ref + 2.0 ** -149 * (4 * terms + 2)
        bad = ~((got.cpu().double().abs() - ref).abs() <= tol)
        assert not bool(bad.any()), (what, int(bad.sum()), got.cpu().flatten()[bad.flatten()][:4], ref.flatten()[bad.flatten()][:4])

    f, go = f.double().abs(), go.double().abs()
    near(o, s * sg * f, s * f + 0 * sg, C_FWD, "o")
    grads = e4b.e4b_block_norm_backward(desc, grad_o=torch.from_numpy(go.float().numpy()).cuda(), f=f.float().cuda(),
                                        gate=kw["gate"])   # positive terms: the sums do not cancel
    near(grads["grad_f"], s * sg * go, s * go + 0 * sg, C_BWD, "grad_f")
    full, terms = s * go * f * dg, s * go * f + 0 * dg
    red = {1: lambda t: t.sum(1), 2: lambda t: t.sum(0), 3: lambda t: t}[kind]
    near(grads["grad_gate"], red(full), red(terms), C_BWD + {1: H, 2: T, 3: 0}[kind], "grad_gate")


@pytest.mark.parametrize("T,H", [(20, 72), (4000, 256)])
def test_bf16_sigmoid_gates_near_one(e4b, T, H):
    """The gradient of a bf16 gate of 8 to 20 keeps its relative error: g (1 - g) without the
    cancellation of 1 - g.  The fast exponential is off by 2 + 1.17 |x| units, 51 half units at 20."""
    g = torch.Generator().manual_seed(10)
    gate = torch.tensor([8.0, 12.0, 16.0, 20.0, -8.0, -20.0, 0.0, 3.0]).repeat(T * H // 8).view(T, H).to(torch.bfloat16)
    f, go = torch.randn(T, H, generator=g).to(torch.bfloat16), torch.randn(T, H, generator=g).to(torch.bfloat16)
    desc = e4b.make_block_desc(H, gate=3, gate_sigmoid=True, residual_scale=0.7)
    got = e4b.e4b_block_norm_backward(desc, grad_o=go.cuda(), f=f.cuda(), gate=gate.cuda())
    ref = _ops.block_backward(None, f, None, gate, 3, True, None, 0.0, 0.0, desc.residual_scale, go, go)
    x = gate.double()
    e = torch.exp(-x.abs())
    dg = desc.residual_scale * go.double() * f.double() * e / (1 + e).pow(2)
    _ops.assert_near(got["grad_gate"].cpu(), dg, dg.abs(), C_BWD, "grad_gate")
    _ops.assert_near(got["grad_f"].cpu(), *ref["grad_f"], C_BWD, "grad_f")


def _off(t, fill=None):
    """A copy of t (or a tensor like it, filled) that starts one element into its memory."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    buf[1:] = t.flatten() if fill is None else fill
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(50, 64), (3000, 256), (1400, 1003)])
@pytest.mark.parametrize("kind", [1, 3])
def test_tensors_off_a_16_byte_boundary_against_the_formulas(e4b, T, H, dtype, kind):
    """Every row tensor one element off, outputs filled with NaN before the call: dense branch,
    combine branch with f_out, and the backward."""
    nan = float("nan")
    v = _inputs(T, H, dtype, kind, 73)
    desc = e4b.make_block_desc(H, dtype, eps=1e-5, gate=kind, gate_sigmoid=True, residual_scale=0.7)
    gate = _off(_dev(v["gate"])) if kind == 3 else _dev(v["gate"])
    kw = dict(post_w=_dev(v["post_w"]), gate=gate, pre_w=_dev(v["pre_w"]))
    h, f = _off(_dev(v["h"])), _off(_dev(v["f"]))
    o, n = e4b.e4b_block_norm_forward(desc, h, f=f, o=_off(h, nan), n=_off(h, nan), **kw)
    args = (v["post_w"], v["gate"], kind, True, v["pre_w"], desc.eps, 0.0, desc.residual_scale)
    ro, om, rn, nm = _ops.block_forward(v["h"], v["f"], *args)
    _ops.assert_near(o.cpu(), ro, om, C_FWD, "o")
    _ops.assert_near(n.cpu(), rn, nm + rn.abs(), C_FWD, "n")

    got = e4b.e4b_block_norm_backward(desc, o, f=f, grad_o=_off(_dev(v["go"])), grad_n=_off(_dev(v["gn"])),
                                      grad_h=_off(h, nan), grad_f=_off(h, nan), **kw)
    ref = _ops.block_backward(o.cpu(), v["f"], *args, v["go"], v["gn"])
    for name, (r, m) in ref.items():
        c = C_BWD + (T if name in ("grad_post_w", "grad_pre_w") else 0)
        _ops.assert_near(got[name].cpu(), r, m, c, name)

    k, g = 3, torch.Generator().manual_seed(5)
    rows = torch.randn(T * k, H, generator=g).to(dtype)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    w = torch.randn(T, k, generator=g)
    f_out = _off(h, nan)
    o, n = e4b.e4b_block_norm_forward(desc, h, rows=_off(rows.cuda()), inv_perm=inv.cuda(), topk_w=w.cuda(),
                                      f_out=f_out, o=_off(h, nan), n=_off(h, nan), **kw)
    f64, fm = _ops.combine(rows, inv, w)
    _ops.assert_near(f_out.cpu(), f64, fm, k, "f_out")
    # the combine's error reaches the row's rms too (as in test_branch_from_grouped_rows)
    fm = fm + f64.abs() * (fm.pow(2).mean(1, keepdim=True) / (f64.pow(2).mean(1, keepdim=True) + 1e-30)).sqrt()
    ro, om, rn, nm = _ops.block_forward(v["h"], f64, *args, fm)
    _ops.assert_near(o.cpu(), ro, om, C_FWD, "o of the combine")
    nm = nm + rn.abs() * (om.pow(2).mean(1, keepdim=True) / ro.pow(2).mean(1, keepdim=True)).sqrt()
    _ops.assert_near(n.cpu(), rn, nm, C_FWD, "n of the combine")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H", [(4096, 8, 256), (3000, 2, 1003), (1200, 5, 2880)])
def test_branch_from_grouped_rows_of_a_prompt(e4b, T, k, H, dtype):
    """As many tokens as keep every block busy for several rows."""
    test_branch_from_grouped_rows(e4b, T, k, H, dtype)
