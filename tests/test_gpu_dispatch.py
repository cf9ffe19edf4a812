"""e4b_moe_dispatch / combine and their gradients against a plain loop in 64 bits: maps exact,
copied rows bit-identical, sums within the roundings they make."""
import pytest
import torch

from tests import _ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def e4b():
    import bit_quantized_mixture_nf4_b200 as m
    m.lib
    return m


def _idx(T, k, E, seed, pad=0, hole=0.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.topk(torch.randn(T, E, generator=g) + torch.randn(E, generator=g), k, dim=1).indices.to(torch.int32)
    if hole:   # pairs without an expert, by both kinds of bad index
        m = torch.rand(T, k, generator=g) < hole
        idx = torch.where(m, torch.where(torch.rand(T, k, generator=g) < 0.5, -1, E).to(torch.int32), idx)
    if pad:
        idx[T - pad:] = -1
    return idx


CASES = [
    # T, k, E, H, dtype, pad, hole      (1024 pairs: the last size of the one-launch form)
    (1, 1, 1, 1, torch.float32, 0, 0.0),
    (1, 8, 8, 2048, torch.bfloat16, 0, 0.0),
    (3, 2, 4, 65, torch.bfloat16, 0, 0.0),
    (7, 6, 256, 100, torch.bfloat16, 2, 0.3),
    (128, 8, 64, 192, torch.bfloat16, 0, 0.0),
    (129, 8, 64, 192, torch.bfloat16, 0, 0.0),
    (256, 8, 64, 192, torch.bfloat16, 0, 0.0),
    (257, 8, 64, 192, torch.bfloat16, 0, 0.0),
    (2048, 1, 8, 33, torch.float32, 0, 0.0),
    (2049, 1, 8, 33, torch.float32, 5, 0.0),
    (1000, 3, 5, 320, torch.float32, 0, 0.2),
    (1500, 7, 256, 130, torch.bfloat16, 100, 0.1),
    (4096, 8, 128, 64, torch.bfloat16, 0, 0.0),
    (5000, 2, 255, 24, torch.bfloat16, 5000, 0.0),      # nothing routed anywhere
    (300, 8, 9, 72, torch.bfloat16, 0, 1.0),
    (9000, 8, 200, 40, torch.bfloat16, 7, 0.1),         # the scan kernel
    (30000, 8, 256, 8, torch.bfloat16, 0, 0.0),
]


@pytest.mark.parametrize("T,k,E,H,dtype,pad,hole", CASES)
def test_dispatch_and_back(e4b, T, k, E, H, dtype, pad, hole):
    idx = _idx(T, k, E, 11 * T + k, pad, hole)
    offs, perm, inv = _ops.sort_pairs(idx, E)
    n = int(offs[-1])
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).to(dtype)
    rows = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    got_perm = torch.full((T * k,), -9, dtype=torch.int32, device="cuda")
    r, o, p, i = e4b.e4b_moe_dispatch(E, idx.cuda(), x.cuda(), rows=rows, perm=got_perm)
    assert torch.equal(o.cpu(), offs) and torch.equal(i.cpu(), inv)
    assert torch.equal(p[:n].cpu(), perm) and bool((p[n:] == -9).all())
    assert torch.equal(r[:n].cpu(), x[perm.long() // k]) and bool((r[n:] == 7).all())
    r2, o2, p2, i2 = e4b.e4b_moe_dispatch(E, idx.cuda())          # the maps alone
    assert r2 is None and torch.equal(o2, o) and torch.equal(i2, i) and torch.equal(p2[:n], p[:n])

    rows = torch.randn(T * k, H, generator=g).to(dtype)
    rows[n:] = float("nan")                                       # rows that no pair has are never read
    w = torch.randn(T, k, generator=g)
    ref, mag = _ops.combine(rows.nan_to_num(), inv, w)
    y = e4b.e4b_moe_combine(rows.cuda(), i, w.cuda())
    _ops.assert_near(y.cpu(), ref, mag, k, "combine")
    ref, mag = _ops.combine(rows.nan_to_num(), inv, None)
    gx = e4b.e4b_moe_dispatch_backward(rows.cuda(), i)
    _ops.assert_near(gx.cpu(), ref, mag, k, "grad_x")

    gy = torch.randn(T, H, generator=g).to(dtype)
    grad_rows = torch.full((T * k, H), 5.0, dtype=dtype, device="cuda")
    gr, gw = e4b.e4b_moe_combine_backward(rows.cuda(), i, w.cuda(), gy.cuda(), grad_rows=grad_rows)
    full = (gy[:, None].double() * w[..., None].double()).reshape(T * k, H)[perm.long()]
    _ops.assert_near(gr[:n].cpu(), full, full.abs(), 1, "grad_rows")
    assert bool((gr[n:] == 5).all())
    prod = torch.zeros(T * k, H, dtype=torch.float64)
    prod[perm.long()] = gy.double()[perm.long() // k] * rows[:n].double()
    _ops.assert_near(gw.cpu(), prod.sum(1).view(T, k), prod.abs().sum(1).view(T, k), H + 2, "grad_w")
    # each alone gives the same bits
    assert torch.equal(e4b.e4b_moe_combine_backward(None, i, w.cuda(), gy.cuda(), want_grad_w=False)[0][:n], gr[:n])
    assert torch.equal(e4b.e4b_moe_combine_backward(rows.cuda(), i, None, gy.cuda(), want_grad_rows=False)[1], gw)
    gr1 = e4b.e4b_moe_combine_backward(None, i, None, gy.cuda(), want_grad_w=False)[0]     # weights 1
    assert torch.equal(gr1[:n].cpu(), gy[perm.long() // k])


def test_same_expert_twice_in_a_token(e4b):
    idx = torch.tensor([[2, 2, 0], [0, 0, 0], [1, 2, 1]], dtype=torch.int32)
    x = torch.arange(3 * 16, dtype=torch.float32).view(3, 16)
    offs, perm, inv = _ops.sort_pairs(idx, 3)
    r, o, p, i = e4b.e4b_moe_dispatch(3, idx.cuda(), x.cuda())
    assert torch.equal(o.cpu(), offs) and torch.equal(p.cpu(), perm) and torch.equal(i.cpu(), inv)
    assert torch.equal(e4b.e4b_moe_dispatch_backward(r, i).cpu(), 3 * x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_rows(e4b, dtype):
    """Tensors that start one element into their memory take narrower vectors."""
    T, k, E, H = 40, 2, 6, 64
    idx = _idx(T, k, E, 3).cuda()
    flat = torch.randn(T * H + 1, device="cuda").to(dtype)
    x = flat[1:].view(T, H)
    r, o, p, i = e4b.e4b_moe_dispatch(E, idx, x)
    assert torch.equal(r, x[p.long() // k])
    y = torch.empty(T * H + 1, dtype=dtype, device="cuda")[1:].view(T, H)
    e4b.e4b_moe_dispatch_backward(r, i, grad_x=y)
    assert torch.equal(y, (2 * x.float()).to(dtype))


def test_infinities_and_nan_stay_in_their_tokens(e4b):
    T, k, E, H = 64, 2, 8, 128
    idx = _idx(T, k, E, 4).cuda()
    x = torch.randn(T, H, device="cuda")
    x[5] = float("inf")
    x[9] = float("nan")
    r, o, p, i = e4b.e4b_moe_dispatch(E, idx, x)
    y = e4b.e4b_moe_combine(r, i, torch.full((T, k), 0.5, device="cuda"))
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[9] = False
    assert torch.equal(y[keep], x[keep]) and bool(y[9].isnan().all())


def test_empty_batch(e4b):
    idx = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    r, o, p, i = e4b.e4b_moe_dispatch(16, idx, torch.empty(0, 64, device="cuda"))
    assert o.tolist() == [0] * 17 and r.shape == (0, 64)
    assert e4b.e4b_moe_combine(r, i).shape == (0, 64)
    gr, gw = e4b.e4b_moe_combine_backward(r, i, None, torch.empty(0, 64, device="cuda"))
    assert gr.shape == (0, 64) and gw.shape == (0, 4)


def test_rows_past_31_bit_offsets(e4b):
    """4.4e9 elements of rows: their offsets need more than 32 bits."""
    T, k, E, H = 134400, 8, 8, 4096
    idx = torch.arange(T * k, device="cuda").remainder(E).to(torch.int32).view(T, k)
    x = torch.arange(T, device="cuda").remainder(251).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    r, o, p, i = e4b.e4b_moe_dispatch(E, idx, x)
    assert r.numel() > 2 ** 32
    assert o.tolist() == [T * e for e in range(E + 1)]
    for e in (0, E - 1):
        assert torch.equal(r[e * T:(e + 1) * T], x)
    gx = e4b.e4b_moe_combine(r, i, torch.full((T, k), 0.125, device="cuda"))
    assert torch.equal(gx, x)


def test_streams_and_graphs(e4b):
    """A call on a side stream, and a captured run replayed on changed inputs, next to an eager one."""
    T, k, E, H = 600, 4, 16, 256
    idx = _idx(T, k, E, 8).cuda()
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    w = torch.rand(T, k, device="cuda")

    def step(stream=None):
        r, o, p, i = e4b.e4b_moe_dispatch(E, idx, x, stream=stream)
        return r, o, e4b.e4b_moe_combine(r, i, w, stream=stream)

    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    idx.copy_(_idx(T, k, E, 9))
    x.neg_()
    eager = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("E", [16, 256])
def test_short_calls_in_the_largest_batchs_workspace(e4b, E):
    """One workspace, sized for 9000 tokens and no larger, for smaller batches of every form."""
    k, H = 8, 16
    ws = torch.full((e4b.e4b_moe_dispatch_workspace_size(E, k, 9000),), 0xFF, dtype=torch.uint8, device="cuda")
    for T in (1, 128, 129, 1000, 1152, 1153, 2000, 4095, 9000):
        idx = _idx(T, k, E, T)
        offs, perm, inv = _ops.sort_pairs(idx, E)
        _, o, p, i = e4b.e4b_moe_dispatch(E, idx.cuda(), ws=ws)
        assert torch.equal(o.cpu(), offs) and torch.equal(p.cpu(), perm) and torch.equal(i.cpu(), inv), T
