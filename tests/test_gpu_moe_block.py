"""A non-gated expert block from the operators, as a program runs them: pre-norm, router, dispatch,
two grouped linears, combine with gate, post-norm and scaled residual, next pre-norm; its
gradients; one decode token; and the whole step captured in a graph.  The reference is the same
block in 64 bits under autograd, on the weights' stored values."""
import pytest
import torch

from tests.test_gpu_linear import _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def e4b():
    import bit_quantized_mixture_nf4_b200 as m
    m.lib
    return m


class Block:
    """E experts H -> I -> H with SiLU between, biases, post- and pre-norms and a sigmoid token gate."""

    def __init__(self, e4b, T, k, E, H, I, seed, pad=0):
        self.e4b, self.T, self.k, self.E, self.H, self.I = e4b, T, k, E, H, I
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.w1, self.v1, self.b1 = _weights(e4b, E, I, H, "nf4", True, seed)
        self.w2, self.v2, self.b2 = _weights(e4b, E, H, I, "nf4", True, seed + 1)
        self.d1 = e4b.make_linear_desc(H, I, E=E, activation=e4b.LINEAR_ACT_SILU)
        self.d2 = e4b.make_linear_desc(I, H, E=E)
        self.pre = e4b.make_block_desc(H)
        self.post = e4b.make_block_desc(H, gate=e4b.GATE_TOKEN, gate_sigmoid=True, residual_scale=0.8)
        self.h = (r(T, H) * 1.5).to(torch.bfloat16)
        self.idx = torch.topk(r(T, E), k, dim=1).indices.to(torch.int32)
        if pad:
            self.idx[T - pad:] = -1
        self.w = torch.softmax(r(T, k), dim=1)
        self.gate = r(T)
        self.n1, self.n2, self.n3 = (1 + 0.1 * r(H) for _ in range(3))
        self.go, self.gn = r(T, H).to(torch.bfloat16), r(T, H).to(torch.bfloat16)
        for n in ("h", "idx", "w", "gate", "n1", "n2", "n3", "go", "gn"):
            setattr(self, "c_" + n, getattr(self, n).cuda())

    def forward(self, save=True, fused=False):
        e, c = self.e4b, lambda n: getattr(self, "c_" + n)  # noqa: E731
        _, x = e.e4b_block_norm_forward(self.pre, c("h"), pre_w=c("n1"))
        rows, offs, perm, inv = e.e4b_moe_dispatch(self.E, c("idx"), x)
        P = rows.shape[0]
        saved = torch.empty(P, self.I, dtype=torch.bfloat16, device="cuda") if save else None
        u = e.e4b_linear_forward(self.d1, self.w1, rows, offsets=offs, saved_d=saved)
        y = e.e4b_linear_forward(self.d2, self.w2, u, offsets=offs)
        kw = dict(post_w=c("n2"), gate=c("gate"), pre_w=c("n3"))
        if fused:
            o, n = e.e4b_block_norm_forward(self.post, c("h"), rows=y, inv_perm=inv, topk_w=c("w"), **kw)
            return o, n
        f = e.e4b_moe_combine(y, inv, c("w"))
        o, n = e.e4b_block_norm_forward(self.post, c("h"), f=f, **kw)
        self.kept = (rows, offs, inv, saved, y, f, o)
        return o, n

    def backward(self):
        e, c = self.e4b, lambda n: getattr(self, "c_" + n)  # noqa: E731
        rows, offs, inv, saved, y, f, o = self.kept
        g = e.e4b_block_norm_backward(self.post, o, f=f, post_w=c("n2"), gate=c("gate"), pre_w=c("n3"), grad_o=c("go"),
                                      grad_n=c("gn"))
        gy, gw = e.e4b_moe_combine_backward(y, inv, c("w"), g["grad_f"])
        gu, gb2 = e.e4b_linear_backward(self.d2, self.w2, gy, offsets=offs)
        gr, gb1 = e.e4b_linear_backward(self.d1, self.w1, gu, offsets=offs, saved_d=saved)
        gx = e.e4b_moe_dispatch_backward(gr, inv)
        first = e.e4b_block_norm_backward(self.pre, c("h"), pre_w=c("n1"), grad_o=g["grad_h"], grad_n=gx)
        return {"h": first["grad_h"], "w": gw, "gate": g["grad_gate"], "n1": first["grad_pre_w"],
                "n2": g["grad_post_w"], "n3": g["grad_pre_w"], "b1": gb1, "b2": gb2}

    def reference(self):
        f64 = lambda t: t.double().requires_grad_()  # noqa: E731
        v = {n: f64(getattr(self, n)) for n in ("h", "w", "gate", "n1", "n2", "n3")}
        v["b1"], v["b2"] = f64(self.b1), f64(self.b2)
        rms = lambda t, w, eps: t / torch.sqrt(t.pow(2).mean(1, keepdim=True) + eps) * w  # noqa: E731
        x = rms(v["h"], v["n1"], self.pre.eps)
        f = torch.zeros(self.T, self.H, dtype=torch.float64)
        for j in range(self.k):
            for e in range(self.E):
                t = (self.idx[:, j] == e).nonzero()[:, 0]
                if len(t):
                    u = torch.nn.functional.silu(x[t] @ self.v1[e].t() + v["b1"][e])
                    y = u @ self.v2[e].t() + v["b2"][e]
                    f = f.index_add(0, t, v["w"][t, j][:, None] * y)
        b = rms(f, v["n2"], self.post.eps) * torch.sigmoid(v["gate"])[:, None]
        o = v["h"] + self.post.residual_scale * b
        n = rms(o, v["n3"], self.post.eps)
        ((o * self.go.double()).sum() + (n * self.gn.double()).sum()).backward()
        return o.detach(), n.detach(), {k: t.grad for k, t in v.items()}


def _rel(got, ref):
    return ((got.cpu().double() - ref).norm() / ref.norm().clamp_min(1e-30)).item()


# The chain rounds to bf16 at seven places in the forward and eight more in the backward (u = 2^-8
# each), and a row's relative error grows at most by the norms' and products' conditioning, a small
# factor for these random inputs; 2-norms average it.  15 u = 0.06 bounds the sum of the roundings.
TOL = 15 * 2.0 ** -8


@pytest.mark.parametrize("T,k,E,H,I,pad", [(40, 2, 4, 128, 192, 0), (600, 4, 16, 256, 128, 50), (3, 2, 8, 320, 64, 1)])
def test_block_and_its_gradients(e4b, T, k, E, H, I, pad):
    b = Block(e4b, T, k, E, H, I, 100 + T, pad)
    if pad:   # a token without experts: the branch is zero there, its norm too
        pass
    o, n = b.forward()
    ro, rn, rg = b.reference()
    assert _rel(o, ro) < TOL and _rel(n, rn) < TOL
    got = b.backward()
    for name, g in got.items():
        assert _rel(g, rg[name]) < 2 * TOL, name
    assert e4b.e4b_device_status() == 0
    fo, fn = b.forward(save=False, fused=True)   # serving: the combine inside the block kernel
    assert _rel(fo, ro) < TOL and _rel(fn, rn) < TOL


def test_one_token_and_the_batch_agree(e4b):
    """The single-token form (streamed weights) against the same token in a batch."""
    b = Block(e4b, 300, 2, 4, 256, 192, 7)
    o, n = b.forward(save=False, fused=True)
    for t in (0, 299):
        one = Block(e4b, 300, 2, 4, 256, 192, 7)
        for name in ("h", "idx", "w", "gate"):
            setattr(one, "c_" + name, getattr(b, "c_" + name)[t:t + 1].contiguous())
        o1, n1 = one.forward(save=False, fused=True)
        assert _rel(o1, o[t:t + 1].cpu().double()) < TOL and _rel(n1, n[t:t + 1].cpu().double()) < TOL


def test_training_step_in_a_graph(e4b):
    """Forward and backward captured together, replayed on new inputs, next to eager runs."""
    b = Block(e4b, 500, 2, 8, 128, 128, 9)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = list(b.forward()) + list(b.backward().values())
    b.c_h.neg_()
    b.c_idx.copy_(torch.topk(torch.randn(500, 8), 2, dim=1).indices.to(torch.int32))
    eager = list(b.forward()) + list(b.backward().values())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(eager, outs))


def test_two_streams_at_once(e4b):
    """Two blocks on two streams give what they give one after the other."""
    a, b = Block(e4b, 700, 4, 8, 256, 128, 21), Block(e4b, 400, 2, 16, 128, 192, 22)
    want = [list(x.forward()) + list(x.backward().values()) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = list(x.forward()) + list(x.backward().values())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))


@pytest.mark.parametrize("T,k,E,H,I,pad", [(40, 2, 4, 128, 192, 0), (600, 4, 16, 256, 128, 50)])
def test_every_row_of_the_block(e4b, T, k, E, H, I, pad):
    """Row by row: a rounding is off by at most 2^-8 of each element, so TOL's 15 roundings bound every
    row's 2-norm as they bound the batch's.  The gradient passes a row's two norms, whose conditioning
    varies from row to row: twice the batch's bound.  (A row of another token is off by about 1.)"""
    b = Block(e4b, T, k, E, H, I, 100 + T, pad)
    o, n = b.forward()
    ro, rn, rg = b.reference()
    rows = lambda got, ref: ((got.cpu().double() - ref).norm(dim=1) / ref.norm(dim=1).clamp_min(1e-30)).max().item()  # noqa: E731
    assert rows(o, ro) < TOL and rows(n, rn) < TOL
    assert rows(b.backward()["h"], rg["h"]) < 4 * TOL
    fo, fn = b.forward(save=False, fused=True)
    assert rows(fo, ro) < TOL and rows(fn, rn) < TOL
