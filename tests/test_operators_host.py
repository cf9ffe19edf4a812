"""Argument checks of the operators around the expert layer: every call here is refused (or a
no-op) on the host, before any launch, so no GPU is needed."""
import ctypes

import pytest
import torch

from bit_quantized_mixture_nf4_b200 import build as e4b_build

OK, INVALID, BLOCK, UNSUP, WS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def e4b():
    e4b_build.build()
    import bit_quantized_mixture_nf4_b200 as m
    return m


def test_dispatch_refusals(e4b):
    L = e4b.lib

    def f(E=4, k=2, idx=16, x=16, dt=1, T=8, H=64, rows=16, offs=16, perm=16, inv=16, ws=None, n=0):
        return L.e4b_moe_dispatch(E, k, idx, x, dt, T, H, rows, offs, perm, inv, ws, n, None)
    for kw in (dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(idx=None), dict(dt=2), dict(dt=-1), dict(T=-1),
               dict(H=0), dict(offs=None), dict(perm=None), dict(inv=None), dict(x=None), dict(rows=None),
               dict(T=2 ** 31), dict(x=17, H=63), dict(dt=0, rows=18, x=16)):
        assert f(**kw) == INVALID, kw
    assert f(T=2048) == WS and f(T=2048, ws=16, n=3) == WS     # above one launch a workspace is needed
    assert e4b.e4b_moe_dispatch_workspace_size(4, 2, 512) == 0
    assert e4b.e4b_moe_dispatch_workspace_size(4, 2, 513) > 0
    for bad in ((0, 2, 8), (257, 2, 8), (4, 0, 8), (4, 9, 8), (4, 2, -1), (4, 8, 2 ** 30)):
        assert e4b.e4b_moe_dispatch_workspace_size(*bad) == 0


def test_combine_refusals(e4b):
    L = e4b.lib

    def c(rows=16, inv=16, w=16, dt=1, T=8, H=64, k=2, y=16):
        return L.e4b_moe_combine(rows, inv, w, dt, T, H, k, y, None)
    for kw in (dict(rows=None), dict(inv=None), dict(y=None), dict(dt=3), dict(T=-1), dict(H=0), dict(k=0), dict(k=9),
               dict(rows=17), dict(dt=0, y=18)):
        assert c(**kw) == INVALID, kw
    assert c(T=0, rows=None, y=None, inv=None) == OK
    assert L.e4b_moe_dispatch_backward(None, 16, 1, 8, 64, 2, 16, None) == INVALID
    assert L.e4b_moe_dispatch_backward(None, None, 1, 0, 64, 2, None, None) == OK

    def b(rows=16, inv=16, w=16, gy=16, dt=1, T=8, H=64, k=2, gr=16, gw=16):
        return L.e4b_moe_combine_backward(rows, inv, w, gy, dt, T, H, k, gr, gw, None)
    for kw in (dict(rows=None), dict(inv=None), dict(gy=None), dict(gr=None, gw=None), dict(k=9), dict(gy=17)):
        assert b(**kw) == INVALID, kw
    assert b(T=0, gy=None) == OK


def test_block_norm_refusals(e4b):
    L = e4b.lib

    def branch(**kw):
        return e4b.e4b_block_branch(*[kw.get(k) for k in ("f", "rows", "inv_perm", "topk_w")], kw.get("top_k", 0))

    def f(d=None, br=branch(f=16), h=16, T=4, post=16, gate=None, pre=16, f_out=None, o=16, n=16):
        d = e4b.make_block_desc(64) if d is None else d
        return L.e4b_block_norm_forward(d, br, h, T, post, gate, pre, f_out, o, n, None)
    D = e4b.make_block_desc
    for kw in (dict(T=-1), dict(h=None), dict(n=None), dict(o=None), dict(pre=None), dict(gate=16), dict(f_out=16),
               dict(d=D(0)), dict(d=D(64, eps=-1.0)), dict(d=D(64, eps=float("nan"))), dict(d=D(64, gate=4)),
               dict(d=D(64, gate=-1)), dict(d=D(64, gate=1)), dict(d=D(64, residual_scale=float("inf"))),
               dict(d=D(64, weight_offset=float("nan"))), dict(br=branch(f=16, rows=16, inv_perm=16, top_k=2)),
               dict(br=branch(rows=16, inv_perm=16, top_k=9)), dict(br=branch(rows=16, inv_perm=16, top_k=0)),
               dict(br=branch(rows=16, top_k=2)), dict(br=branch()),           # no branch: no o, no post_w
               dict(br=branch(), o=None), dict(br=branch(), o=None, post=None, pre=None, n=None),
               dict(h=17, d=D(63))):
        assert f(**kw) == INVALID, kw
    assert f(d=D(8193)) == UNSUP
    bad = e4b.e4b_block_desc(64, 5, 1e-6, 0.0, 0, 0, 1.0)
    assert f(d=bad) == INVALID
    assert L.e4b_block_norm_forward(None, None, 16, 4, None, None, 16, None, None, 16, None) == INVALID
    assert f(T=0) == OK

    def b(d=None, o=16, fb=16, T=4, post=16, gate=None, pre=16, go=16, gn=16, gh=16, gf=16, gpost=16, gg=None, gpre=16,
          ws=None, n=0):
        d = D(64) if d is None else d
        return L.e4b_block_norm_backward(d, o, fb, T, post, gate, pre, go, gn, gh, gf, gpost, gg, gpre, ws, n, None)
    for kw in (dict(o=None), dict(gn=None), dict(pre=None), dict(pre=None, gn=None), dict(post=None), dict(gg=16),
               dict(fb=None), dict(gh=None, gf=None, gpost=None, gpre=None),
               dict(pre=None, gn=None, gpre=None, go=None), dict(d=D(64, gate=2)),
               dict(ws=16, n=1 << 30, gf=17, d=D(63))):
        assert b(**kw) == INVALID, kw
    assert b() == WS and b(ws=16, n=8) == WS
    assert e4b.e4b_block_norm_workspace_size(D(64), 4) > 0
    assert e4b.e4b_block_norm_workspace_size(D(8193), 4) == 0
    assert b(T=0, gpost=None, gpre=None) == OK


def test_linear_refusals(e4b):
    L = e4b.lib
    D, Wt = e4b.make_linear_desc, e4b.e4b_linear_weights

    def f(d=None, w=Wt(16, 16, None, None), x=16, P=4, offs=None, res=None, y=16, saved=None, ws=256, n=1 << 40):
        return L.e4b_linear_forward(D(128, 64) if d is None else d, w, x, P, offs, res, y, saved, ws, n, None)
    for kw in (dict(x=None), dict(y=None), dict(P=-1), dict(P=2 ** 31 - 1), dict(d=D(128, 64, E=2)), dict(d=D(128, 64, E=0)),
               dict(d=D(128, 64, E=257)), dict(d=D(0, 64)), dict(d=D(128, 0)), dict(d=D(128, 64, activation=4)),
               dict(d=D(128, 64, activation=-1)), dict(d=D(128, 64, codebook=6)), dict(w=Wt(None, 16, None, None)),
               dict(w=Wt(16, None, 16, None)), dict(w=Wt(16, 16, None, None), d=D(128, 64, codebook=e4b.MXFP4)),
               dict(x=18), dict(res=24), dict(w=Wt(16, 16, None, 20)), dict(ws=264)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(d=D(96, 64)), dict(d=D(128, 32)), dict(d=D(128, 64, blocksize=32)),
               dict(d=D(128, 64, codebook=e4b.MXFP4, blocksize=64))):
        assert f(**kw) == BLOCK, kw
    assert f(d=D(2 ** 24, 64, E=256)) == UNSUP
    assert f(ws=None) == WS and f(n=1) == WS
    assert f(P=0, x=None, y=None) == OK
    need = e4b.e4b_linear_workspace_size
    assert need(D(128, 64), 4) > 0 and need(D(96, 64), 4) == 0 and need(D(128, 64), -1) == 0
    assert need(D(128, 64, codebook=e4b.INT8), 4) >= need(D(128, 64, codebook=e4b.BF16_WEIGHTS), 4) + 128 * 64 * 2

    def b(d=None, x=None, P=4, offs=None, gy=16, saved=None, gx=16, gb=16, ws=256, n=1 << 40):
        w = Wt(16, 16, None, None)
        return L.e4b_linear_backward(D(128, 64) if d is None else d, w, x, P, offs, gy, saved, gx, gb, ws, n, None)
    for kw in (dict(gy=None), dict(gx=None, gb=None), dict(d=D(128, 64, activation=2)), dict(d=D(128, 64, E=3)),
               dict(gy=18), dict(P=-1)):
        assert b(**kw) == INVALID, kw
    assert b(ws=None) == WS
    assert b(P=0, gb=None) == OK


def test_wrapper_checks(e4b):
    """The Python layer refuses host tensors, wrong types, shapes and strides."""
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        e4b.e4b_moe_dispatch(4, idx)
    with pytest.raises(ValueError):
        e4b.e4b_moe_combine(torch.zeros(8, 16), idx)
    with pytest.raises(ValueError):
        e4b.e4b_block_norm_forward(e4b.make_block_desc(16, torch.float32), torch.zeros(4, 16))
    with pytest.raises(ValueError):
        e4b.make_block_desc(16, torch.float16)
    with pytest.raises(ValueError):
        e4b.make_linear_weights(torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        e4b.e4b_linear_forward(e4b.make_linear_desc(64, 64), None, torch.zeros(4, 64))
    assert ctypes.sizeof(e4b.e4b_linear_desc) == 24 and ctypes.sizeof(e4b.e4b_block_desc) == 28


def test_misaligned_arrays_are_refused(e4b):
    """Index, weight and gradient arrays off their element's boundary, workspaces off 16 bytes."""
    L, n = e4b.lib, 1 << 40
    for idx, offs, perm, inv, ws in ((18, 16, 16, 16, 16), (16, 18, 16, 16, 16), (16, 16, 18, 16, 16),
                                     (16, 16, 16, 18, 16), (16, 16, 16, 16, 17), (16, 16, 16, 16, 20)):
        assert L.e4b_moe_dispatch(4, 2, idx, 16, 1, 2048, 64, 16, offs, perm, inv, ws, n, None) == INVALID
    for inv, w in ((18, 16), (16, 18)):
        assert L.e4b_moe_combine(16, inv, w, 1, 8, 64, 2, 16, None) == INVALID
        assert L.e4b_moe_combine_backward(16, inv, w, 16, 1, 8, 64, 2, 16, 16, None) == INVALID
    assert L.e4b_moe_dispatch_backward(16, 18, 1, 8, 64, 2, 16, None) == INVALID
    assert L.e4b_moe_combine_backward(16, 16, 16, 16, 1, 8, 64, 2, 16, 18, None) == INVALID

    D = e4b.make_block_desc
    dense = e4b.e4b_block_branch(16)
    for d, post, gate, pre in ((D(64), 18, None, 16), (D(64), 16, None, 18), (D(64, gate=1), 16, 18, 16),
                               (D(64, gate=2), 16, 18, 16)):
        assert L.e4b_block_norm_forward(d, dense, 16, 4, post, gate, pre, None, 16, 16, None) == INVALID
    for inv, w in ((18, 16), (16, 18)):
        br = e4b.e4b_block_branch(None, 16, inv, w, 2)
        assert L.e4b_block_norm_forward(D(64), br, 16, 4, 16, None, 16, None, 16, 16, None) == INVALID
    for gate, gg, gpost, gpre, ws in ((16, 16, 16, 16, 17), (16, 16, 16, 16, 20), (16, 16, 18, 16, 16),
                                      (16, 16, 16, 18, 16), (16, 18, 16, 16, 16), (18, 16, 16, 16, 16)):
        assert L.e4b_block_norm_backward(D(64, gate=2), 16, 16, 4, 16, gate, 16, 16, 16, 16, 16, gpost, gg, gpre, ws, n,
                                         None) == INVALID

    d, w = e4b.make_linear_desc(128, 64, E=2), e4b.e4b_linear_weights(16, 16, None, None)
    assert L.e4b_linear_forward(d, w, 16, 4, 18, None, 16, None, 256, n, None) == INVALID
    for offs, gb in ((18, 16), (16, 18)):
        assert L.e4b_linear_backward(d, w, None, 4, offs, 16, None, 16, gb, 256, n, None) == INVALID


def test_block_norm_refuses_a_combine_without_rows(e4b):
    d, t = e4b.make_block_desc(16), torch.zeros(4, 16, dtype=torch.bfloat16)
    for kw in (dict(inv_perm=torch.zeros(4, 2, dtype=torch.int32)), dict(topk_w=torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="need rows"):
            e4b.e4b_block_norm_forward(d, t, f=t, **kw)


def test_allocations_for_a_stream_come_from_that_stream(e4b, monkeypatch):
    """With an explicit stream a wrapper's own tensors are allocated while that stream is the current
    one, and marked as used by the stream that was."""
    import ast
    import contextlib
    import inspect
    from types import SimpleNamespace
    seen, current = [], ["main"]

    @contextlib.contextmanager
    def stream(s):
        kept, current[0] = current[0], s
        yield
        current[0] = kept

    def empty(shape, dtype=None, device=None):
        seen.append(("empty", current[0]))
        return SimpleNamespace(numel=lambda: 4, record_stream=lambda s: seen.append(("used by", s)))

    cuda = SimpleNamespace(stream=stream, current_stream=lambda device=None: current[0])
    monkeypatch.setattr(e4b, "torch", SimpleNamespace(empty=empty, cuda=cuda))
    e4b._new((4,), None, 0, "side")
    assert seen == [("empty", "side"), ("used by", "main")]
    seen.clear()
    e4b._new((4,), None, 0, None)
    assert seen == [("empty", "main")]
    # and no function that takes a stream allocates in another way
    for f in ast.walk(ast.parse(inspect.getsource(e4b))):
        if isinstance(f, ast.FunctionDef) and f.name != "_new" and "stream" in [a.arg for a in f.args.args]:
            calls = [c.func for c in ast.walk(f) if isinstance(c, ast.Call)]
            assert not [c for c in calls if isinstance(c, ast.Attribute) and c.attr == "empty"], f.name


@pytest.mark.parametrize("T", [2 ** 31, 2 ** 60, 2 ** 61, 2 ** 62, 2 ** 63 - 1])
def test_token_counts_whose_pairs_pass_64_bits_are_refused(e4b, T):
    """T * k may be 0 or negative in 64 bits; the counts are refused before anything is launched."""
    L, k = e4b.lib, 8
    assert L.e4b_moe_dispatch(4, k, 16, None, 1, T, 64, None, 16, 16, 16, 16, 1 << 40, None) == INVALID
    assert L.e4b_moe_dispatch_backward(16, 16, 1, T, 64, k, 16, None) == INVALID
    assert L.e4b_moe_combine(16, 16, None, 1, T, 64, k, 16, None) == INVALID
    assert L.e4b_moe_combine_backward(16, 16, None, 16, 1, T, 64, k, 16, None, None) == INVALID
    branch = e4b.e4b_block_branch(None, 16, 16, None, k)
    assert L.e4b_block_norm_forward(e4b.make_block_desc(64), branch, 16, T, None, None, 16, None, 16, 16, None) == INVALID
    assert e4b.e4b_moe_dispatch_workspace_size(4, k, T) == 0
    if T > 2 ** 59:   # bytes of a row tensor
        assert e4b.e4b_moe_workspace_size(e4b.make_desc(8, 256, 192, k), T) == 0
        d, dense = e4b.make_block_desc(64), e4b.e4b_block_branch(16)
        assert L.e4b_block_norm_forward(d, dense, 16, T, None, None, 16, None, 16, 16, None) == INVALID
        assert L.e4b_block_norm_backward(d, 16, 16, T, None, None, 16, 16, 16, 16, 16, None, None, None, None, 0,
                                         None) == INVALID
        moe, one = e4b.make_desc(8, 256, 192, k), ctypes.c_void_p(256)
        experts = e4b.e4b_experts(256, 256, 256, 256)
        assert L.e4b_moe_forward(ctypes.byref(moe), ctypes.byref(experts), one, T, None, one, one, one, None, None, None,
                                 None, one, 1 << 62, None) == INVALID


def test_workspace_sizes_cover_every_smaller_call(e4b):
    """A workspace for the largest batch serves every smaller one: sizes never fall with the rows."""
    counts = sorted({*range(0, 1400), *(round(1.03 ** i) for i in range(240, 420)), *(128 * i + d for i in range(1, 90) for d in (-1, 0, 1))})
    for E in (1, 4, 64, 200, 256):
        for k in (1, 2, 3, 7, 8):
            sizes = [e4b.e4b_moe_dispatch_workspace_size(E, k, T) for T in counts]
            assert sizes == sorted(sizes), (E, k)
    for E, i, o in ((1, 2880, 2880), (1, 4096, 256), (1, 64, 64), (1, 256, 14336), (1, 14336, 64), (8, 2048, 1024)):
        for cb, act in ((e4b.NF4, 0), (e4b.INT8, 2)):
            d = e4b.make_linear_desc(i, o, E=E, codebook=cb, activation=act)
            sizes = [e4b.e4b_linear_workspace_size(d, P) for P in counts]
            assert sizes == sorted(sizes), (E, i, o, cb)
    for H in (1, 64, 256, 2880, 8192):
        sizes = [e4b.e4b_block_norm_workspace_size(e4b.make_block_desc(H), T) for T in counts]
        assert sizes == sorted(sizes), H


def test_layer_workspace_sizes_cover_every_smaller_call(e4b):
    """Also from the grouped form down to the decode form of up to 8 tokens."""
    for E, H, I, k in ((8, 4096, 14336, 2), (64, 2048, 1024, 8), (128, 2048, 768, 8)):
        for rank in (0, 16):
            d = e4b.make_desc(E, H, I, k, lora_rank=rank)
            sizes = [e4b.e4b_moe_workspace_size(d, T) for T in range(3000)]
            assert sizes == sorted(sizes), (E, rank)


def test_a_linear_forward_asks_for_no_backward_workspace(e4b):
    """Neither the size for the forward alone nor what a forward requires holds dz or a derivative."""
    need, forward = e4b.e4b_linear_workspace_size, e4b.e4b_linear_forward_workspace_size
    d = e4b.make_linear_desc(4096, 14336, activation=e4b.LINEAR_ACT_SILU)
    assert need(d, 16384) >= 2 * 16384 * 14336 * 2 and forward(d, 16384) < 1 << 16
    eight = e4b.make_linear_desc(128, 64, codebook=e4b.INT8, activation=2)   # the dequantized stack stays
    assert 128 * 64 * 2 <= forward(eight, 4) <= need(eight, 4)
    for E, i, o in ((1, 2880, 2880), (1, 256, 14336), (1, 14336, 64), (8, 2048, 1024)):
        d = e4b.make_linear_desc(i, o, E=E, activation=3)
        sizes = [forward(d, P) for P in range(0, 3000, 7)]
        assert sizes == sorted(sizes) and all(f <= need(d, P) for f, P in zip(sizes, range(0, 3000, 7)))
    assert forward(e4b.make_linear_desc(96, 64), 4) == 0 and forward(e4b.make_linear_desc(64, 64), -1) == 0
