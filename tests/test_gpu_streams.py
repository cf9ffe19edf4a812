"""Calls on a stream that is not the current one: what a wrapper allocates (outputs, maps,
workspaces) may not be memory that work queued on the current stream still uses."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def e4b():
    import bit_quantized_mixture_nf4_b200 as m
    m.lib
    return m


T, K, E, H, I = 1500, 2, 8, 256, 192


def _calls(e4b):
    """{name: call(stream)} with all outputs and workspaces left to the wrappers."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    bf = torch.bfloat16
    idx = torch.topk(torch.randn(T, E, generator=g), K, dim=1).indices.to(torch.int32).cuda()
    x, logits, w = r(T, H).to(bf), r(T, E), torch.softmax(r(T, K), 1).contiguous()
    rows, offs, perm, inv = e4b.e4b_moe_dispatch(E, idx, x)
    wg, wd = r(E, 2 * I, H) * 0.05, r(E, H, I) * 0.05
    pg, ag = e4b.e4b_quantize_nf4(wg)
    pd, ad = e4b.e4b_quantize_nf4(wd)
    p4, s4 = e4b.e4b_quantize_mxfp4(wg)
    experts, moe = e4b.make_experts(pg, pd, ag, ad), e4b.make_desc(E, H, I, K)
    bias = r(E, H)
    lin, wl = e4b.make_linear_desc(I, H, E=E, activation=e4b.LINEAR_ACT_SILU), e4b.make_linear_weights(pd, ad, bias)
    u, gy, saved = r(T * K, I).to(bf), r(T * K, H).to(bf), r(T * K, H).to(bf)
    block = e4b.make_block_desc(H, gate=e4b.GATE_TOKEN, gate_sigmoid=True)
    n1, n2, gate, f = 1 + 0.1 * r(H), 1 + 0.1 * r(H), r(T), r(T, H).to(bf)
    kw = dict(f=f, post_w=n1, gate=gate, pre_w=n2)
    _, ti, tw = e4b.e4b_moe_forward(moe, experts, x, logits)
    keep = dict(locals())
    flat = lambda v: [t for t in v.values() if t is not None]  # noqa: E731
    return keep, {
        "dispatch": lambda s: e4b.e4b_moe_dispatch(E, idx, x, stream=s),
        "dispatch_backward": lambda s: [e4b.e4b_moe_dispatch_backward(rows, inv, stream=s)],
        "combine": lambda s: [e4b.e4b_moe_combine(rows, inv, w, stream=s)],
        "combine_backward": lambda s: e4b.e4b_moe_combine_backward(rows, inv, w, x, stream=s),
        "block_forward": lambda s: e4b.e4b_block_norm_forward(block, x, stream=s, **kw),
        "block_backward": lambda s: flat(e4b.e4b_block_norm_backward(block, x, grad_o=f, grad_n=x, stream=s, **kw)),
        "linear": lambda s: [e4b.e4b_linear_forward(lin, wl, u, offsets=offs, stream=s)],
        "linear_backward": lambda s: e4b.e4b_linear_backward(lin, wl, gy, offsets=offs, saved_d=saved, stream=s),
        "quantize": lambda s: e4b.e4b_quantize_nf4(wg, stream=s),
        "dequantize": lambda s: [e4b.e4b_dequantize_nf4(pg, ag, wg.shape, stream=s)],
        "quantize_mxfp4": lambda s: e4b.e4b_quantize_mxfp4(wg, stream=s),
        "dequantize_mxfp4": lambda s: [e4b.e4b_dequantize_mxfp4(p4, s4, wg.shape, stream=s)],
        "moe_forward": lambda s: e4b.e4b_moe_forward(moe, experts, x, logits, stream=s),
        "moe_forward_noalloc": lambda s: e4b.e4b_moe_forward_noalloc(moe, experts, x, logits, stream=s),
        "moe_backward": lambda s: [t for t in e4b.e4b_moe_backward(moe, experts, x, ti, tw, f, router_logits=logits,
                                                                   stream=s)],
        "moe_backward_dgrad": lambda s: [e4b.e4b_moe_backward_dgrad(moe, experts, x, ti, tw, f, stream=s)],
        "moe_backward_router": lambda s: e4b.e4b_moe_backward_router(moe, experts, x, ti, tw, f, router_logits=logits,
                                                                     stream=s),
    }


def test_a_dropped_temporary_of_the_current_stream_is_not_the_output(e4b):
    """The current stream spins, then overwrites temporaries as large as the call's outputs and its
    workspace; they are dropped at once, and the call runs on a stream that waits for none of it."""
    keep, calls = _calls(e4b)
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        dropped = set()
        for _ in range(3):
            side.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(20_000_000)   # about 10 ms
            temps = [torch.empty_like(t) for t in want] + [torch.empty(1 << 20, dtype=torch.uint8, device="cuda")]
            for t in temps:
                t.fill_(7)
            dropped.update(t.data_ptr() for t in temps)
            del temps, t
            got = call(side)
            assert not dropped & {t.data_ptr() for t in got}, name
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            for a, b in zip(want, got):
                assert torch.equal(a, b), name
    assert e4b.e4b_device_status() == 0


def test_outputs_may_be_used_and_dropped_on_the_current_stream(e4b):
    """After waiting for the call's stream, work on the current stream reads the output, which is then
    dropped and its size asked for again on the call's stream."""
    keep, calls = _calls(e4b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for name in ("combine", "linear", "moe_forward"):
        want = calls[name](None)[0].float().sum()
        torch.cuda.synchronize()
        got = calls[name](side)[0]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(20_000_000)
        total = got.float().sum()
        size = got.shape
        del got
        with torch.cuda.stream(side):
            torch.empty(size, dtype=torch.bfloat16, device="cuda").fill_(9)
        torch.cuda.synchronize()
        assert torch.equal(total, want), name


def test_calls_on_a_forked_stream_in_a_capture(e4b):
    """Inside a capture, calls on a stream that forks from the capturing one and joins it again."""
    keep, calls = _calls(e4b)
    names = ("dispatch", "combine", "block_backward", "linear")
    want = {n: [t.clone() for t in calls[n](None)] for n in names}
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = {n: calls[n](side) for n in names}
        main.wait_stream(side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            for a, b in zip(want[n], got[n]):
                assert torch.equal(a, b), n
