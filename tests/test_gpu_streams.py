"""What a call given a stream allocates belongs to that stream (the dense calls; the window and cache
calls are tested beside their results)."""

import pytest
import torch

import tiled_attention_fa_gb300 as fa

pytestmark = pytest.mark.gpu


def owner(t):
    return [s["stream"] for s in torch.cuda.memory_snapshot()
            if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]


@pytest.mark.parametrize("form", ["object", "handle"])
def test_dense_calls(cuda_lib, form):
    q = torch.randn(2, 256, 4, 128, device="cuda").half()
    codes = torch.zeros(1, 128, 2, 128, dtype=torch.uint8, device="cuda")
    one = torch.randn(2, 1, 4, 128, device="cuda").half()
    want_o, want_lse = fa.fwd(q, q, q, True)
    want = fa.attention_backward(q, q, q, want_o, want_lse, q, True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = side if form == "object" else side.cuda_stream
    o, lse = fa.fwd(q, q, q, True, stream=stream)
    delta = fa.bwd_preprocess(o, q, stream=stream)
    grads = fa.bwd(q, q, q, o, q, lse, delta, True, stream=stream)
    again = fa.attention_backward(q, q, q, o, lse, q, True, stream=stream)
    with torch.cuda.stream(side):
        acc = torch.zeros(fa.workspace_size(2, 256, 4, 128) // 4, device="cuda")
    main = fa.bwd_main(q, q, q, q, lse, delta, acc, True, stream=stream)
    outs = [o, lse, delta, *grads, *again, *main, *fa.fwd_fp8(codes, codes, codes, 1.0, 1.0, 1.0, stream=stream),
            *fa.decode(one, q, q, stream=stream)]
    torch.cuda.synchronize()
    fa.check_device_error()
    for t in outs:
        assert owner(t) == [side.cuda_stream]
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse) and torch.equal(delta, want[3])
    for a, b, c, w in zip(grads[1:], again[1:3], main, want[1:3]):
        assert torch.equal(a, w) and torch.equal(b, w) and torch.equal(c, w)


def test_the_default_stream_by_its_handle(cuda_lib):
    """Stream 0 named from under another current stream."""
    q = torch.randn(1, 200, 2, 64, device="cuda").half()
    want, _ = fa.fwd(q, q, q)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        o, lse = fa.fwd(q, q, q, stream=0)
    torch.cuda.synchronize()
    assert owner(o) == [0] and owner(lse) == [0] and torch.equal(o, want)


def _work(seed):
    """Inputs of one run through the window and cache calls, and the run."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()
    B, H, Hkv, D, page, P = 3, 8, 2, 128, 32, 60
    x, y, do = rnd(2, 500, H, D), rnd(2, 500, Hkv, D), rnd(2, 500, H, D)
    q = rnd(B, 2, H, D)
    pools = [rnd(B * (P + 10), page, Hkv, D) for _ in range(2)]
    table = torch.randperm(B * (P + 10), device="cuda", generator=g).int().view(B, P + 10)
    src, dst = table[:, :P].contiguous(), table[:, P:].contiguous()
    lens = torch.tensor([1900, 700 + seed, 33], dtype=torch.int32, device="cuda")
    w = torch.rand(B, Hkv, P * page, device="cuda", generator=g)

    def run():
        o, lse = fa.window_fwd(x, y, y, 130, 4)
        grads = fa.window_attention_backward(x, y, y, o, lse, do, 130, 4)
        kw = fa.key_weights(x, y, lse, True, 130, 4)
        wi = w.clone()
        d, dl = fa.paged_decode(q, *pools, src, lens, weights=wi)
        kept, nl, nw = fa.paged_evict(*pools, src, lens, wi, dst, 300, 4, 50)
        e, el = fa.paged_decode(q, *pools, dst, nl, 64, 2, weights=nw)
        return [o, lse, *grads[1:], kw, wi, d, dl, kept, nl, nw, e, el]      # (dQ is summed by atomics)
    return run


def test_two_streams_at_once(cuda_lib):
    """Every call on two streams at the same time, many rounds: the same bits as alone."""
    runs = [_work(1), _work(2)]
    alone = [r() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                outs.append(r())
        torch.cuda.synchronize()
        for got, want in zip(outs, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    fa.check_device_error()


def test_two_graphs_at_once(cuda_lib):
    """The same captured, both graphs replayed at the same time, eager calls between."""
    runs = [_work(3), _work(4)]
    alone = [r() for r in runs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in runs]
    for r in runs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(r())
        graphs.append(gr)
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = runs[0]()
        torch.cuda.synchronize()
        for got, want in zip(outs + [eager], alone + [alone[0]]):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    fa.check_device_error()
