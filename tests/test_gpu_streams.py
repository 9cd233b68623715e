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
