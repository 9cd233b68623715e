"""Sliding-window attention with sinks, forward and backward, against the 64-bit reference at the
derived element-wise bounds (tests/cache_ref.py)."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import make_qkv_kv

pytestmark = pytest.mark.gpu


def within(got, want, bound, name):
    got = np.asarray(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    over = np.abs(got - want) - bound
    at = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over.max() <= 0, f"{name}: {int((over > 0).sum())} values out of bounds, worst {at}: {got[at]} for {want[at]} +- {bound[at]}"


def both(B, Lq, Lk, H, Hkv, D, dtype, window, sinks, seed, train=True):
    q, k, v, do = make_qkv_kv(B, Lq, Lk, H, Hkv, D, dtype, seed, with_do=True)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.window_fwd(*dev[:3], window, sinks)
    grads = fa.window_attention_backward(*dev[:3], o, lse, dev[3], window, sinks) if train else None
    torch.cuda.synchronize()
    fa.check_device_error()
    return [to64(x) for x in (q, k, v, do)], to64(o), to64(lse), grads and [to64(x) for x in grads[:3]]


CASES = [
    # B, Lq, Lk, H, Hkv, D, dtype, window, sinks
    (1, 1, 1, 1, 1, 64, "fp16", 1, 0),
    (1, 1, 700, 4, 2, 128, "bf16", 300, 4),
    (2, 128, 128, 2, 1, 64, "bf16", 1, 0),        # each query sees itself alone
    (1, 300, 300, 2, 2, 128, "fp16", 1, 3),
    (1, 257, 257, 4, 2, 128, "bf16", 128, 0),
    (1, 640, 640, 2, 1, 64, "fp16", 127, 1),
    (2, 777, 777, 4, 4, 64, "fp16", 200, 1),
    (1, 1000, 1000, 4, 1, 128, "bf16", 129, 130),  # sinks over two tiles
    (1, 512, 1500, 2, 2, 128, "fp16", 256, 0),     # keys that no query sees
    (1, 384, 1111, 2, 1, 64, "bf16", 100, 7),
    (1, 900, 900, 2, 2, 128, "fp16", 5000, 10),    # wider than the sequence: causal
    (1, 500, 500, 2, 2, 64, "bf16", 64, 500),      # every key a sink: causal
    (3, 200, 1200, 8, 2, 128, "bf16", 1024, 4),
]


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,dtype,window,sinks", CASES)
def test_window_forward_and_backward(cuda_lib, B, Lq, Lk, H, Hkv, D, dtype, window, sinks):
    (q, k, v, do), o, lse, grads = both(B, Lq, Lk, H, Hkv, D, dtype, window, sinks, seed=Lq + Lk + window)
    mask = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks)
    O, L, bound = ref.forward(q, k, v, mask, dtype)
    within(o, O, bound, "O")
    within(lse, L, np.full(L.shape, ref.FP32), "LSE")
    for name, g, r, e in zip(("dQ", "dK", "dV"), grads, *ref.backward(q, k, v, do, mask, dtype)):
        within(g, r, e, name)
    unseen = ~mask.any(axis=0)
    assert not grads[1][:, unseen].any() and not grads[2][:, unseen].any()


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_window_many_tiles(cuda_lib, D, dtype):
    """More K/V tiles and Q pairs than SMs: the persistent CTAs' shares of sink and window tiles."""
    B, L, H, Hkv, window, sinks = 2, 2304, 16, 8, 333, 4
    (q, k, v, do), o, lse, grads = both(B, L, L, H, Hkv, D, dtype, window, sinks, seed=D)
    mask = ref.seen(np.arange(L), L, window, sinks)
    O, lse_r, bound = ref.forward(q, k, v, mask, dtype)
    within(o, O, bound, "O")
    within(lse, lse_r, np.full(lse_r.shape, ref.FP32), "LSE")
    for name, g, r, e in zip(("dQ", "dK", "dV"), grads, *ref.backward(q, k, v, do, mask, dtype)):
        within(g, r, e, name)


def test_a_wide_window_is_the_causal_call(cuda_lib):
    """Bit for bit where both run the same schedule (more Q tiles than SMs)."""
    q, k, v, _ = make_qkv_kv(2, 600, 900, 32, 2, 128, "bf16", 3)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    o1, l1 = fa.fwd(qd, kd, vd, causal=True)
    o2, l2 = fa.window_fwd(qd, kd, vd, 900)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_rising_maxima(cuda_lib):
    """Every tile's scores lie far above the last one's, so the running max moves at every tile, and
    from -inf where a row's window starts behind the first tile of its pair."""
    L, D, window = 700, 64, 150
    q, k, v, do = make_qkv_kv(1, L, L, 2, 2, D, "fp16", 9, with_do=True)
    q[...] = 0.0
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(L) / 16.0).view(1, L, 1).to(k.dtype)
    o, lse = fa.window_fwd(q.cuda(), k.cuda(), v.cuda(), window, 0)
    torch.cuda.synchronize()
    mask = ref.seen(np.arange(L), L, window)
    O, lse_r, bound = ref.forward(to64(q), to64(k), to64(v), mask, "fp16")
    within(to64(o), O, bound, "O")
    # scores up to 44, exact in fp32 but for their scaling (2^-23 relative)
    within(to64(lse), lse_r, ref.FP32 + np.abs(lse_r) * 2.0 ** -20, "LSE")


def test_gradients_against_differences(cuda_lib):
    """<gradient, d> against (f(x + h d) - f(x - h d)) / 2h of the 64-bit forward."""
    Lq, Lk, window, sinks = 150, 260, 70, 2
    (q, k, v, do), _, _, grads = both(1, Lq, Lk, 2, 1, 64, "fp16", window, sinks, seed=4)
    mask = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks)
    _, bounds = ref.backward(q, k, v, do, mask, "fp16")
    f = lambda a, b, c: float((ref.forward(a, b, c, mask, "fp16")[0] * do).sum())  # noqa: E731
    r, h = np.random.default_rng(1), 1e-5
    for i, (x, g, e) in enumerate(zip((q, k, v), grads, bounds)):
        d = r.standard_normal(x.shape)
        args = [[q, k, v], [q, k, v]]
        args[0][i], args[1][i] = x + h * d, x - h * d
        slope = (f(*args[0]) - f(*args[1])) / (2 * h)
        assert abs(slope - (g * d).sum()) <= (e * np.abs(d)).sum() + 1e-5 * abs(slope)


def test_captured_and_replayed(cuda_lib):
    """One graph of forward and backward, replayed with other inputs in the same buffers."""
    args = (2, 300, 300, 4, 2, 128, "bf16")
    a, b = (make_qkv_kv(*args, seed, with_do=True) for seed in (1, 2))
    bufs = [x.cuda() for x in a]
    o, lse = fa.window_fwd(*bufs[:3], 100, 4)
    acc = fa.alloc_window_workspace(2, 300, 300, 4, 2, 128, 100, 4, "cuda")
    fa.window_attention_backward(*bufs[:3], o, lse, bufs[3], 100, 4, dq_accum=acc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.window_fwd(*bufs[:3], 100, 4)
        grads = fa.window_attention_backward(*bufs[:3], o, lse, bufs[3], 100, 4, dq_accum=acc)
    for data in (b, a):
        for dst, src in zip(bufs, data):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        mask = ref.seen(np.arange(300), 300, 100, 4)
        q, k, v, do = (to64(x) for x in data)
        O, _, bound = ref.forward(q, k, v, mask, "bf16")
        within(to64(o), O, bound, "O")
        for name, g, r, e in zip(("dQ", "dK", "dV"), grads, *ref.backward(q, k, v, do, mask, "bf16")):
            within(to64(g), r, e, name)


def test_on_another_stream(cuda_lib):
    q, k, v, _ = make_qkv_kv(1, 400, 400, 4, 4, 64, "fp16", 5)
    dev = [x.cuda() for x in (q, k, v)]
    want, _ = fa.window_fwd(*dev, 130, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = torch.empty_like(dev[0]), torch.empty(1, 4, 400, device="cuda")
    fa.window_fwd(*dev, 130, 1, out=out, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_refusals(cuda_lib):
    q, k, v, _ = make_qkv_kv(1, 8, 8, 2, 2, 64, "fp16", 0)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(_lib.FAError) as e:
            fa.window_fwd(q, k, v, window, sinks)
        assert e.value.status == _lib.FA_ERR_INVALID_ARG
    with pytest.raises(_lib.FAError):
        fa.window_fwd(q, k[:, :4].contiguous(), v[:, :4].contiguous(), 4)    # more queries than keys
    with pytest.raises(ValueError):
        fa.window_fwd(q, k[:, :4], v, 4)
    big = torch.zeros(1, 600, 2, 64, dtype=torch.float16, device="cuda")
    lse = torch.zeros(1, 2, 600, device="cuda")
    with pytest.raises(_lib.FAError) as e:                       # no room for the sink keys' parts
        fa.window_bwd(big, big, big, big, lse, lse, 100, 4, dq_accum=fa.alloc_workspace(1, 600, 2, 64, "cuda"))
    assert e.value.status == _lib.FA_ERR_SCRATCH_TOO_SMALL
    with pytest.raises(TypeError):
        fa.window_fwd(q.cpu(), k, v, 4)


@pytest.mark.parametrize("B,H,Lq,Lk,D,window,sinks", [(1, 1, 128, 128, 64, 40, 0), (1, 2, 129, 129, 128, 129, 0),
                                                      (1, 4, 100, 2000, 128, 1500, 200), (2, 8, 300, 1300, 64, 500, 4)])
def test_one_tile_per_cta(cuda_lib, B, H, Lq, Lk, D, window, sinks):
    """Few Q tiles: the two warpgroups share one tile's steps (an odd and an even number of them, one
    alone, and rows that see nothing of one warpgroup's steps)."""
    (q, k, v, do), o, lse, _ = both(B, Lq, Lk, H, H, D, "bf16", window, sinks, seed=Lq + D, train=False)
    mask = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks)
    O, lse_r, bound = ref.forward(q, k, v, mask, "bf16")
    within(o, O, bound, "O")
    within(lse, lse_r, np.full(lse_r.shape, ref.FP32), "LSE")


def test_a_refused_backward_leaves_everything_alone():
    """No part of a refused call runs, the step that sums O dO among them."""
    x = torch.randn(1, 200, 2, 64, device="cuda").half()
    lse = torch.zeros(1, 2, 200, device="cuda")
    delta, dq, ws = torch.full_like(lse, 7.0), torch.full_like(x, 7.0), torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")
    for window, sinks, w in ((0, 0, ws), (64, -1, ws), (64, 0, ws[:1024])):
        with pytest.raises(_lib.FAError):
            _lib.check("fa_window_bwd", _lib.binding().window_bwd(
                x, x, x, x, lse, x, delta, window, sinks, dq, None, None, w, False, None))
    torch.cuda.synchronize()
    assert (delta == 7).all() and (dq == 7).all() and (ws == 7).all()


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,dtype,window,sinks", [
    (1, 735, 735, 16, 2, 128, "bf16", 723, 4),      # eight heads a unit's share each, no far units
    (1, 900, 1100, 12, 2, 64, "fp16", 200, 130),    # six heads, two sink tiles with far units, a past
    (2, 640, 640, 8, 1, 128, "fp16", 100, 1),
    (1, 130, 1500, 8, 1, 64, "bf16", 300, 700),     # tiles that no query sees
])
def test_few_units_are_cut_by_heads(cuda_lib, B, Lq, Lk, H, Hkv, D, dtype, window, sinks):
    """dK and dV of a K/V head added up from several units' query heads."""
    (q, k, v, do), _, _, grads = both(B, Lq, Lk, H, Hkv, D, dtype, window, sinks, seed=H)
    own = B * Hkv * -(-Lk // 128) * 2 * 128 * D * 4
    size = fa.window_workspace_size(B, Lq, Lk, H, Hkv, D, window, sinks)
    assert size >= _lib.load().fa_bwd_workspace_size(B, Lq, H, D) + 2 * own  # (so it is cut)
    mask = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks)
    for name, g, r, e in zip(("dQ", "dK", "dV"), grads, *ref.backward(q, k, v, do, mask, dtype)):
        within(g, r, e, name)
    unseen = ~mask.any(axis=0)
    assert not grads[1][:, unseen].any() and not grads[2][:, unseen].any()
