"""Decoding over a paged key/value cache, and writing into it, against the 64-bit reference
(tests/cache_ref.py).  Slots that no query may use hold NaN."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_window import within
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import storage_dtype

pytestmark = pytest.mark.gpu

# A key's accumulated weight is a sum of probabilities, each off by at most FP32 relative.
W_REL, W_ABS = ref.FP32, 1e-7


def cache(B, Hkv, D, dtype, page, lens, seed, P=None, window=0, sinks=0, Lq=1, joint=False):
    """Pools with the sequences' keys in pages in random order and NaN in every slot that no query
    sees; pages wholly unseen are absent from the table (-1)."""
    g = torch.Generator().manual_seed(seed)
    P = P or max(1, -(-max(lens) // page))
    dt = storage_dtype(dtype)
    pages = B * P + 3
    kv = torch.randn(pages, 2, page, Hkv, D, generator=g).to(dt)
    table = torch.randperm(pages, generator=g)[: B * P].view(B, P).to(torch.int32)
    use = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            if not window or t > max(n - Lq, 0) - window or t < sinks:
                use[table[b, t // page], t % page] = True
    kv.permute(0, 2, 1, 3, 4)[~use] = float("nan")
    for b in range(B):
        for j in range(P):
            if not use[table[b, j]].any():
                table[b, j] = -1
    kv = kv.cuda()
    k, v = kv[:, 0], kv[:, 1]
    if not joint:
        k, v = k.contiguous(), v.contiguous()
    return k, v, table, torch.tensor(lens, dtype=torch.int32)


def check(B, Lq, H, Hkv, D, dtype, page, lens, window=0, sinks=0, seed=0, P=None, joint=False, weigh=True):
    k, v, table, ln = cache(B, Hkv, D, dtype, page, lens, seed, P, window, sinks, Lq, joint)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(B, Lq, H, D, generator=g).to(storage_dtype(dtype))
    w0 = torch.rand(B, Hkv, table.shape[1] * page + 5, generator=g)
    w = w0.cuda()
    o, lse = fa.paged_decode(q.cuda(), k, v, table.cuda(), ln.cuda(), window, sinks, weights=w if weigh else None)
    torch.cuda.synchronize()
    fa.check_device_error()
    k64, v64 = (np.nan_to_num(to64(x)) for x in (k, v))    # hidden slots are multiplied by 0 there
    O, L, bound, W = ref.paged_decode(to64(q), k64, v64, table.numpy(), lens, dtype, window, sinks, to64(w0))
    within(to64(o), O, bound, "O")
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(to64(lse)), empty)
    within(np.where(empty, 0, to64(lse)), np.where(empty, 0, L), np.full(L.shape, ref.FP32), "LSE")
    if weigh:
        within(to64(w), W, W_REL * (W - to64(w0)) + W_ABS + 2.0 ** -23 * W, "weights")


CASES = [
    # B, Lq, H, Hkv, D, dtype, page, lens, window, sinks
    (1, 1, 1, 1, 64, "fp16", 16, [1], 0, 0),
    (1, 1, 8, 8, 128, "bf16", 16, [500], 0, 0),
    (3, 1, 8, 2, 128, "bf16", 64, [1, 0, 777], 0, 0),
    (2, 1, 4, 4, 64, "bf16", 128, [128, 129], 0, 0),
    (5, 1, 32, 8, 128, "fp16", 32, [0, 4096, 3, 2049, 127], 0, 0),
    (2, 3, 8, 1, 64, "fp16", 16, [1000, 2], 0, 0),          # three drafted tokens, two keys: an empty query
    (2, 5, 4, 2, 128, "bf16", 256, [513, 700], 0, 0),
    (1, 16, 16, 2, 128, "bf16", 64, [900], 0, 0),           # 128 packed rows
    (2, 9, 5, 1, 64, "bf16", 32, [300, 44], 0, 0),          # 45 packed rows
    (1, 30, 1, 1, 128, "fp16", 16, [257], 0, 0),
    (2, 12, 1, 1, 64, "fp16", 16, [64, 100], 0, 0),         # 12 packed rows
    (2, 1, 4, 2, 128, "bf16", 16, [1500, 90], 200, 4),
    (3, 4, 8, 2, 64, "fp16", 64, [1000, 300, 2], 130, 1),
    (2, 2, 4, 1, 128, "bf16", 128, [2000, 600], 128, 300),  # sinks over three tiles
    (1, 1, 2, 2, 128, "fp16", 32, [1025], 1, 0),            # a token sees itself alone
]


@pytest.mark.parametrize("B,Lq,H,Hkv,D,dtype,page,lens,window,sinks", CASES)
def test_paged_decode(cuda_lib, B, Lq, H, Hkv, D, dtype, page, lens, window, sinks):
    check(B, Lq, H, Hkv, D, dtype, page, lens, window, sinks, seed=sum(lens) + D)


def test_many_unequal_sequences(cuda_lib):
    """More sequences than threads that scan them, most of them short or empty."""
    lens = [(37 * i * i) % 211 if i % 3 else 0 for i in range(300)]
    check(300, 1, 4, 2, 64, "fp16", 16, lens, seed=3)


def test_wide_table_and_joint_pool(cuda_lib):
    """A table wider than any sequence needs, K and V as halves of one pool."""
    check(2, 1, 8, 2, 128, "bf16", 32, [700, 40], seed=5, P=200, joint=True)


def test_long_sequence(cuda_lib):
    check(1, 1, 8, 2, 128, "bf16", 64, [40000], seed=6)


def test_rising_scores(cuda_lib):
    """Each tile's scores lie above the last one's, so the running max moves at every tile."""
    n, D, page = 1400, 64, 16
    k, v, table, ln = cache(1, 2, D, "fp16", page, [n], 8)
    flat = table[0].long()
    k[...] = 0
    k[flat, :, :, 0] = (torch.arange(len(flat) * page) / 16.0).view(-1, page, 1).to(k.dtype).cuda()
    v.nan_to_num_()
    q = torch.zeros(1, 2, 4, D, dtype=torch.float16)
    q[..., 0] = 8.0
    w = torch.zeros(1, 2, table.shape[1] * page, device="cuda")
    o, lse = fa.paged_decode(q.cuda(), k, v, table.cuda(), ln.cuda(), weights=w)
    torch.cuda.synchronize()
    O, L, bound, W = ref.paged_decode(to64(q), to64(k), to64(v), table.numpy(), [n], "fp16", weights=np.zeros((1, 2, w.shape[2])))
    within(to64(o), O, bound, "O")
    # scores up to 88, scaled in fp32 (2^-22 relative): as much off a probability's exponent
    within(to64(lse), L, ref.FP32 + np.abs(L) * 2.0 ** -20, "LSE")
    within(to64(w), W, (W_REL + 88 * 2.0 ** -21) * W + W_ABS, "weights")


def test_wrong_tables_and_lengths_stay_in_bounds(cuda_lib):
    """Page ids outside the pool read as zeros; lengths are clamped to the table."""
    k, v, table, _ = cache(3, 2, 64, "bf16", 16, [64, 64, 64], 4)
    table[0, 1], table[1, 2] = 10 ** 9, -(10 ** 9)
    ln = [64, 10 ** 9, -5]
    q = torch.randn(3, 1, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o, lse = fa.paged_decode(q.cuda(), k, v, table.cuda(), torch.tensor(ln, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    fa.check_device_error()
    k64, v64 = to64(k), to64(v)
    zero = np.zeros((1,) + k64.shape[1:])
    t = np.where((table.numpy() < 0) | (table.numpy() >= len(k64)), len(k64), table.numpy())
    O, L, bound, _ = ref.paged_decode(to64(q), np.concatenate([k64, zero]), np.concatenate([v64, zero]), t, [64, 64, 0], "bf16")
    within(to64(o), O, bound, "O")
    within(to64(lse)[:2], L[:2], np.full(L[:2].shape, ref.FP32), "LSE")
    assert np.isneginf(to64(lse)[2]).all()


def test_sequences_that_share_pages(cuda_lib):
    """A common prefix: the same pages in two tables; each sequence has weights of its own."""
    k, v, table, ln = cache(2, 2, 128, "fp16", 16, [320, 320], 9)
    table[1, :10] = table[0, :10]
    q = torch.randn(2, 1, 4, 128, generator=torch.Generator().manual_seed(2)).to(torch.float16)
    w = torch.zeros(2, 2, 320, device="cuda")
    fa.paged_decode(q.cuda(), k, v, table.cuda(), ln.cuda(), weights=w)
    first = w.clone()
    w.zero_()
    fa.paged_decode(q.cuda(), k, v, table.cuda(), ln.cuda(), weights=w)
    torch.cuda.synchronize()
    assert torch.equal(first, w)
    _, _, _, W = ref.paged_decode(to64(q), to64(k), to64(v), table.numpy(), [320, 320], "fp16", weights=np.zeros((2, 2, 320)))
    within(to64(w), W, W_REL * W + W_ABS, "weights")


def test_write(cuda_lib):
    B, L, Hkv, D, page, P = 3, 37, 2, 64, 16, 5
    g = torch.Generator().manual_seed(1)
    kv = torch.randn(20, 2, page, Hkv, D, generator=g).to(torch.float16).cuda()
    kc, vc = kv[:, 0], kv[:, 1]
    before = kv.clone()
    table = torch.randperm(20, generator=g)[: B * P].view(B, P).to(torch.int32)
    table[2, 1] = 99                                            # not a page: skipped
    start, counts = torch.tensor([5, 60, -2], dtype=torch.int32), torch.tensor([37, 30, 25], dtype=torch.int32)
    k, v = (torch.randn(B, L, Hkv, D, generator=g).to(torch.float16).cuda() for _ in range(2))
    w = torch.full((B, Hkv, P * page + 3), 7.0, device="cuda")
    nw = torch.rand(B, Hkv, L, generator=g).cuda()
    fa.paged_write(k, v, kc, vc, table.cuda(), start.cuda(), counts.cuda(), w, nw)
    torch.cuda.synchronize()
    want, ww = before.clone(), torch.full_like(w, 7.0)
    for b in range(B):
        for j in range(int(counts[b])):
            pos = int(start[b]) + j
            if 0 <= pos < P * page and int(table[b, pos // page]) < 20:
                pid = int(table[b, pos // page])
                want[pid, 0, pos % page], want[pid, 1, pos % page] = k[b, j], v[b, j]
                ww[b, :, pos] = nw[b, :, j]
    assert torch.equal(kv, want) and torch.equal(w, ww)
    fa.paged_write(k, v, kc, vc, table.cuda(), start.cuda(), weights=w)
    torch.cuda.synchronize()
    assert not w[0, :, 5:42].any() and (w[0, :, 42:] == 7).all()


def test_prompt_then_steps(cuda_lib):
    """A run as it is used: a prompt with a window, its keys written to the cache, then tokens one
    by one, each equal to the dense window attention over the sequence so far."""
    B, L, H, Hkv, D, page, window, sinks, steps = 2, 150, 4, 2, 64, 16, 60, 3, 4
    g = torch.Generator().manual_seed(3)
    n = L + steps
    q, k, v = (torch.randn(B, n, h, D, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    P = -(-n // page)
    kc = torch.full((B * P, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = torch.randperm(B * P, generator=g).view(B, P).to(torch.int32).cuda()
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    prompt, _ = fa.window_fwd(q[:, :L].contiguous(), k[:, :L].contiguous(), v[:, :L].contiguous(), window, sinks)
    fa.paged_write(k[:, :L].contiguous(), v[:, :L].contiguous(), kc, vc, table, start)
    lens = start + L
    mask = ref.seen(np.arange(n), n, window, sinks)
    O, _, bound = ref.forward(to64(q), to64(k), to64(v), mask, "bf16")
    within(to64(prompt), O[:, :L], bound[:, :L], "O of the prompt")
    for t in range(L, n):
        one = [x[:, t: t + 1].contiguous() for x in (q, k, v)]
        fa.paged_write(one[1], one[2], kc, vc, table, lens)
        lens += 1
        o, _ = fa.paged_decode(one[0], kc, vc, table, lens, window, sinks)
        torch.cuda.synchronize()
        within(to64(o), O[:, t: t + 1], bound[:, t: t + 1], f"O at {t}")


def test_captured_step(cuda_lib):
    """Write, decode and weights in one graph; lengths and tokens change between replays."""
    B, H, Hkv, D, page, n = 2, 8, 2, 128, 16, 200
    k, v, table, _ = cache(B, Hkv, D, "bf16", page, [n + 3, n + 3], 5)
    g = torch.Generator().manual_seed(9)
    tok = [[torch.randn(B, 1, h, D, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv)] for _ in range(2)]
    q, kn, vn = (x.cuda() for x in tok[0])
    start = torch.tensor([n, 77], dtype=torch.int32, device="cuda")
    lens = start + 1
    tab = table.cuda()
    w = torch.zeros(B, Hkv, tab.shape[1] * page, device="cuda")
    ws = torch.empty(fa.paged_decode_workspace_size(B, 1, H, Hkv, D, page, tab.shape[1], True), dtype=torch.uint8, device="cuda")
    def step():
        fa.paged_write(kn, vn, k, v, tab, start, weights=w)
        return fa.paged_decode(q, k, v, tab, lens, weights=w, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    w.zero_()
    W = np.zeros(w.shape)
    for i, (a, b, c) in enumerate(tok):
        q.copy_(a)
        kn.copy_(b)
        vn.copy_(c)
        start.copy_(torch.tensor([n + i, 77 + i], dtype=torch.int32))
        lens.copy_(start + 1)
        graph.replay()
        torch.cuda.synchronize()
        ln = [n + i + 1, 78 + i]
        W[0, :, n + i], W[1, :, 77 + i] = 0, 0
        O, L, bound, W = ref.paged_decode(to64(a), to64(k), to64(v), table.numpy(), ln, "bf16", weights=W)
        within(to64(o), O, bound, "O")
        within(to64(w), W, W_REL * W + W_ABS, "weights")


def test_two_calls_at_once(cuda_lib):
    """Two streams, each with a workspace of its own."""
    args = [cache(4, 2, 64, "fp16", 32, [900, 31, 500, 1200], s) for s in (1, 2)]
    qs = [torch.randn(4, 1, 8, 64, generator=torch.Generator().manual_seed(s)).to(torch.float16).cuda() for s in (3, 4)]
    args = [(k, v, t.cuda(), n.cuda()) for k, v, t, n in args]
    want = [fa.paged_decode(q, *a)[0] for q, a in zip(qs, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(fa.paged_decode_workspace_size(4, 1, 8, 2, 64, 32, a[2].shape[1]), dtype=torch.uint8, device="cuda") for a in args]
    outs = [(torch.empty_like(q), torch.empty(4, 8, 1, device="cuda")) for q in qs]
    for _ in range(20):
        for q, a, s, x, (o, lse) in zip(qs, args, streams, ws, outs):
            fa.paged_decode(q, *a, out=o, lse=lse, workspace=x, stream=s)
    torch.cuda.synchronize()
    for (o, _), r in zip(outs, want):
        assert torch.equal(o, r)


def test_refusals(cuda_lib):
    k, v, table, ln = cache(2, 2, 64, "fp16", 16, [40, 20], 1)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.float16, device="cuda")
    t, n = table.cuda(), ln.cuda()
    fa.paged_decode(q, k, v, t, n)
    for bad, kw in ((_lib.FA_ERR_INVALID_ARG, dict(window=-1)), (_lib.FA_ERR_INVALID_ARG, dict(sinks=-1)),
                    (_lib.FA_ERR_SCRATCH_TOO_SMALL, dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(_lib.FAError) as e:
            fa.paged_decode(q, k, v, t, n, **kw)
        assert e.value.status == bad
    with pytest.raises(_lib.FAError) as e:
        fa.paged_decode(q.expand(2, 70, 4, 64).contiguous(), k, v, t, n)      # 140 packed rows
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        fa.paged_decode(q, k, v, t.long(), n)
    with pytest.raises(TypeError):
        fa.paged_decode(q.to(torch.bfloat16), k, v, t, n)
    with pytest.raises(ValueError):
        fa.paged_decode(q, k, v, t[:1], n)
    with pytest.raises(ValueError):
        fa.paged_decode(q, k, v, t, n, weights=torch.zeros(2, 2, 8, device="cuda"))
    with pytest.raises(ValueError):
        fa.paged_decode(q, k[:, :, :, :32], v[:, :, :, :32], t, n)
    odd = torch.zeros(4, 24, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(_lib.FAError) as e:
        fa.paged_decode(q, odd, odd, t, n)
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    fa.check_device_error()


def test_what_a_call_allocates_belongs_to_its_stream():
    """With a stream argument, outputs and workspace come from that stream's memory: the current
    stream's next allocation cannot get them while the kernels run."""
    B, H, Hkv, D, page = 2, 8, 2, 128, 64
    k, v, table, lens = cache(B, Hkv, D, "bf16", page, [200, 300], 5)
    table, lens = table.cuda(), lens.cuda()
    q = torch.randn(B, 1, H, D).bfloat16().cuda()
    x = torch.randn(B, 256, H, D).bfloat16().cuda()
    y = torch.randn(B, 256, Hkv, D).bfloat16().cuda()
    w = torch.rand(B, Hkv, table.shape[1] * page).cuda()
    dst = torch.tensor([[11], [12]], dtype=torch.int32).cuda()
    pools = [torch.zeros(13, page, Hkv, D, dtype=torch.bfloat16).cuda() for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = list(fa.paged_decode(q, k, v, table, lens, stream=side))
    o, lse = fa.window_fwd(x, y, y, 100, 4, stream=side)
    outs += [o, lse, fa.key_weights(x, y, lse, True, 100, 4, stream=side)]
    outs += fa.window_attention_backward(x, y, y, o, lse, o, 100, 4, stream=side)[:3]
    outs += fa.paged_evict(*pools, table % 11, lens, w, dst, 32, stream=side)
    torch.cuda.synchronize()
    fa.check_device_error()
    for t in outs:
        owner = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert owner == [side.cuda_stream]


@pytest.mark.parametrize("B,Lq,page,lo,hi", [(14, 1, 64, 8000, 16384), (32, 1, 64, 100, 700), (8, 8, 32, 300, 6000),
                                             (8, 32, 32, 300, 6000)])
def test_many_runs_under_load_give_the_same_bits(B, Lq, page, lo, hi):
    """Loads that land late or out of order change nothing.  (Zeroing the unseen rows of an item's
    last V tile once reached the tile that had the stage before, in four runs of ten at the first
    of these shapes.)"""
    P = -(-hi // page)
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(B * P, page, 8, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(B, Lq, 32, 128, device="cuda", generator=g).bfloat16()
    for _ in range(5):
        table = torch.randperm(B * P, device="cuda", generator=g).int().view(B, P)
        lens = torch.randint(lo, hi + 1, (B,), device="cuda", generator=g).int()
        outs = torch.stack([fa.paged_decode(q, k, v, table, lens)[0] for _ in range(40)])
        torch.cuda.synchronize()
        fa.check_device_error()
        differ = [i for i, o in enumerate(outs) if not torch.equal(o, outs[0])]
        assert not differ


@pytest.mark.parametrize("Lq,H,D,dtype,page,n", [(1, 4, 128, "bf16", 64, 9000), (16, 8, 128, "fp16", 64, 5000),
                                                 (1, 2, 64, "fp16", 128, 9999), (5, 3, 64, "bf16", 16, 3000)])
def test_one_item_in_many_parts(Lq, H, D, dtype, page, n):
    """One sequence and K/V head: every part ends together and counts itself in at the same word."""
    for seed in (1, 2):
        check(1, Lq, H, 1, D, dtype, page, [n], seed=seed)
