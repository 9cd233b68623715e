"""The append to the paged cache with the rotation on the way: the same bits as rope_fwd and
paged_write one after the other, which are tested against 64 bits."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref, rope_ref
from tests.helpers import to64
from tests.test_gpu_rope import BASE, freqs
from tests.test_gpu_window import within
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import storage_dtype

pytestmark = pytest.mark.gpu

CASES = [
    # B, L, H, Hkv, D, dtype, page, rotary, axes (0: none given), interleaved, counts, weights
    (1, 1, 1, 1, 64, "fp16", 16, 64, 0, False, False, None),
    (1, 1, 32, 8, 128, "bf16", 16, 128, 1, False, False, "zero"),
    (3, 37, 4, 2, 64, "fp16", 16, 32, 2, True, True, "new"),
    (5, 2, 7, 1, 128, "bf16", 256, 128, 3, False, False, None),
    (70, 1, 8, 8, 64, "bf16", 64, 16, 0, True, False, "zero"),
    (2, 300, 6, 3, 128, "fp16", 32, 96, 1, False, True, None),
]


@pytest.mark.parametrize("B,L,H,Hkv,D,dtype,page,rotary,axes,inter,ragged,weigh", CASES)
@pytest.mark.parametrize("joint", [False, True])
def test_append(cuda_lib, B, L, H, Hkv, D, dtype, page, rotary, axes, inter, ragged, weigh, joint):
    g = torch.Generator().manual_seed(L + D + B)
    dt = storage_dtype(dtype)
    P = -(-(L + 40) // page)
    pages = B * P + 2
    kv = torch.randn(pages, 2, page, Hkv, D, generator=g).to(dt).cuda()
    qkv = torch.randn(B, L, H + 2 * Hkv, D, generator=g).to(dt).cuda()
    q, k, v = qkv.split([H, Hkv, Hkv], 2)
    bt = torch.randperm(pages, generator=g)[: B * P].view(B, P).to(torch.int32)
    start = torch.randint(-3, 45, (B,), generator=g, dtype=torch.int32)    # some begin before, end behind the table
    if B > 1:
        bt[1, 0], bt[0, P - 1] = 10 ** 6, -4                               # not pages: skipped
    bt, start = bt.cuda(), start.cuda()
    counts = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32).cuda() if ragged else None
    pos = torch.randint(0, 100000, (axes, B, L), generator=g, dtype=torch.int32).cuda() if axes else None
    table = fa.rope_table(D, BASE, rotary, axes=torch.randint(0, max(axes, 1), (rotary // 2,), generator=g).tolist())
    w = torch.full((B, Hkv, P * page + 3), 7.0, device="cuda") if weigh else None
    nw = torch.rand(B, Hkv, L, generator=g).cuda() if weigh == "new" else None
    want_kv, want_w = kv.clone(), None if w is None else w.clone()
    at = pos if axes else (start[:, None] + torch.arange(L, device="cuda", dtype=torch.int32))[None].contiguous()
    want_q, kr = fa.rope_fwd(q, k, table, at, inter)
    fa.paged_write(kr, v.contiguous(), want_kv[:, 0], want_kv[:, 1], bt, start, counts, want_w, nw)
    pools = (kv[:, 0], kv[:, 1]) if joint else (kv[:, 0].contiguous(), kv[:, 1].contiguous())
    got = fa.paged_append(q, k, v, *pools, bt, start, table, pos, counts, inter, w, nw)
    torch.cuda.synchronize()
    assert torch.equal(got, want_q)
    assert torch.equal(pools[0], want_kv[:, 0]) and torch.equal(pools[1], want_kv[:, 1])
    assert w is None or torch.equal(w, want_w)
    again = fa.paged_append(q, k, v, *pools, bt, start, table, pos, counts, inter, w, nw, out=q)   # in place
    torch.cuda.synchronize()
    assert again.data_ptr() == q.data_ptr() and torch.equal(q, want_q) and torch.equal(pools[0], want_kv[:, 0])


def test_slots_past_32_bits(cuda_lib):
    """Pages whose elements lie beyond 2^31 and 2^32 of the pool's first (9 GB)."""
    page, Hkv, D = 16, 8, 128
    pages = (1 << 32) // (page * Hkv * D) + 3
    pool = torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    bt = torch.tensor([[pages - 1], [pages // 2 + 1]], dtype=torch.int32, device="cuda")
    start = torch.tensor([15, 3], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(2, 1, h, D, generator=g).bfloat16().cuda() for h in (16, 8))
    table = fa.rope_table(D)
    keep = pool[[pages - 1, pages // 2 + 1]].clone()
    # K and V into one pool: position 0 turns nothing, so both write the same
    fa.paged_append(q, k, k, pool, pool, bt, start, table, torch.zeros(1, 2, 1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    keep[0, 15], keep[1, 3] = k[0, 0], k[1, 0]
    assert torch.equal(pool[[pages - 1, pages // 2 + 1]], keep)


def test_prompt_then_steps(cuda_lib):
    """As it is used: a prompt appended and attended to, then tokens one by one, each against the 64-bit
    attention over the turned sequence (its values as they are stored)."""
    B, L, H, Hkv, D, page, steps = 2, 70, 4, 2, 64, 16, 3
    g = torch.Generator().manual_seed(3)
    n = L + steps
    qkv = torch.randn(B, n, H + 2 * Hkv, D, generator=g).bfloat16()
    q, k, v = qkv.split([H, Hkv, Hkv], 2)
    table, dev = fa.rope_table(D), qkv.cuda()
    turned = fa.rope_fwd(*dev.split([H, Hkv, Hkv], 2)[:2], table)
    pos = np.broadcast_to(np.arange(n), (1, B, n))
    for x, y in zip((q, k), turned):
        within(to64(y), *rope_ref.turned(to64(x), pos, freqs(D), [0] * 32, D, False, "bf16"), "turned")
    O, _, bound = cache_ref.forward(to64(turned[0]), to64(turned[1]), to64(v), cache_ref.seen(np.arange(n), n), "bf16")
    P = -(-n // page)
    kc, vc = (torch.full((B * P, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.randperm(B * P, generator=g).view(B, P).to(torch.int32).cuda()
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    t = 0
    for count in [L] + [1] * steps:
        x, y, z = dev[:, t: t + count].split([H, Hkv, Hkv], 2)
        qr = fa.paged_append(x, y, z, kc, vc, bt, start, table)
        if count == L:
            o, _ = fa.fwd(qr, turned[1][:, :L].contiguous(), z.contiguous(), True)
        else:
            o, _ = fa.paged_decode(qr, kc, vc, bt, start + 1)
        torch.cuda.synchronize()
        within(to64(o), O[:, t: t + count], bound[:, t: t + count], f"O at {t}")
        start += count
        t += count
    fa.check_device_error()


def test_captured(cuda_lib):
    """In a graph: new tokens, places and positions between replays."""
    B, H, Hkv, D, page = 3, 8, 2, 128, 16
    g = torch.Generator().manual_seed(9)
    kc, vc = (torch.zeros(12, page, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
    qkv = torch.zeros(B, 1, H + 2 * Hkv, D, dtype=torch.float16, device="cuda")
    q, k, v = qkv.split([H, Hkv, Hkv], 2)
    bt = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    start, pos = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(1, B, 1, dtype=torch.int32, device="cuda")
    table = fa.rope_table(D)
    out = fa.paged_append(q, k, v, kc, vc, bt, start, table, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.paged_append(q, k, v, kc, vc, bt, start, table, pos)
    for i in range(3):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        start.copy_(torch.randint(0, 64, (B,), generator=g))
        pos.copy_(torch.randint(0, 10 ** 6, pos.shape, generator=g))
        want = kc.clone(), vc.clone()
        wq = fa.paged_append(q, k, v, *want, bt, start, table, pos)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wq) and torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_refusals(cuda_lib):
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.float16, device="cuda")
    q, k = (torch.zeros(2, 3, h, 64, dtype=torch.float16, device="cuda") for h in (4, 2))
    bt, start = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    table = fa.rope_table(64)
    good = dict(q=q, k=k, v=k, k_cache=kc, v_cache=kc, block_table=bt, start=start, table=table)
    call = lambda **kw: fa.paged_append(**dict(good, counts=start, **kw) if "counts" not in kw else dict(good, **kw))  # noqa: E731
    call()                                                                  # (no token counts: nothing is written)
    for err, kw in ((TypeError, dict(positions=torch.zeros(1, 2, 3, device="cuda"))), (ValueError, dict(positions=start)),
                    (TypeError, dict(counts=start.long())), (ValueError, dict(counts=start[:1])),
                    (ValueError, dict(weights=torch.zeros(2, 2, 5, device="cuda"))), (ValueError, dict(out=q[:, :2]))):
        with pytest.raises(err):
            call(**kw)
    for kw in (dict(q=q[:, :, :3]), dict(new_weights=torch.zeros(2, 2, 3, device="cuda"))):
        with pytest.raises(_lib.FAError) as e:
            fa.paged_append(**dict(good, counts=start, **kw))
        assert e.value.status == _lib.FA_ERR_INVALID_ARG
    for kw in (dict(k=q), dict(v=k.contiguous()[:, :2]), dict(start=start[:1]), dict(block_table=bt[:1])):
        with pytest.raises(ValueError):
            fa.paged_append(**dict(good, counts=start, **kw))
    torch.cuda.synchronize()
