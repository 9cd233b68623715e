"""Eviction from a paged cache by accumulated weight: whole numbers and moved bits, so equal."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_window import within
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import make_qkv_kv, storage_dtype

pytestmark = pytest.mark.gpu


def setup(B, Hkv, D, dtype, page, lens, keep, seed, joint=False):
    g = torch.Generator().manual_seed(seed)
    P, P2 = max(1, -(-max(lens) // page)), -(-keep // page)
    pages = B * (P + P2) + 2
    order = torch.randperm(pages, generator=g)[: B * (P + P2)].view(B, P + P2).to(torch.int32)
    kv = torch.randn(pages, 2, page, Hkv, D, generator=g).to(storage_dtype(dtype)).cuda()
    k, v = kv[:, 0], kv[:, 1]
    if not joint:
        k, v = k.contiguous(), v.contiguous()
    w = torch.exp(2 * torch.randn(B, Hkv, P * page + 3, generator=g))
    return k, v, order[:, :P].contiguous(), order[:, P:].contiguous(), torch.tensor(lens, dtype=torch.int32), w


def check(k, v, table, dst, lens, w, keep, sinks, recent):
    B, Hkv = w.shape[:2]
    page = k.shape[1]
    k0, v0, n0 = k.clone(), v.clone(), lens.clone()
    wd = w.cuda()
    kept, new_lens, new_w = fa.paged_evict(k, v, table.cuda(), lens.cuda(), wd, dst.cuda(), keep, sinks, recent)
    torch.cuda.synchronize()
    fa.check_device_error()
    assert torch.equal(wd.cpu(), w) or torch.isnan(w).any()
    kept, new_w = kept.cpu(), new_w.cpu()
    cap = table.shape[1] * page
    want_k, want_v = k0.clone(), v0.clone()
    for b in range(B):
        n = min(max(int(n0[b]), 0), cap)
        assert int(new_lens[b]) == min(n, keep)
        for h in range(Hkv):
            idx = ref.survivors(w[b, h].numpy(), n, keep, sinks, recent)
            assert kept[b, h].tolist() == idx + [-1] * (keep - len(idx)), (b, h)
            np.testing.assert_array_equal(new_w[b, h, : len(idx)].numpy(), w[b, h, idx].numpy())
            assert not new_w[b, h, len(idx):].any()
            src = torch.tensor(idx, dtype=torch.long)
            to = torch.arange(len(idx))
            t, d = table[b].long(), dst[b].long()
            want_k[d[to // page], to % page, h] = k0[t[src // page], src % page, h]
            want_v[d[to // page], to % page, h] = v0[t[src // page], src % page, h]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


CASES = [
    # B, Hkv, D, dtype, page, lens, keep, sinks, recent
    (1, 1, 64, "fp16", 16, [1], 1, 0, 0),
    (1, 2, 128, "bf16", 16, [40], 40, 4, 10),            # just as long as the budget
    (3, 2, 64, "bf16", 32, [41, 0, 500], 40, 4, 10),
    (2, 4, 128, "fp16", 64, [1000, 999], 300, 0, 0),
    (2, 1, 64, "fp16", 128, [700, 129], 128, 28, 100),   # nothing left to choose
    (1, 8, 128, "bf16", 16, [5000], 1, 0, 0),
    (1, 2, 64, "fp16", 256, [3000], 2999, 1, 2000),
    (2, 2, 128, "bf16", 16, [33, 4097], 32, 32, 0),
]


@pytest.mark.parametrize("B,Hkv,D,dtype,page,lens,keep,sinks,recent", CASES)
def test_evict(cuda_lib, B, Hkv, D, dtype, page, lens, keep, sinks, recent):
    check(*setup(B, Hkv, D, dtype, page, lens, keep, seed=keep + D), keep, sinks, recent)


def test_ties_zeros_and_odd_values(cuda_lib):
    k, v, table, dst, lens, w = setup(2, 3, 64, "bf16", 16, [900, 600], 200, 7)
    w[0, 0] = 1.0                                          # all equal
    w[0, 1] = torch.where(torch.arange(w.shape[2]) % 3 == 0, 0.0, -0.0)
    w[0, 2, ::5] = float("nan")
    w[0, 2, 1::7] = float("inf")
    w[1, 0] = -w[1, 0]
    w[1, 1] = torch.randint(0, 3, w.shape[2:]).float()     # few values, many ties
    w[1, 2, 100:] = 2.0 ** -140                            # subnormal
    check(k, v, table, dst, lens, w, 200, 4, 50)


def test_longer_than_shared_memory(cuda_lib):
    """More keys than eight CTAs hold in shared memory."""
    check(*setup(1, 1, 64, "fp16", 256, [420000], 500, 3), 500, 4, 100)


def test_lengths_are_clamped_and_bad_pages_skipped(cuda_lib):
    k, v, table, dst, lens, w = setup(2, 2, 64, "fp16", 16, [64, 64], 32, 2, joint=True)
    lens[0], lens[1] = 10 ** 9, -4
    check(k, v, table, dst, lens, w, 32, 0, 0)
    dst[0, 1] = -1                                         # this page's survivors go nowhere
    lens[0] = 64
    k0 = k.clone()
    kept, _, _ = fa.paged_evict(k, v, table.cuda(), lens.cuda(), w.cuda(), dst.cuda(), 32)
    torch.cuda.synchronize()
    changed = (k != k0).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {int(dst[0, 0])}


def test_shared_prefix_pages_are_left_alone(cuda_lib):
    k, v, table, dst, lens, w = setup(2, 2, 128, "bf16", 16, [300, 300], 100, 4)
    table[1, :8] = table[0, :8]
    check(k, v, table, dst, lens, w, 100, 4, 20)


def test_prompt_decode_evict_decode(cuda_lib):
    """The run: a prompt and its key weights, into the cache; a token with weights; eviction; a token
    over the survivors, against the 64-bit reference at every stage."""
    B, L, H, Hkv, D, page, keep, sinks, recent = 2, 300, 8, 2, 128, 32, 120, 4, 40
    q, k, v, _ = make_qkv_kv(B, L + 2, L + 2, H, Hkv, D, "bf16", 11)
    P, P2 = -(-(L + 1) // page), -(-(keep + 1) // page)
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(B * (P + P2), generator=g).view(B, P + P2).to(torch.int32)
    table, dst = order[:, :P].contiguous(), order[:, P:].contiguous()
    kc = torch.full((B * (P + P2), page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    pq, pk, pv = (x[:, :L].contiguous().cuda() for x in (q, k, v))
    _, lse = fa.fwd(pq, pk, pv, True)
    w = torch.zeros(B, Hkv, P * page, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    fa.paged_write(pk, pv, kc, vc, table.cuda(), lens - L, weights=w, new_weights=fa.key_weights(pq, pk, lse, True))
    one = [x[:, L: L + 1].contiguous().cuda() for x in (q, k, v)]
    fa.paged_write(one[1], one[2], kc, vc, table.cuda(), lens, weights=w)
    o, _ = fa.paged_decode(one[0], kc, vc, table.cuda(), lens + 1, weights=w)
    kept, new_lens, new_w = fa.paged_evict(kc, vc, table.cuda(), lens + 1, w, dst.cuda(), keep, sinks, recent)
    two = [x[:, L + 1:].contiguous().cuda() for x in (q, k, v)]
    fa.paged_write(two[1], two[2], kc, vc, dst.cuda(), new_lens, weights=new_w)
    o2, _ = fa.paged_decode(two[0], kc, vc, dst.cuda(), new_lens + 1, weights=new_w)
    torch.cuda.synchronize()
    fa.check_device_error()
    q, k, v = to64(q), to64(k), to64(v)
    O, _, bound = ref.forward(q[:, L: L + 1], k[:, : L + 1], v[:, : L + 1], np.ones((1, L + 1), bool), "bf16")
    within(to64(o), O, bound, "O")
    kept, w, group = kept.cpu().numpy(), w.cpu().numpy(), H // Hkv
    for b in range(B):
        for h in range(Hkv):
            mine = ref.survivors(w[b, h], L + 1, keep, sinks, recent)
            assert kept[b, h].tolist() == mine
            idx = mine + [L + 1]
            total = w[b, h, mine].astype(np.float64)
            for x in range(h * group, (h + 1) * group):
                args = (q[b, L + 1:, x], k[b, idx, h], np.ones((1, len(idx)), bool))
                r, _, e = ref.unit_forward(args[0], args[1], v[b, idx, h], args[2], "bf16")
                within(to64(o2)[b, :, x], r, e, "O over the survivors")
                P_ = ref.unit(*args)[0][0]
                total = total + P_[:-1]
            got = to64(new_w)[b, h, :keep]
            within(got, total, 2.0 ** -12 * total + 1e-7, "weights over the survivors")


def test_captured(cuda_lib):
    keep, sinks, recent = 64, 4, 16
    k, v, table, dst, lens, w = setup(2, 2, 64, "fp16", 16, [300, 200], keep, 1)
    t, d, n, wd = table.cuda(), dst.cuda(), lens.cuda(), w.cuda()
    fa.paged_evict(k, v, t, n, wd, d, keep, sinks, recent)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, new_lens, _ = fa.paged_evict(k, v, t, n, wd, d, keep, sinks, recent)
    for seed, ln in ((5, [299, 40]), (6, [77, 200])):
        w2 = torch.exp(torch.randn(w.shape, generator=torch.Generator().manual_seed(seed)))
        wd.copy_(w2)
        n.copy_(torch.tensor(ln, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            for h in range(2):
                idx = ref.survivors(w2[b, h].numpy(), ln[b], keep, sinks, recent)
                assert kept[b, h].tolist() == idx + [-1] * (keep - len(idx))


def test_refusals(cuda_lib):
    k, v, table, dst, lens, w = setup(2, 2, 64, "fp16", 16, [64, 64], 32, 2)
    t, d, n, wd = table.cuda(), dst.cuda(), lens.cuda(), w.cuda()
    for args in ((32, -1, 0), (32, 20, 13), (33, 0, 0)):
        with pytest.raises(_lib.FAError) as e:
            fa.paged_evict(k, v, t, n, wd, d, *args)
        assert e.value.status == _lib.FA_ERR_INVALID_ARG
    with pytest.raises(_lib.FAError):
        fa.paged_evict(k, v, t, n, wd, t, 32)              # into the pages it reads
    with pytest.raises(ValueError):
        fa.paged_evict(k, v, t, n, wd, d, 0)
    with pytest.raises(ValueError):
        fa.paged_evict(k, v, t, n, wd[:, :, :20].contiguous(), d, 32)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n,B,Hkv", [(4097, 1, 1), (9000, 2, 2), (33000, 1, 1), (20000, 40, 8)])
def test_clusters_of_every_size(cuda_lib, n, B, Hkv):
    """One CTA to eight per pair, shares that end in the middle of a warp's, ties across shares."""
    k, v, table, dst, lens, w = setup(B, Hkv, 64, "bf16", 256, [n - 37 * b for b in range(B)], 300, n)
    w[0, 0] = (w[0, 0] * 4).round()
    w[-1, -1] = torch.randint(0, 2, w.shape[2:], generator=torch.Generator().manual_seed(1)).float()
    check(k, v, table, dst, lens, w, 300, 4, 30)


@pytest.mark.parametrize("n,B,Hkv,keep", [(600, 3, 8, 200), (33000, 1, 2, 500), (20000, 40, 8, 300)])
def test_lengths_cut_in_place(cuda_lib, n, B, Hkv, keep):
    """new_lens = lens, every head and CTA of a sequence still choosing from its whole length; and a
    second call on what the first one left (all survive)."""
    lens = [max(n - 977 * b, 50) for b in range(B)]
    k, v, table, dst, ln, w = setup(B, Hkv, 64, "bf16", 256, lens, keep, n)
    n_d, wd = ln.cuda(), w.cuda()
    for _ in range(5):
        n_d.copy_(ln)
        kept, out, new_w = fa.paged_evict(k, v, table.cuda(), n_d, wd, dst.cuda(), keep, 4, 30, new_lens=n_d)
        assert out.data_ptr() == n_d.data_ptr()
        torch.cuda.synchronize()
        assert n_d.tolist() == [min(x, keep) for x in lens]
        got = kept.cpu()
        for b in range(B):
            for h in range(Hkv):
                idx = ref.survivors(w[b, h].numpy(), lens[b], keep, 4, 30)
                assert got[b, h].tolist() == idx + [-1] * (keep - len(idx)), (b, h)
                np.testing.assert_array_equal(new_w[b, h, : len(idx)].cpu().numpy(), w[b, h, idx].numpy())
    kept, _, _ = fa.paged_evict(k, v, table.cuda(), n_d, wd, dst.cuda(), keep, 4, 30, new_lens=n_d)
    assert (kept[0, :, : min(lens[0], keep)].cpu() == torch.arange(min(lens[0], keep))).all()


def test_outputs_on_inputs_are_refused(cuda_lib):
    k, v, table, dst, lens, w = setup(2, 2, 64, "fp16", 16, [64, 64], 32, 2)
    t, d, n = table.cuda(), dst.cuda(), lens.cuda()
    wd = torch.rand(2, 2, 64, device="cuda")
    for kw in (dict(new_weights=wd.flatten()[:128].view(2, 2, 32)),
               dict(kept=wd.flatten()[128:].view(torch.int32).view(2, 2, 32))):
        with pytest.raises(_lib.FAError) as e:
            fa.paged_evict(k, v, t, n, wd, d, 32, **kw)
        assert e.value.status == _lib.FA_ERR_INVALID_ARG
    torch.cuda.synchronize()


@pytest.mark.parametrize("n,B,Hkv,sinks,recent", [(9000, 2, 2, 100, 200), (33000, 1, 1, 300, 0), (33000, 3, 2, 0, 300)])
def test_clusters_with_nothing_to_choose(cuda_lib, n, B, Hkv, sinks, recent):
    """keep = sinks + recent over several CTAs per pair: their counts are exchanged without any pass
    over the weights before."""
    check(*setup(B, Hkv, 64, "bf16", 256, [n - 1500 * b for b in range(B)], 300, n), sinks + recent, sinks, recent)
