"""Pools and weight rows whose offsets pass 32 bits."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_window import within

pytestmark = pytest.mark.gpu


def test_pools_beyond_32_bits(cuda_lib):
    """2^32 elements and more in each pool: written, decoded and evicted at their far end, beside pages at
    the near end that an offset cut to 32 bits would hit."""
    page, Hkv, D, pages, n = 256, 8, 128, 17000, 1000
    assert pages * page * Hkv * D > 2 ** 32 + 2 ** 27
    k, v = (torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    near = pages - 2 ** 32 // (page * Hkv * D)
    k[: near + 1] = 9.0
    v[: near + 1] = 9.0
    table = torch.tensor([[pages - 1, pages - 3, pages - 2, pages - 5]], dtype=torch.int32, device="cuda")
    dst = torch.tensor([[pages - 6]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(0)
    nk, nv = (torch.randn(1, n, Hkv, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1, 1, 16, D, generator=g).bfloat16()
    w = torch.zeros(1, Hkv, 1024, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    fa.paged_write(nk.cuda(), nv.cuda(), k, v, table, lens - n)
    o, _ = fa.paged_decode(q.cuda(), k, v, table, lens, weights=w)
    kept, new_lens, _ = fa.paged_evict(k, v, table, lens, w, dst, 200, 4, 20)
    torch.cuda.synchronize()
    fa.check_device_error()
    O, _, bound = ref.forward(to64(q), to64(nk), to64(nv), np.ones((1, n), bool), "bf16")
    within(to64(o), O, bound, "O")
    assert (k[: near + 1] == 9).all() and (v[: near + 1] == 9).all() and new_lens.tolist() == [200]
    for h in range(Hkv):
        idx = kept[0, h].long().cpu()
        assert idx.tolist() == ref.survivors(w[0, h].cpu().numpy(), n, 200, 4, 20)
        assert torch.equal(k[pages - 6, :200, h].cpu(), nk[0, idx, h]) and torch.equal(v[pages - 6, :200, h].cpu(), nv[0, idx, h])


def test_weight_rows_beyond_32_bits(cuda_lib):
    """Weights [70, 2, 2^25]: the last rows lie past 2^32 elements."""
    B, Hkv, D, page, cap, n = 70, 2, 64, 16, 128, 100
    w = torch.zeros(B, Hkv, 2 ** 25, device="cuda")
    assert w.numel() > 2 ** 32
    P = cap // page
    k, v = (torch.randn(B * P, page, Hkv, D, device="cuda").half() for _ in range(2))
    table = torch.randperm(B * P, device="cuda").int().view(B, P)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(B, 1, 4, D, device="cuda").half()
    fa.paged_decode(q, k, v, table, lens, weights=w)
    small = torch.zeros(B, Hkv, cap, device="cuda")
    fa.paged_decode(q, k, v, table, lens, weights=small)
    torch.cuda.synchronize()
    fa.check_device_error()
    assert torch.equal(w[:, :, :cap], small) and not w[:, :, cap:cap + 4096].any()
    assert ((small.sum(2) - 2).abs() < 2 * 2 * ref.FP32).all()      # two heads' weights of one query each
