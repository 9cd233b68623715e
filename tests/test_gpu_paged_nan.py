"""Paged decoding where a visible key or a query holds NaN: the rows that see it are NaN, in O, in LSE and
in the weights they add; every other row, and every key hidden from them, is as without it."""

import pytest
import torch

import tiled_attention_fa_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Lq,H,Hkv,D,page,n,window", [
    (1, 3, 4, 2, 128, 64, 6000, 0),       # items cut into many parts
    (1, 3, 4, 2, 64, 16, 6000, 700),
    (40, 3, 16, 8, 128, 32, 300, 0),      # items inside one CTA
    (40, 2, 16, 2, 64, 64, 260, 100),
    (2, 32, 8, 2, 128, 64, 1500, 0),      # one softmax group
    (1, 1, 2, 2, 64, 16, 100, 0),
])
def test_nan_reaches_the_rows_that_see_it(cuda_lib, B, Lq, H, Hkv, D, page, n, window):
    g = torch.Generator(device="cuda").manual_seed(n)
    P = -(-n // page)
    k, v = (torch.randn(B * P, page, Hkv, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(B, Lq, H, D, device="cuda", generator=g).bfloat16()
    table = torch.randperm(B * P, device="cuda", generator=g).int().view(B, P)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    w0 = torch.zeros(B, Hkv, P * page, device="cuda")
    w1, w2 = w0.clone(), w0.clone()
    o0, lse0 = fa.paged_decode(q, k, v, table, lens, window, weights=w0)
    # the last key of sequence 0, K/V head 1: seen by the last query's heads of that group alone
    k[table[0, (n - 1) // page].long(), (n - 1) % page, 1, 3] = float("nan")
    o1, lse1 = fa.paged_decode(q, k, v, table, lens, window, weights=w1)
    # an early key, before every window
    k[table[0, 0].long(), 1, 0] = float("nan")
    o2, lse2 = fa.paged_decode(q, k, v, table, lens, window, weights=w2)
    torch.cuda.synchronize()
    fa.check_device_error()
    grp = H // Hkv
    bad = torch.zeros(B, Lq, H, dtype=torch.bool, device="cuda")
    bad[0, -1, grp: 2 * grp] = True
    assert torch.isnan(o1[bad]).all() and torch.isnan(lse1.transpose(1, 2)[bad]).all()
    assert torch.equal(o1[~bad], o0[~bad]) and torch.equal(lse1.transpose(1, 2)[~bad], lse0.transpose(1, 2)[~bad])
    last = torch.arange(P * page, device="cuda")
    seen = (last < n) & ((last > n - 1 - window) if window else True)   # by the last query
    assert torch.isnan(w1[0, 1, seen]).all()
    keep = torch.ones(B, Hkv, P * page, dtype=torch.bool, device="cuda")
    keep[0, 1, seen] = False
    assert torch.equal(w1[keep], w0[keep])
    if window:
        assert torch.equal(torch.nan_to_num(o2, 7.0), torch.nan_to_num(o1, 7.0))
        assert torch.equal(torch.nan_to_num(w2, 7.0), torch.nan_to_num(w1, 7.0))
    else:
        bad[0, :, :grp] = True
        assert torch.isnan(o2[bad]).all() and torch.isnan(lse2.transpose(1, 2)[bad]).all()
        assert torch.equal(o2[~bad], o0[~bad])


def test_a_query_of_nan(cuda_lib):
    q = torch.randn(2, 2, 4, 64, device="cuda").half()
    k, v = (torch.randn(20, 16, 2, 64, device="cuda").half() for _ in range(2))
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    lens = torch.tensor([160, 37], dtype=torch.int32, device="cuda")
    o0, lse0 = fa.paged_decode(q, k, v, table, lens)
    q[1, 0, 2] = float("nan")
    o, lse = fa.paged_decode(q, k, v, table, lens)
    torch.cuda.synchronize()
    bad = torch.zeros(2, 2, 4, dtype=torch.bool, device="cuda")
    bad[1, 0, 2] = True
    assert torch.isnan(o[bad]).all() and torch.isnan(lse.transpose(1, 2)[bad]).all()
    assert torch.equal(o[~bad], o0[~bad]) and torch.equal(lse.transpose(1, 2)[~bad], lse0.transpose(1, 2)[~bad])
