"""Paged decoding under a window: the width of the table changes nothing."""

import pytest
import torch

import tiled_attention_fa_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Lq,H,Hkv,D,window,sinks,n", [(16, 8, 1, 128, 4096, 4, 6000), (1, 4, 1, 64, 1000, 0, 8000),
                                                       (4, 16, 2, 128, 700, 300, 5000)])
def test_windowed_results_do_not_depend_on_the_width(cuda_lib, Lq, H, Hkv, D, window, sinks, n):
    """Bit for bit: an item is cut by what its window lets it visit, not by what the table could hold."""
    page, P = 64, 128
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn(P, page, Hkv, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1, Lq, H, D, device="cuda", generator=g).bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    narrow = torch.randperm(P, device="cuda", generator=g).int().view(1, P)
    wide = torch.full((1, 16 * P), -1, dtype=torch.int32, device="cuda")
    wide[:, :P] = narrow
    a = fa.paged_decode(q, k, v, narrow, lens, window, sinks)
    b = fa.paged_decode(q, k, v, wide, lens, window, sinks)
    torch.cuda.synchronize()
    fa.check_device_error()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
