"""Scores that rise from tile to tile, so that every tile moves the maximum and rescales O: one tile of
rows and two, D 64 and 128, own keys in CTAs of their own and in the prefixes' list."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_prefix import expected, setup
from tests.test_gpu_window import within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,B", [(1, 3), (1, 70), (20, 2)])
def test_every_tile_rescales(cuda_lib, D, Lq, B):
    H, Hkv, n, own = 8, 2, 1500, 300
    args = setup(Lq, H, Hkv, D, "fp16", 16, [n], [B], [own] * B, 8 + B)
    q, k, v, ptable, _, table, _, _ = args
    k.zero_(), v.nan_to_num_(), q.zero_()
    q[..., 0] = 8.0
    rise = lambda a, pages: ((a + torch.arange(pages * 16)) / 16.0).view(pages, 16, 1).to(k.dtype).cuda()  # noqa: E731
    k[ptable[0].long(), :, :, 0] = rise(0, ptable.shape[1])
    for b in range(B):
        k[table[b].long(), :, :, 0] = rise(n, table.shape[1])
    o, lse = fa.paged_prefix_decode(*args)
    torch.cuda.synchronize()
    fa.check_device_error()
    O, L, bound = expected(*args, "fp16")
    within(to64(o), O, bound, "O")
    # scores up to 113 (8 x 112.5 / 8), scaled in fp32 (2^-22 relative)
    within(to64(lse), L, ref.FP32 + np.abs(L) * 2.0 ** -20, "LSE")
