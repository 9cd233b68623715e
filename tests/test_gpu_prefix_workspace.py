"""Partials of prefixes lie at the rows before them, whatever the groups' sizes: nothing is written
outside the workspace, and no two chunks share a row."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_prefix import expected, setup
from tests.test_gpu_window import within

pytestmark = pytest.mark.gpu

CASES = [
    # Lq, H, Hkv, D, dtype, page, plens, sizes, lens
    (1, 32, 8, 128, "bf16", 64, [700, 30, 5000, 1], [33, 1, 2, 70], 9),              # one tile, two and a rest
    (1, 7, 1, 64, "fp16", 16, [900] * 30, [(5 * i) % 7 for i in range(30)], 20),     # 126 rows a tile, empty groups
    (5, 6, 2, 128, "fp16", 32, [3000, 40, 800], [2, 9, 25], 30),                     # 15 rows a sequence
    (8, 16, 4, 64, "bf16", 128, [2500, 2500], [1, 12], 300),                         # 32 rows
    (20, 4, 1, 64, "fp16", 64, [1500, 200], [3, 2], 700),                            # 80 rows: own keys in the list
    (1, 1, 1, 64, "bf16", 16, [40000], [1], 3),                                      # one row in many parts
]


@pytest.mark.parametrize("Lq,H,Hkv,D,dtype,page,plens,sizes,hi", CASES)
def test_inside_the_workspace(cuda_lib, Lq, H, Hkv, D, dtype, page, plens, sizes, hi):
    g = torch.Generator().manual_seed(sum(sizes))
    lens = torch.randint(0, hi + 1, (sum(sizes),), generator=g).tolist()
    args = setup(Lq, H, Hkv, D, dtype, page, plens, sizes, lens, 21)
    n = fa.paged_prefix_decode_workspace_size(len(lens), Lq, H, Hkv, D, page, len(plens), args[3].shape[1], args[5].shape[1])
    guard = 1 << 20
    buf = torch.full((n + 2 * guard,), 255, dtype=torch.uint8, device="cuda")        # (NaN, and no part's number)
    o, lse = fa.paged_prefix_decode(*args, workspace=buf[guard: guard + n])
    torch.cuda.synchronize()
    fa.check_device_error()
    assert (buf[:guard] == 255).all() and (buf[guard + n:] == 255).all()
    O, L, bound = expected(*args, dtype)
    within(to64(o), O, bound, "O")
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(to64(lse)), empty)
    within(np.where(empty, 0, to64(lse)), np.where(empty, 0, L), np.full(L.shape, ref.FP32), "LSE")


def test_a_group_for_every_sequence(cuda_lib):
    """256 sequences, each behind a prefix of its own, in the memory that one group needs and two
    ints a group and head."""
    lens = [1 + (i * 37) % 90 for i in range(256)]
    plens = [(i * 53) % 600 for i in range(256)]
    args = setup(1, 8, 2, 64, "bf16", 32, plens, [1] * 256, lens, 22)
    assert fa.paged_prefix_decode_workspace_size(256, 1, 8, 2, 64, 32, 256, args[3].shape[1], args[5].shape[1]) < 16 << 20
    o, lse = fa.paged_prefix_decode(*args)
    torch.cuda.synchronize()
    fa.check_device_error()
    O, L, bound = expected(*args, "bf16")
    within(to64(o), O, bound, "O")
    within(to64(lse), L, np.full(L.shape, ref.FP32), "LSE")
