"""What the attention behind shared prefixes needs of a workspace (no GPU): rows count, not groups."""

import os

import pytest

from tiled_attention_fa_gb300 import _lib


@pytest.fixture(scope="module")
def size():
    if not os.path.exists(_lib.LIB_PATH):
        from tiled_attention_fa_gb300 import build
        build.build(quiet=True)
    return _lib.load().fa_paged_prefix_decode_workspace_size


@pytest.mark.parametrize("B,Lq,H,Hkv,D", [(256, 1, 32, 8, 128), (256, 4, 32, 8, 64), (1000, 1, 16, 16, 64)])
def test_groups_cost_a_pair_of_ints_a_head(size, B, Lq, H, Hkv, D):
    one = size(B, Lq, H, Hkv, D, 64, 1, 100, 10)
    for groups in (2, B // 2, B, 1 << 15):
        assert size(B, Lq, H, Hkv, D, 64, groups, 100, 10) - one == (groups - 1) * Hkv * 8


def test_a_row_is_there_twice_and_256_for_a_part(size):
    """D floats and an LSE of every query row, in a prefix's partials and in the own keys'."""
    B, Lq, H, Hkv, D = 64, 2, 32, 8, 128
    more = size(2 * B, Lq, H, Hkv, D, 64, 1, 100, 10) - size(B, Lq, H, Hkv, D, 64, 1, 100, 10)
    rows = B * Lq * H
    tiles = B * Lq // 32 // 2
    assert more == 2 * rows * (D + 1) * 4 + (tiles + B) * Hkv * 8
