"""Frequencies of more than a turn a position at the far end of int32, where a table that is off shows."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests.helpers import to64
from tests.test_rope_table_exact import turns

pytestmark = pytest.mark.gpu


def near_whole(f, count):
    """Positions near 2^31 at which f comes within 2^-14 of a whole number of turns, and how far."""
    step = round(turns(f) * 2 ** 120)
    found = []
    for n in range(2 ** 31 - 1, 0, -1):
        r = (n * step + 2 ** 119) % 2 ** 120 - 2 ** 119
        if abs(r) < 2 ** 106:
            found.append((n, float(Fraction(r, 2 ** 120))))
            if len(found) == count:
                return found


def test_far_turns(cuda_lib):
    """(1, 0) turned by t is (cos t, sin t), and a small sin t keeps its bits in 16."""
    freqs, L, D = [6.9, -12.9, 100.1, 1000.7, 43.21, 7.77, -300.3, 25.6], 4, 64
    n = len(freqs)
    found = [near_whole(f, L) for f in freqs]
    pos = torch.tensor([[p for p, _ in x] for x in found], dtype=torch.int32).view(n, 1, L).cuda()
    q = torch.zeros(1, L, 1, D, dtype=torch.float16)
    q[..., :n] = 1.0
    y, _ = fa.rope_fwd(q.cuda(), None, fa.rope_table(D, rotary=2 * n, freqs=freqs, axes=list(range(n)), device="cuda"), pos)
    y = to64(y)[0, :, 0]
    want = np.sin(2 * math.pi * np.array([[t for _, t in x] for x in found]).T)
    # The table's half step of 2^-57 times 2^31 positions and the cut to 32 bits, in radians; sin in
    # fp32 (2^-20 relative is ample); half a step of fp16, 2^-25 at least.
    bound = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32) + np.abs(want) * (2.0 ** -11 + 2.0 ** -20) + 2.0 ** -25
    assert (np.abs(y[:, n: 2 * n] - want) <= bound).all()
    assert (np.abs(y[:, :n] - 1) <= 2.0 ** -20).all() and (y[:, 2 * n:] == 0).all()
