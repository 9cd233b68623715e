"""Rotary positions on torch tensors: queries and keys (and their gradients)
turned by their positions, on one axis or several."""

from __future__ import annotations

import math

import torch

from .cache import _raise_on
from . import _lib


def _pi(bits: int) -> int:
    """pi 2^bits, less than 1 off (Machin: pi = 16 atan(1/5) - 4 atan(1/239), with 32 bits more)."""
    def atan_inverse(x):
        term = total = (1 << bits + 32) // x
        n, sign = 1, 1
        while term:
            term //= x * x
            n, sign = n + 2, -sign
            total += sign * (term // n)
        return total
    return (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> 32


def _turns(f: float) -> int:
    """f / (2 pi) modulo 1 as a fraction of 2^56.  Up to a radian the quotient of doubles, at most
    2^-55.4 off.  Above, where it is off by 2^-53 of its whole turns and 2^31 positions multiply
    that, in integers, rounded once."""
    if abs(f) <= 1.0:
        return round(f / (2 * math.pi) * 2.0 ** 56) % 2 ** 56
    n, d = f.as_integer_ratio()
    bits = 128 + math.frexp(f)[1]
    d *= 2 * _pi(bits)
    return (2 * (n << bits + 56) + d) // (2 * d) % 2 ** 56


def rope_table(head_dim: int, base: float = 10000.0, rotary=None, sections=None, axes=None, freqs=None,
               device="cuda"):
    """The frequencies and axes of a head's pairs, for ``rope_fwd``,
    ``rope_bwd`` and ``paged_append``: an int64 tensor [rotary / 2], made once.

    The first ``rotary`` dims of a head (a multiple of 16; all ``head_dim``
    when None) are turned.  Pair i turns by ``freqs``[i] radians a position, or
    base^(-2i / rotary).  Its axis, the row of the positions that counts for
    it, is 0, or follows from ``sections`` (how many pairs in a row each axis
    has, [16, 24, 24] for time, height and width of 64 pairs) or is ``axes``[i].
    The angles of these calls are within 2^-21 rad of frequency times position
    at every int32 position, whatever the frequencies."""
    rotary = head_dim if rotary is None else int(rotary)
    n = rotary // 2
    if rotary < 16 or rotary > head_dim or rotary % 16:
        raise ValueError(f"rotary = {rotary} is not a multiple of 16 in [16, {head_dim}]")
    if sections is not None and axes is not None:
        raise ValueError("sections or axes, not both")
    if sections is not None:
        if any(int(c) < 0 for c in sections) or sum(int(c) for c in sections) != n:
            raise ValueError(f"sections {list(sections)} do not add up to {n} pairs")
        axes = [a for a, c in enumerate(sections) for _ in range(int(c))]
    axes = [0] * n if axes is None else [int(a) for a in axes]
    if len(axes) != n or any(not 0 <= a < 256 for a in axes):
        raise ValueError(f"axes must be {n} numbers in [0, 256)")
    if freqs is None:
        if not base > 0 or not math.isfinite(base):
            raise ValueError(f"base = {base} is not positive")
        freqs = [base ** (-2.0 * i / rotary) for i in range(n)]
    freqs = [float(f) for f in freqs]
    if len(freqs) != n or not all(math.isfinite(f) for f in freqs):
        raise ValueError(f"freqs must be {n} finite numbers")
    # Turns a position adds; positions are whole, so whole turns do not count.
    words = [(_turns(f) << 8) | a for f, a in zip(freqs, axes)]
    return torch.tensor([w - 2 ** 64 if w >> 63 else w for w in words], dtype=torch.int64, device=device)


def rope_fwd(q, k, table, positions=None, interleaved: bool = False, out_q=None, out_k=None, stream=None):
    """q [B, L, H, D] and k [B, L, Hkv, D] (or None) turned by their
    positions: pair i (x, y) of a head becomes (x cos t - y sin t,
    x sin t + y cos t), t the token's position on the pair's axis times its
    frequency.  Pairs are dims i and i + rotary / 2, or 2i and 2i + 1 when
    ``interleaved``; ``table`` comes from ``rope_table``.  ``positions``
    [axes, B, L] int32, any values; None: 0 .. L - 1 on one axis.  Inputs and
    outputs may have any strides (multiples of 8) between tokens and batch
    entries; an output may be its input.  Returns the turned q and k."""
    return _raise_on("fa_rope", _lib.binding().rope(q, k, table, positions, interleaved, False, out_q, out_k, stream))


def rope_bwd(dq, dk, table, positions=None, interleaved: bool = False, out_q=None, out_k=None, stream=None):
    """The gradients of ``rope_fwd``'s inputs from those of its outputs (the
    turn by the opposite angles), with the same arguments."""
    return _raise_on("fa_rope", _lib.binding().rope(dq, dk, table, positions, interleaved, True, out_q, out_k, stream))
