"""The paged key/value cache and its eviction on torch tensors.

These calls run once per generated token and layer; their argument checks,
output allocations and the call of the C entry point are one C++ function each
(``csrc/binding.cpp``).  TypeError and ValueError name the argument that does
not fit; what the library refuses raises ``FAError``.
"""

from __future__ import annotations

from . import _lib


def _raise_on(fn: str, r):
    """Outputs pass through; a status becomes an error."""
    if r.__class__ is int:
        _lib.check(fn, r)
    return r


def paged_write(k, v, k_cache, v_cache, block_table, start, counts=None, weights=None,
                new_weights=None, stream=None) -> None:
    """Write new keys and values k, v [B, L, Hkv, D] into the pages of
    k_cache, v_cache [pages, page, Hkv, D]: token j of sequence b goes to
    position start[b] + j, in page block_table[b, position // page].
    block_table [B, P], start [B] and counts [B] (tokens of each sequence that
    count, all L when None) are int32.  ``weights`` [B, Hkv, >= P * page] fp32
    gets ``new_weights`` [B, Hkv, L] (or 0) at the positions written."""
    _raise_on("fa_paged_write", _lib.binding().paged_write(
        k, v, k_cache, v_cache, block_table, start, counts, weights, new_weights, stream))


def paged_decode_workspace_size(B: int, Lq: int, H: int, Hkv: int, D: int, page: int, max_pages: int,
                                weights: bool = False) -> int:
    """Bytes of the workspace ``paged_decode`` needs on the current device."""
    return int(_lib.load().fa_paged_decode_workspace_size(B, Lq, H, Hkv, D, page, max_pages,
                                                          int(weights)))


def paged_decode(q, k_cache, v_cache, block_table, lens, window: int = 0, sinks: int = 0,
                 weights=None, out=None, lse=None, workspace=None, stream=None):
    """O, LSE of the last Lq tokens of every sequence, q [B, Lq, H, D], over
    its keys and values in the pages of k_cache, v_cache [pages, page, Hkv, D].
    block_table [B, P] and lens [B] are int32; lens counts all keys, the new
    tokens' own included: query i sits at position a = lens[b] - Lq + i and
    sees key j iff j <= a and (window == 0 or j > a - window or j < sinks).  A
    query that sees nothing gives O = 0, LSE = -inf.  (H / Hkv) * Lq <= 128.
    ``weights`` [B, Hkv, >= P * page] fp32 is added to in place: each key's
    attention weight over the queries and the group's heads.  ``workspace`` (a
    CUDA byte tensor of at least ``paged_decode_workspace_size`` bytes) is
    allocated when not given."""
    return _raise_on("fa_paged_decode", _lib.binding().paged_decode(
        q, k_cache, v_cache, block_table, lens, window, sinks, weights, out, lse, workspace, stream))


def paged_append(q, k, v, k_cache, v_cache, block_table, start, table, positions=None, counts=None,
                 interleaved: bool = False, weights=None, new_weights=None, out=None, stream=None):
    """``rope_fwd`` of the queries and ``paged_write`` of the turned keys and
    the values in one pass.  q [B, L, H, D], k, v [B, L, Hkv, D], with any
    strides between tokens and batch entries (parts of a fused projection);
    k_cache, v_cache, block_table, start, counts, weights and new_weights as
    for ``paged_write``, ``table`` (from ``rope_table``), ``positions``
    [axes, B, L] int32 and ``interleaved`` as for ``rope_fwd``, except that
    without positions a token's is its slot, start[b] + j.  Returns the turned
    queries, of every token, counted or not (``out`` may be q itself)."""
    return _raise_on("fa_paged_append", _lib.binding().paged_append(
        q, k, v, k_cache, v_cache, block_table, start, table, positions, counts, interleaved, weights, new_weights,
        out, stream))


def paged_prefix_decode_workspace_size(B: int, Lq: int, H: int, Hkv: int, D: int, page: int, groups: int,
                                       prefix_pages: int, max_pages: int) -> int:
    """Bytes of the workspace ``paged_prefix_decode`` needs on the current device."""
    return int(_lib.load().fa_paged_prefix_decode_workspace_size(B, Lq, H, Hkv, D, page, groups, prefix_pages,
                                                                 max_pages))


def paged_prefix_decode(q, k_cache, v_cache, prefix_table, prefix_lens, block_table, lens, group_starts=None,
                        out=None, lse=None, workspace=None, stream=None):
    """``paged_decode`` for sequences that share key/value prefixes, each
    prefix read once for every two tiles of 128 / (H / Hkv) tokens of its
    sequences, not once a sequence.  O, LSE of the last Lq tokens of every
    sequence, q [B, Lq, H, D].  Group i is the sequences group_starts[i] up to
    group_starts[i + 1] (int32 [G + 1], never falling; None with one group: all
    of them), its prefix the first prefix_lens[i] keys in the pages of
    prefix_table [G, PP]; block_table [B, P] and lens [B] are the sequences'
    own keys behind it, the new tokens' included.  Query i of sequence b sees
    its group's prefix and its own keys j <= lens[b] - Lq + i; where that is
    negative (an unused slot) O = 0, LSE = -inf.  (H / Hkv) * Lq <= 128.
    ``workspace`` (a CUDA byte tensor of at least
    ``paged_prefix_decode_workspace_size`` bytes) is allocated when not
    given."""
    return _raise_on("fa_paged_prefix_decode", _lib.binding().paged_prefix_decode(
        q, k_cache, v_cache, prefix_table, prefix_lens, block_table, lens, group_starts, out, lse, workspace, stream))


def paged_evict(k_cache, v_cache, block_table, lens, weights, dst_table, keep: int, sinks: int = 0,
                recent: int = 0, kept=None, new_lens=None, new_weights=None, stream=None):
    """Cut every sequence's paged keys and values down to ``keep`` per K/V
    head: its first ``sinks``, its last ``recent`` and the heaviest others by
    ``weights`` [B, Hkv, >= P * page] fp32 (ties to the lower position).  The
    survivors move, in their order, into the pages of dst_table [B, P2] int32
    (P2 * page >= keep), which no sequence of the call may read from; the old
    pages stay as they are.
    Returns kept [B, Hkv, keep] int32 (old positions, -1 behind the last),
    new_lens [B] int32 = min(lens, keep) and new_weights [B, Hkv, P2 * page]
    (zero behind the survivors).  ``new_lens`` may be ``lens`` itself; the other
    outputs must not share memory with the inputs."""
    return _raise_on("fa_paged_evict", _lib.binding().paged_evict(
        k_cache, v_cache, block_table, lens, weights, dst_table, keep, sinks, recent, kept, new_lens,
        new_weights, stream))


def key_weights_workspace_size() -> int:
    """Bytes of the workspace ``key_weights`` needs on the current device."""
    return int(_lib.load().fa_key_weights_workspace_size())


def key_weights(q, k, lse, causal: bool = False, window: int = 0, sinks: int = 0, out=None,
                workspace=None, stream=None):
    """The attention each key has received: W [B, Hkv, Lk] fp32, the sum over
    the group's heads and the queries of exp(q . k / sqrt(D) - LSE), where
    ``lse`` [B, H, Lq] is what ``fwd`` or (window > 0, causal) ``window_fwd``
    gave for q [B, Lq, H, D] and k [B, Lk, Hkv, D] under the same mask.
    ``workspace`` (a CUDA byte tensor of at least
    ``key_weights_workspace_size`` bytes) is allocated when not given."""
    return _raise_on("fa_key_weights", _lib.binding().key_weights(
        q, k, lse, causal, window, sinks, out, workspace, stream))
