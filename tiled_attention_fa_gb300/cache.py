"""Python binding of the paged key/value cache and its eviction: argument
marshalling only, like ``api``.

These calls run once per generated token and layer, so the checks are written
for their cost on the host: one expression per tensor, and sizes of workspaces
remembered per shape (a pure function of the shape and the device).
"""

from __future__ import annotations

import functools

import torch

from . import _lib
from .api import _device, _dtype_code, _nbytes, _need, _ptr, _stream, _want

_F32, _I32 = torch.float32, torch.int32


def _pools(k_cache, v_cache, dtype, device: int):
    """(num_pages, page, Hkv, D) and the page strides in elements of two pools
    whose pages may lie apart but are contiguous in themselves (halves of one
    tensor, for instance)."""
    try:
        shape = k_cache.shape
        pages, page, hkv, d = shape
        inner = (hkv * d, d, 1)
        ks, vs = k_cache.stride(), v_cache.stride()
        if (k_cache.dtype is dtype and v_cache.dtype is dtype and v_cache.shape == shape
                and ks[1:] == inner and vs[1:] == inner and k_cache.is_cuda and v_cache.is_cuda
                and k_cache.get_device() == device and v_cache.get_device() == device):
            if pages == 1:
                return pages, page, hkv, d, page * hkv * d, page * hkv * d
            return pages, page, hkv, d, ks[0], vs[0]
    except (AttributeError, ValueError):
        pass
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.dim() != 4 or t.shape != k_cache.shape:
            raise ValueError(f"{name} must be [pages, page, Hkv, D], both pools alike")
        if t.get_device() != device:
            raise ValueError(f"{name} lies on cuda:{t.get_device()}, the current device is "
                             f"cuda:{device}")
    raise ValueError("the pages of k_cache and v_cache must be contiguous")


def _row_stride(weights, name: str, B: int, Hkv: int, cap: int, device: int) -> int:
    """Elements between the rows of key weights [B, Hkv, >= cap] fp32."""
    _need(weights, name, dtype=_F32)
    if weights.dim() != 3 or weights.shape[:2] != (B, Hkv) or weights.shape[2] < cap:
        raise ValueError(f"{name} has shape {tuple(weights.shape)}, expected ({B}, {Hkv}, >= {cap})")
    _want(weights, name, weights.shape, _F32, device)
    return weights.shape[2]


def paged_write(k, v, k_cache, v_cache, block_table, start, counts=None, weights=None,
                new_weights=None, stream=None) -> None:
    """Write new keys and values k, v [B, L, Hkv, D] into the pages of
    k_cache, v_cache [pages, page, Hkv, D]: token j of sequence b goes to
    position start[b] + j, in page block_table[b, position // page].
    block_table [B, P], start [B] and counts [B] (tokens of each sequence that
    count, all L when None) are int32.  ``weights`` [B, Hkv, >= P * page] fp32
    gets ``new_weights`` [B, Hkv, L] (or 0) at the positions written."""
    dt, dev = k.dtype, _device()
    pages, page, Hkv, D, kst, vst = _pools(k_cache, v_cache, dt, dev)
    B, L = k.shape[:2]
    P = block_table.shape[-1]
    _want(k, "k", (B, L, Hkv, D), dt, dev)
    _want(v, "v", (B, L, Hkv, D), dt, dev)
    _want(block_table, "block_table", (B, P), _I32, dev)
    _want(start, "start", (B,), _I32, dev)
    if counts is not None:
        _want(counts, "counts", (B,), _I32, dev)
    wst = 0
    if weights is not None:
        wst = _row_stride(weights, "weights", B, Hkv, P * page, dev)
    if new_weights is not None:
        _want(new_weights, "new_weights", (B, Hkv, L), _F32, dev)
    st = _lib.load().fa_paged_write(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kst, vst,
        block_table.data_ptr(), start.data_ptr(), _ptr(counts), _ptr(weights), wst,
        _ptr(new_weights), B, L, Hkv, D, page, P, pages, _dtype_code(k), _stream(stream))
    if st:
        _lib.check("fa_paged_write", st)


@functools.lru_cache(maxsize=1024)
def _decode_ws(device, *sizes) -> int:
    return int(_lib.load().fa_paged_decode_workspace_size(*sizes))


def paged_decode_workspace_size(B: int, Lq: int, H: int, Hkv: int, D: int, page: int, max_pages: int,
                                weights: bool = False) -> int:
    """Bytes of the workspace ``paged_decode`` needs on the current device."""
    return _decode_ws(_device(), B, Lq, H, Hkv, D, page, max_pages, int(weights))


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
    dt, dev = q.dtype, _device()
    pages, page, Hkv, D, kst, vst = _pools(k_cache, v_cache, dt, dev)
    B, Lq, H, _ = q.shape
    P = block_table.shape[-1]
    _want(q, "q", (B, Lq, H, D), dt, dev)
    _want(block_table, "block_table", (B, P), _I32, dev)
    _want(lens, "lens", (B,), _I32, dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want(out, "out", (B, Lq, H, D), dt, dev)
    if lse is None:
        lse = q.new_empty((B, H, Lq), dtype=_F32)
    else:
        _want(lse, "lse", (B, H, Lq), _F32, dev)
    wst, wp = 0, None
    if weights is not None:
        wst, wp = _row_stride(weights, "weights", B, Hkv, P * page, dev), weights.data_ptr()
    if workspace is None:
        n = _decode_ws(dev, B, Lq, H, Hkv, D, page, P, int(wp is not None))
        workspace = q.new_empty(max(n, 16), dtype=torch.uint8)
    else:
        n = _nbytes(workspace)
        _want(workspace, "workspace", workspace.shape, workspace.dtype, dev)
    st = _lib.load().fa_paged_decode(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kst, vst, block_table.data_ptr(),
        lens.data_ptr(), out.data_ptr(), lse.data_ptr(), wp, wst, workspace.data_ptr(), n, B, Lq, H,
        Hkv, D, page, P, pages, window, sinks, _dtype_code(q), _stream(stream))
    if st:
        _lib.check("fa_paged_decode", st)
    return out, lse


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
    (zero behind the survivors)."""
    dt, dev = k_cache.dtype, _device()
    pages, page, Hkv, D, kst, vst = _pools(k_cache, v_cache, dt, dev)
    B, P = block_table.shape
    P2 = dst_table.shape[-1]
    _want(block_table, "block_table", (B, P), _I32, dev)
    _want(lens, "lens", (B,), _I32, dev)
    _want(dst_table, "dst_table", (B, P2), _I32, dev)
    wst = _row_stride(weights, "weights", B, Hkv, P * page, dev)
    if keep < 1:
        raise ValueError("keep must be at least 1")
    if kept is None:
        kept = lens.new_empty((B, Hkv, keep))
    else:
        _want(kept, "kept", (B, Hkv, keep), _I32, dev)
    if new_lens is None:
        new_lens = torch.empty_like(lens)
    else:
        _want(new_lens, "new_lens", (B,), _I32, dev)
    if new_weights is None:
        new_weights = weights.new_empty((B, Hkv, P2 * page))
    else:
        _want(new_weights, "new_weights", (B, Hkv, P2 * page), _F32, dev)
    st = _lib.load().fa_paged_evict(
        k_cache.data_ptr(), v_cache.data_ptr(), kst, vst, block_table.data_ptr(), lens.data_ptr(),
        weights.data_ptr(), wst, dst_table.data_ptr(), keep, sinks, recent, kept.data_ptr(),
        new_lens.data_ptr(), new_weights.data_ptr(), B, Hkv, D, page, P, P2, pages,
        _dtype_code(k_cache), _stream(stream))
    if st:
        _lib.check("fa_paged_evict", st)
    return kept, new_lens, new_weights


@functools.lru_cache(maxsize=64)
def _weights_ws(device) -> int:
    return int(_lib.load().fa_key_weights_workspace_size())


def key_weights_workspace_size() -> int:
    """Bytes of the workspace ``key_weights`` needs on the current device."""
    return _weights_ws(_device())


def key_weights(q, k, lse, causal: bool = False, window: int = 0, sinks: int = 0, out=None,
                workspace=None, stream=None):
    """The attention each key has received: W [B, Hkv, Lk] fp32, the sum over
    the group's heads and the queries of exp(q . k / sqrt(D) - LSE), where
    ``lse`` [B, H, Lq] is what ``fwd`` or (window > 0, causal) ``window_fwd``
    gave for q [B, Lq, H, D] and k [B, Lk, Hkv, D] under the same mask.
    ``workspace`` (a CUDA byte tensor of at least
    ``key_weights_workspace_size`` bytes) is allocated when not given."""
    dt, dev = q.dtype, _device()
    B, L, H, D = q.shape
    _, Lk, Hkv, _ = k.shape
    _want(q, "q", (B, L, H, D), dt, dev)
    _want(k, "k", (B, Lk, Hkv, D), dt, dev)
    _want(lse, "lse", (B, H, L), _F32, dev)
    if out is None:
        out = lse.new_empty((B, Hkv, Lk))
    else:
        _want(out, "out", (B, Hkv, Lk), _F32, dev)
    if workspace is None:
        n = _weights_ws(dev)
        workspace = q.new_empty(n, dtype=torch.uint8)
    else:
        n = _nbytes(workspace)
        _want(workspace, "workspace", workspace.shape, workspace.dtype, dev)
    st = _lib.load().fa_key_weights(
        q.data_ptr(), k.data_ptr(), lse.data_ptr(), out.data_ptr(), workspace.data_ptr(), n, B, L, Lk,
        H, Hkv, D, 1 if causal else 0, window, sinks, _dtype_code(q), _stream(stream))
    if st:
        _lib.check("fa_key_weights", st)
    return out
