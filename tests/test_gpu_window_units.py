"""The window backward's units: long runs of K/V tiles that no query sees."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_window import within
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import make_qkv_kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,dtype,window,sinks,cut", [
    (2, 130, 16384, 8, 8, 64, "fp16", 700, 4, False),       # 2064 units, 112 of 128 tiles a head unseen
    (4, 256, 8192, 8, 8, 128, "bf16", 1024, 4, False),      # 2080 units, 53 of 64
    (1, 200, 40000, 4, 4, 64, "bf16", 100, 0, False),       # 1252 units, three tiles of 313 seen
    (1, 1024, 10240, 32, 2, 128, "bf16", 1024, 4, True),    # cut by heads: zeros in fp32 parts, 648 units
    (1, 1024, 10240, 32, 2, 64, "fp16", 1024, 4, True),
])
def test_many_units_that_no_query_sees(cuda_lib, B, Lq, Lk, H, Hkv, D, dtype, window, sinks, cut):
    """A CTA's units are mostly K/V tiles that no query sees, several in a row with seen ones behind
    them.  (They once went through the pipeline, where nothing held the MMA warp back while the
    compute warps still stored the zeros of the one before.)"""
    q, k, v, do = make_qkv_kv(B, Lq, Lk, H, Hkv, D, dtype, Lk + D, with_do=True)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.window_fwd(*dev[:3], window, sinks)
    parts = fa.window_workspace_size(B, Lq, Lk, H, Hkv, D, window, sinks) - _lib.load().fa_bwd_workspace_size(B, Lq, H, D)
    assert (parts >= 2 * B * Hkv * (Lk // 128) * 2 * 128 * D * 4) == cut
    for _ in range(3):
        dk, dv = (torch.full_like(dev[1], 7.0) for _ in range(2))
        delta = fa.bwd_preprocess(o, dev[3])
        dq, dk, dv = fa.window_bwd(*dev[:3], dev[3], lse, delta, window, sinks, dk=dk, dv=dv)
        torch.cuda.synchronize()
        fa.check_device_error()
        mask = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks)
        seen = torch.from_numpy(mask.any(axis=0))
        unseen = (~seen).cuda()
        assert not dk[:, unseen].any() and not dv[:, unseen].any()
    got = [to64(x) for x in (dq, dk[:, ~unseen], dv[:, ~unseen])]
    want = ref.backward(to64(q), to64(k[:, seen]), to64(v[:, seen]), to64(do), mask[:, seen.numpy()], dtype)
    for name, g, r, e in zip(("dQ", "dK", "dV"), got, *want):
        within(g, r, e, name)


@pytest.mark.parametrize("D,dtype,window,sinks", [(64, "fp16", 1, 1000), (128, "bf16", 100, 1152), (64, "bf16", 300, 129)])
def test_many_far_units(cuda_lib, D, dtype, window, sinks):
    """Sink tiles whose later queries make more units than are worth their parts: longer units."""
    B, L, H, Hkv = 2, 2304, 8, 8
    q, k, v, do = make_qkv_kv(B, L, L, H, Hkv, D, dtype, sinks, with_do=True)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.window_fwd(*dev[:3], window, sinks)
    grads = fa.window_attention_backward(*dev[:3], o, lse, dev[3], window, sinks)[:3]
    torch.cuda.synchronize()
    fa.check_device_error()
    mask = ref.seen(np.arange(L), L, window, sinks)
    for name, g, r, e in zip(("dQ", "dK", "dV"), grads, *ref.backward(*(to64(x) for x in (q, k, v, do)), mask, dtype)):
        within(to64(g), r, e, name)


@pytest.mark.parametrize("window,sinks", [(200, 500), (200, 499), (1, 699), (1, 698)])
def test_hiding_no_key_or_one(cuda_lib, window, sinks):
    """sinks + window reaches the length (plain causal) or misses it by one key."""
    L, D, dtype = 700, 64, "fp16"
    q, k, v, do = make_qkv_kv(1, L, L, 4, 2, D, dtype, sinks, with_do=True)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.window_fwd(*dev[:3], window, sinks)
    grads = fa.window_attention_backward(*dev[:3], o, lse, dev[3], window, sinks)[:3]
    torch.cuda.synchronize()
    fa.check_device_error()
    mask = ref.seen(np.arange(L), L, window, sinks)
    assert (~np.tril(mask) & np.tril(np.ones((L, L), bool))).sum() == max(0, L - window - sinks)
    for name, g, r, e in zip(("dQ", "dK", "dV"), grads, *ref.backward(*(to64(x) for x in (q, k, v, do)), mask, dtype)):
        within(to64(g), r, e, name)
