"""Key weights of a prompt against the 64-bit reference.

A weight is a sum of exp(s - LSE) terms.  Each is off by at most FP32 relative (cache_ref: the fp32
score and the exponential; the LSE argument's own rounding, 2^-24 of at most 16, is inside that), and
the fp32 sums add at most 2^-24 relative per level of adding: FP32 covers both."""

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


def check(B, Lq, Lk, H, Hkv, D, dtype, causal, window, sinks, seed, empty=()):
    q, k, v, _ = make_qkv_kv(B, Lq, Lk, H, Hkv, D, dtype, seed)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    lse = (fa.window_fwd(qd, kd, vd, window, sinks) if window else fa.fwd(qd, kd, vd, causal))[1]
    for e in empty:
        lse[e] = float("-inf")
    out = torch.full((B, Hkv, Lk), float("nan"), device="cuda")
    fa.key_weights(qd, kd, lse, causal, window, sinks, out=out)
    torch.cuda.synchronize()
    fa.check_device_error()
    mask = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks) if causal else np.ones((Lq, Lk), bool)
    W = ref.key_weights(to64(q), to64(k), to64(lse), mask)
    within(to64(out), W, ref.FP32 * W + 1e-30, "W")
    return out


CASES = [
    # B, Lq, Lk, H, Hkv, D, dtype, causal, window, sinks
    (1, 1, 1, 1, 1, 64, "fp16", True, 0, 0),
    (1, 1, 300, 4, 2, 128, "bf16", True, 0, 0),
    (2, 130, 130, 2, 1, 64, "bf16", True, 0, 0),
    (1, 500, 77, 2, 2, 128, "fp16", False, 0, 0),
    (2, 200, 333, 4, 1, 64, "fp16", False, 0, 0),
    (2, 1001, 1001, 8, 2, 64, "fp16", True, 0, 0),
    (1, 700, 1500, 4, 4, 128, "bf16", True, 0, 0),
    (1, 640, 640, 2, 2, 128, "fp16", True, 100, 3),
    (1, 300, 1500, 4, 2, 64, "bf16", True, 128, 0),       # keys that no query sees: 0
    (1, 300, 2000, 2, 1, 128, "bf16", True, 1, 200),
    (1, 900, 900, 2, 1, 64, "fp16", True, 4000, 7),
    (2, 2048, 2048, 16, 4, 128, "bf16", True, 0, 0),      # parts that begin and end inside items
]


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,dtype,causal,window,sinks", CASES)
def test_key_weights(cuda_lib, B, Lq, Lk, H, Hkv, D, dtype, causal, window, sinks):
    check(B, Lq, Lk, H, Hkv, D, dtype, causal, window, sinks, seed=Lq + Lk + D)


def test_empty_rows_add_nothing(cuda_lib):
    out = check(1, 200, 260, 4, 2, 64, "fp16", True, 0, 0, 3, empty=[(0, 1, slice(0, 150)), (0, 2), (0, 3)])
    assert not out[0, 1].any()


def test_the_same_twice(cuda_lib):
    """Sums in a fixed order: bit for bit the same, and the same under a graph and on a stream."""
    q, k, v, _ = make_qkv_kv(1, 1500, 1500, 8, 2, 128, "bf16", 2)
    qd, kd = q.cuda(), k.cuda()
    _, lse = fa.fwd(qd, kd, v.cuda(), True)
    first = fa.key_weights(qd, kd, lse, True)
    for _ in range(5):
        assert torch.equal(fa.key_weights(qd, kd, lse, True), first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(first)
    fa.key_weights(qd, kd, lse, True, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    ws = torch.empty(fa.key_weights_workspace_size(), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.key_weights(qd, kd, lse, True, out=out, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_refusals(cuda_lib):
    q, k, _, _ = make_qkv_kv(1, 8, 8, 2, 2, 64, "fp16", 0)
    q, k, lse = q.cuda(), k.cuda(), torch.zeros(1, 2, 8, device="cuda")
    for args, status in (((False, 4), _lib.FA_ERR_INVALID_ARG), ((True, -1), _lib.FA_ERR_INVALID_ARG),
                         ((True, 4, -1), _lib.FA_ERR_INVALID_ARG)):
        with pytest.raises(_lib.FAError) as e:
            fa.key_weights(q, k, lse, *args)
        assert e.value.status == status
    with pytest.raises(_lib.FAError) as e:
        fa.key_weights(q, k, lse, True, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == _lib.FA_ERR_SCRATCH_TOO_SMALL
    with pytest.raises(ValueError):
        fa.key_weights(q, k, lse[:, :1].contiguous(), True)
