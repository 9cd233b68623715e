"""The rotary calls through the C entry points, on a stream of the caller's."""

import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tiled_attention_fa_gb300 import _lib

pytestmark = pytest.mark.gpu


def test_rope_on_a_stream(cuda_lib):
    B, L, H, Hkv, D = 2, 33, 4, 2, 64
    q, k = (torch.randn(B, L, h, D, generator=torch.Generator().manual_seed(h)).half().cuda() for h in (H, Hkv))
    table, side = fa.rope_table(D), torch.cuda.Stream()
    want = fa.rope_fwd(q, k, table)
    out = [torch.empty_like(x) for x in (q, k)]
    torch.cuda.synchronize()
    row = lambda x: (x.stride(0), x.stride(1))  # noqa: E731
    st = _lib.load().fa_rope(q.data_ptr(), *row(q), k.data_ptr(), *row(k), out[0].data_ptr(), *row(out[0]), out[1].data_ptr(),
                             *row(out[1]), table.data_ptr(), None, 1, B, L, H, Hkv, D, D, 0, 0, _lib.FA_F16, side.cuda_stream)
    assert st == _lib.FA_OK
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
