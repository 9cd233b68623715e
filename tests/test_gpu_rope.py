"""Rotary positions, forward and backward, against the 64-bit reference (tests/rope_ref.py)."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import rope_ref as ref
from tests.helpers import to64
from tests.test_gpu_window import within
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import storage_dtype

pytestmark = pytest.mark.gpu

BASE = 10000.0


def freqs(rotary):
    return [BASE ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def rand(g, *shape, dt):
    return torch.randn(*shape, generator=g).to(dt)


CASES = [
    # B, L, H, Hkv, D, dtype, rotary, axes, interleaved
    (1, 1, 1, 1, 64, "fp16", 64, 1, False),
    (1, 1, 32, 8, 128, "bf16", 128, 1, False),
    (2, 7, 3, 1, 128, "fp16", 128, 3, False),
    (3, 33, 4, 4, 64, "bf16", 32, 2, True),
    (1, 130, 5, 5, 64, "fp16", 16, 1, True),
    (2, 65, 7, 2, 128, "bf16", 96, 3, False),       # 7 query heads, 2 of keys
    (1, 257, 56, 8, 128, "bf16", 112, 2, True),
    (5, 3, 1, 2, 128, "fp16", 48, 1, False),
    (1, 700, 40, 40, 64, "bf16", 64, 1, False),
]


@pytest.mark.parametrize("B,L,H,Hkv,D,dtype,rotary,axes,inter", CASES)
def test_rope(cuda_lib, B, L, H, Hkv, D, dtype, rotary, axes, inter):
    g = torch.Generator().manual_seed(L + rotary)
    dt = storage_dtype(dtype)
    q, k, dq, dk = (rand(g, B, L, h, D, dt=dt) for h in (H, Hkv, H, Hkv))
    pos = torch.randint(-70000, 200000, (axes, B, L), generator=g, dtype=torch.int32)
    which = torch.randint(0, axes, (rotary // 2,), generator=g).tolist()
    table = fa.rope_table(D, BASE, rotary, axes=which)
    got = [*fa.rope_fwd(q.cuda(), k.cuda(), table, pos.cuda(), inter),
           *fa.rope_bwd(dq.cuda(), dk.cuda(), table, pos.cuda(), inter)]
    torch.cuda.synchronize()
    for name, x, y, sign in zip(("q", "k", "dq", "dk"), (q, k, dq, dk), got, (1, 1, -1, -1)):
        want, bound = ref.turned(to64(x), pos.numpy(), freqs(rotary), which, rotary, inter, dtype, sign)
        within(to64(y), want, bound, name)
        assert torch.equal(y.cpu()[..., rotary:], x[..., rotary:])      # dims that are not turned: copies


def test_far_positions_and_plain_ones(cuda_lib):
    """The ends of int32, and no positions: 0 .. L - 1."""
    g = torch.Generator().manual_seed(1)
    q = rand(g, 1, 6, 2, 128, dt=torch.float16)
    table = fa.rope_table(128)
    pos = torch.tensor([[[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 123456789, -1, 0]]], dtype=torch.int32)
    y, none = fa.rope_fwd(q.cuda(), None, table, pos.cuda())
    assert none is None
    want, bound = ref.turned(to64(q), pos.numpy(), freqs(128), [0] * 64, 128, False, "fp16")
    within(to64(y), want, bound, "q")
    assert torch.equal(y[:, 5].cpu(), q[:, 5])                          # position 0 turns nothing
    y, _ = fa.rope_fwd(q.cuda(), None, table)
    want, bound = ref.turned(to64(q), np.arange(6)[None, None], freqs(128), [0] * 64, 128, False, "fp16")
    within(to64(y), want, bound, "q")


def test_other_frequencies(cuda_lib):
    """Frequencies of one's own, some backwards, some of more than a turn a position."""
    g = torch.Generator().manual_seed(2)
    f = [(-1.0) ** i * 9.0 * 0.7 ** i for i in range(32)]
    q = rand(g, 2, 9, 3, 64, dt=torch.float16)
    pos = torch.randint(-1000, 1000, (1, 2, 9), generator=g, dtype=torch.int32)
    y, _ = fa.rope_fwd(q.cuda(), None, fa.rope_table(64, freqs=f), pos.cuda())
    want, bound = ref.turned(to64(q), pos.numpy(), f, [0] * 32, 64, False, "fp16")
    within(to64(y), want, bound, "q")


def test_strides(cuda_lib):
    """Parts of a fused projection's rows in and out, in place, a repeated input, tokens first."""
    g = torch.Generator().manual_seed(3)
    B, L, H, Hkv, D = 2, 37, 4, 2, 64
    qkv = rand(g, B, L, H + 2 * Hkv, D, dt=torch.bfloat16).cuda()
    table = fa.rope_table(D)
    q, k = qkv[:, :, :H], qkv[:, :, H: H + Hkv]
    want = fa.rope_fwd(q.contiguous(), k.contiguous(), table)
    got = fa.rope_fwd(q, k, table)
    assert all(torch.equal(a, b) and b.is_contiguous() for a, b in zip(want, got))
    other = torch.full_like(qkv, 7.0)
    fa.rope_fwd(q, k, table, out_q=other[:, :, Hkv: H + Hkv], out_k=other[:, :, :Hkv])
    assert torch.equal(other[:, :, Hkv: H + Hkv], want[0]) and torch.equal(other[:, :, :Hkv], want[1])
    assert (other[:, :, H + Hkv:] == 7).all()
    v = qkv[:, :, H + Hkv:].clone()
    fa.rope_fwd(q, k, table, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, H + Hkv:], v)
    one = rand(g, 1, 1, H, D, dt=torch.bfloat16).cuda()
    y, _ = fa.rope_fwd(one.expand(B, L, H, D), None, table)
    assert torch.equal(y, fa.rope_fwd(one.expand(B, L, H, D).contiguous(), None, table)[0])
    t = rand(g, L, B, H, D, dt=torch.bfloat16).cuda().transpose(0, 1)
    out = torch.empty(L, B, H, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    fa.rope_fwd(t, None, table, out_q=out)
    assert torch.equal(out, fa.rope_fwd(t.contiguous(), None, table)[0])


def test_not_numbers_stay_in_their_pair(cuda_lib):
    q = torch.randn(1, 3, 2, 64, generator=torch.Generator().manual_seed(4)).half()
    q[0, 1, 0, 5], q[0, 2, 1, 60] = float("nan"), float("inf")
    table = fa.rope_table(64, rotary=32)
    y = fa.rope_fwd(q.cuda(), None, table)[0].cpu()
    bad = torch.zeros(1, 3, 2, 64, dtype=torch.bool)
    bad[0, 1, 0, 5] = bad[0, 1, 0, 21] = bad[0, 2, 1, 60] = True
    assert torch.equal(~torch.isfinite(y), bad) and torch.isinf(y[0, 2, 1, 60])


def test_backward_is_the_gradient(cuda_lib):
    """Against central differences of the 64-bit form, and back and forth gives the inputs again."""
    g = torch.Generator().manual_seed(5)
    B, L, H, D = 1, 5, 1, 64
    x, dy = (rand(g, B, L, H, D, dt=torch.float16) for _ in range(2))
    pos = torch.randint(0, 5000, (1, B, L), generator=g, dtype=torch.int32)
    table = fa.rope_table(D)
    dx = to64(fa.rope_bwd(dy.cuda(), None, table, pos.cuda())[0])
    f = lambda z: (ref.turned(z, pos.numpy(), freqs(D), [0] * 32, D, False, "fp16")[0] * to64(dy)).sum()  # noqa: E731
    x64 = to64(x)
    for i in range(0, x64.size, 7):
        e = np.zeros(x64.size)
        e[i] = 1.0
        e = e.reshape(x64.shape)
        diff = (f(x64 + e) - f(x64 - e)) / 2                           # (linear: exact at any step)
        # two terms, a rounding each in fp32, the store's half step
        assert abs(dx.ravel()[i] - diff) <= 2.0 ** -11 * abs(diff) + 2.0 ** -18 * np.abs(to64(dy)).max()
    y, _ = fa.rope_fwd(x.cuda(), None, table, pos.cuda())
    back = to64(fa.rope_bwd(y, None, table, pos.cuda())[0])
    # y is off by half a step of each of its pair, which the turn back mixes; then the store
    n = D // 2
    pair = np.abs(x64) + np.abs(np.roll(x64, n, -1))
    within(back, x64, 2.0 ** -11 * (2 * pair) + 2.0 ** -18 * pair + 2.0 ** -11 * np.abs(x64) + 1e-7, "x")


def test_training_step(cuda_lib):
    """As it is used: turned queries and keys into the attention, its gradients turned back; the whole
    against the 64-bit chain of the oracle."""
    from oracle import fa_oracle as orc
    from tests.helpers import assert_close
    g = torch.Generator().manual_seed(6)
    B, L, H, Hkv, D = 1, 150, 4, 2, 64
    q, k, v, do = (rand(g, B, L, h, D, dt=torch.float16) for h in (H, Hkv, Hkv, H))
    pos = torch.randint(0, 4000, (2, B, L), generator=g, dtype=torch.int32)
    which = [0] * 16 + [1] * 16
    table = fa.rope_table(D, sections=[16, 16])
    qr, kr = fa.rope_fwd(q.cuda(), k.cuda(), table, pos.cuda())
    o, lse = fa.fwd(qr, kr, v.cuda(), True)
    grads = fa.attention_backward(qr, kr, v.cuda(), o, lse, do.cuda(), True)
    dq, dk = fa.rope_bwd(grads[0], grads[1], table, pos.cuda())
    torch.cuda.synchronize()
    fa.check_device_error()
    turn = lambda x, s: ref.turned(x, pos.numpy(), freqs(D), which, D, False, "fp16", s)[0]  # noqa: E731
    dq64, dk64, dv64 = orc.backward(turn(to64(q), 1), turn(to64(k), 1), to64(v), to64(do), True)[:3]
    # the attention's own tolerance, and as much again for the turned inputs' rounding
    for name, got, want in (("dq", dq, turn(dq64, -1)), ("dk", dk, turn(dk64, -1)), ("dv", grads[2], dv64)):
        assert_close(to64(got), want, rtol=2e-2, atol=2e-2, name=name)


def test_refusals(cuda_lib):
    table = fa.rope_table(64)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.float16, device="cuda")
    pos = torch.zeros(1, 2, 3, dtype=torch.int32, device="cuda")
    fa.rope_fwd(q, q, table, pos)
    for err, call in (
            (TypeError, lambda: fa.rope_fwd(q.float(), None, table)), (TypeError, lambda: fa.rope_fwd(q, q.bfloat16(), table)),
            (TypeError, lambda: fa.rope_fwd(q, None, table.int())), (TypeError, lambda: fa.rope_fwd(q, None, table.cpu())),
            (TypeError, lambda: fa.rope_fwd(q, None, table, pos.long())), (ValueError, lambda: fa.rope_fwd(q, None, table, pos[0])),
            (ValueError, lambda: fa.rope_fwd(q, None, table, pos[:, :1])), (ValueError, lambda: fa.rope_fwd(q[0], None, table)),
            (ValueError, lambda: fa.rope_fwd(q, q[:1], table)), (ValueError, lambda: fa.rope_fwd(q, None, table, out_k=q)),
            (ValueError, lambda: fa.rope_fwd(q, None, table, out_q=q[:1])),
            (ValueError, lambda: fa.rope_fwd(q.transpose(2, 3), None, table)),
            (ValueError, lambda: fa.rope_fwd(q[:, :, ::2], None, table))):
        with pytest.raises(err):
            call()
    flat = torch.zeros(4096, dtype=torch.float16, device="cuda")
    for bad, call in (
            (_lib.FA_ERR_UNSUPPORTED, lambda: fa.rope_fwd(q, None, table[:12])),                     # 24 dims
            (_lib.FA_ERR_UNSUPPORTED, lambda: fa.rope_fwd(q, None, torch.cat([table, table]))),      # 128 of 64
            (_lib.FA_ERR_INVALID_ARG, lambda: fa.rope_fwd(q, None, table, out_q=q[:1, :1].expand_as(q))),
            (_lib.FA_ERR_INVALID_ARG, lambda: fa.rope_fwd(flat.as_strided((1, 3, 4, 64), (0, 256, 64, 1)), None, table,
                                                          out_q=flat.as_strided((1, 3, 4, 64), (0, 256, 64, 1), 256))),
            (_lib.FA_ERR_INVALID_ARG, lambda: fa.rope_fwd(flat.as_strided((1, 3, 4, 64), (0, 260, 64, 1)), None, table)),
            (_lib.FA_ERR_INVALID_ARG, lambda: fa.rope_fwd(flat[1:769].view(1, 3, 4, 64), None, table))):
        with pytest.raises(_lib.FAError) as e:
            call()
        assert e.value.status == bad
    torch.cuda.synchronize()
