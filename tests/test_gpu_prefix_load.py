"""Decoding behind shared prefixes while other work runs on the GPU: the same bits in every call, O and
LSE, wherever its CTAs come to lie and in whatever order they end."""

import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests.test_gpu_prefix import setup

pytestmark = pytest.mark.gpu

CASES = [
    # Lq, H, Hkv, D, page, plens, sizes, longest own
    (1, 32, 8, 128, 64, [9000], [64], 700),                  # both kinds of CTAs
    (4, 32, 8, 128, 16, [3001], [20], 500),                  # 16 rows, two tiles and a half
    (8, 16, 4, 128, 128, [5000, 300], [12, 5], 900),         # 32 rows
    (16, 16, 4, 128, 64, [4000], [10], 600),                 # 64 rows: own keys in the prefixes' list
    (1, 16, 16, 64, 32, [4000, 1500, 700], [20, 9, 11], 400),
]


def inputs(i):
    Lq, H, Hkv, D, page, plens, sizes, hi = CASES[i]
    g = torch.Generator().manual_seed(i)
    lens = torch.randint(Lq, hi + 1, (sum(sizes),), generator=g).tolist()
    return setup(Lq, H, Hkv, D, "bf16", page, plens, sizes, lens, 30 + i)


def same(got, want):
    return torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("i", range(len(CASES)))
def test_beside_products_and_copies(cuda_lib, i):
    args = inputs(i)
    want = fa.paged_prefix_decode(*args)
    a = torch.randn(3000, 3000, device="cuda").bfloat16()
    src, dst = (torch.empty(1 << 27, dtype=torch.uint8, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    products, copies = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for n in range(40):
        with torch.cuda.stream(products):
            for _ in range(1 + n % 3):
                torch.matmul(a[: 500 + 60 * n], a)
        with torch.cuda.stream(copies):
            dst[: (n % 7 + 1) << 23].copy_(src[: (n % 7 + 1) << 23])
        outs.append(fa.paged_prefix_decode(*args))
    torch.cuda.synchronize()
    fa.check_device_error()
    assert not [n for n, o in enumerate(outs) if not same(o, want)]


def test_beside_one_another(cuda_lib):
    """All cases at once, a stream each, none waiting for another."""
    cases = [inputs(i) for i in range(len(CASES))]
    want = [fa.paged_prefix_decode(*a) for a in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(15):
        for s, a, g in zip(streams, cases, got):
            with torch.cuda.stream(s):
                g.append(fa.paged_prefix_decode(*a))
    torch.cuda.synchronize()
    fa.check_device_error()
    for w, g in zip(want, got):
        assert all(same(o, w) for o in g)
