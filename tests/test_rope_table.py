"""The table of frequencies and axes, and what the rotary, append and shared-prefix calls refuse
(no GPU)."""

import math
import os

import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests.test_cache_abi import INVALID, SMALL, UNSUPPORTED, caller
from tiled_attention_fa_gb300 import _lib

M = 1 << 20  # apart buffers at M, 2M, ...: never dereferenced, every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from tiled_attention_fa_gb300 import build
        build.build(quiet=True)
    return _lib.load()


def test_table():
    t = fa.rope_table(128, base=500000.0, sections=[16, 24, 24], device="cpu")
    assert t.dtype == torch.int64 and t.shape == (64,)
    words = [int(w) & (2 ** 64 - 1) for w in t]
    assert [w & 255 for w in words] == [0] * 16 + [1] * 24 + [2] * 24
    for i, w in enumerate(words):
        turns = 500000.0 ** (-2 * i / 128) / (2 * math.pi)
        assert abs((w >> 8) / 2.0 ** 56 - turns) <= 2.0 ** -53 * turns + 2.0 ** -57
    # backwards, more than a turn a position, axes one by one, part of a head
    t = fa.rope_table(64, rotary=16, freqs=[-1.0, 2 * math.pi + 0.5] + [0.0] * 6, axes=[1, 0] * 4, device="cpu")
    words = [int(w) & (2 ** 64 - 1) for w in t]
    assert [w & 255 for w in words] == [1, 0] * 4
    assert abs((words[0] >> 8) / 2.0 ** 56 - (1 - 1 / (2 * math.pi))) < 2.0 ** -50
    assert abs((words[1] >> 8) / 2.0 ** 56 - 0.5 / (2 * math.pi)) < 2.0 ** -50
    assert all(w >> 8 == 0 for w in words[2:])


@pytest.mark.parametrize("kw", [dict(rotary=24), dict(rotary=144), dict(rotary=0), dict(sections=[30, 30]),
                                dict(sections=[70, -6]), dict(sections=[64], axes=[0] * 64), dict(axes=[0] * 63),
                                dict(axes=[256] * 64), dict(base=0.0), dict(base=float("inf")), dict(freqs=[1.0] * 63),
                                dict(freqs=[float("nan")] * 64)])
def test_table_refusals(kw):
    with pytest.raises(ValueError):
        fa.rope_table(128, device="cpu", **kw)


def test_rope(lib):
    names = ("Q qb qt K kb kt Qo qob qot Ko kob kot table pos axes B L H Hkv D rotary inter back dtype").split()
    call = caller(lib.fa_rope, names, [M, 7 * 256, 256, 2 * M, 7 * 128, 128, 3 * M, 7 * 256, 256, 4 * M, 7 * 128, 128,
                                       5 * M, 6 * M, 2, 2, 7, 4, 2, 64, 64, 0, 0, 0])
    for kw in (dict(Q=None), dict(Q=M + 2), dict(K=None), dict(Ko=None), dict(Qo=None), dict(table=None), dict(table=M + 8),
               dict(pos=None), dict(pos=6 * M + 2), dict(axes=0), dict(axes=257), dict(B=0), dict(L=0), dict(H=0), dict(Hkv=-1),
               dict(Hkv=0), dict(Hkv=1 << 21), dict(qt=252), dict(qb=-8), dict(kt=-128), dict(qot=248), dict(qob=6 * 256),
               dict(kot=0), dict(kob=0), dict(Q=3 * M + 16), dict(Q=3 * M, qt=264), dict(Qo=M + 7 * 256 * 2 * 2 - 16),
               dict(Ko=2 * M + 16), dict(qb=1 << 38)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=96), dict(dtype=2), dict(rotary=8), dict(rotary=72), dict(rotary=80), dict(rotary=0)):
        assert call(**kw) == UNSUPPORTED, kw


def test_paged_append(lib):
    names = ("Q qb qt K kb kt V vb vt Qo qob qot kc vc kst vst bt start counts table pos axes w wst nw B L H Hkv D rotary inter "
             "page max_pages num_pages dtype").split()
    call = caller(lib.fa_paged_append, names,
                  [M, 7 * 256, 256, 2 * M, 7 * 128, 128, 3 * M, 7 * 128, 128, 4 * M, 7 * 256, 256, 5 * M, 6 * M, 2048, 2048,
                   7 * M, 8 * M, None, 9 * M, None, 1, None, 0, None, 2, 7, 4, 2, 64, 64, 0, 16, 10, 30, 0])
    for kw in (dict(Q=None), dict(K=None), dict(V=3 * M + 8), dict(Qo=None), dict(kc=None), dict(vc=6 * M + 4), dict(bt=None),
               dict(start=8 * M + 1), dict(counts=7), dict(table=None), dict(axes=2), dict(pos=3), dict(kst=2040),
               dict(nw=10 * M), dict(w=10 * M, wst=100), dict(w=10 * M, wst=160, nw=10 * M), dict(Hkv=0), dict(H=5),
               dict(L=0), dict(max_pages=0), dict(num_pages=0), dict(vt=4), dict(Qo=M + 16), dict(qot=128)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(page=24), dict(rotary=40), dict(D=80)):
        assert call(**dict(kw, kst=1 << 20, vst=1 << 20)) == UNSUPPORTED, kw


def test_paged_prefix_decode(lib):
    names = ("Q K V kst vst ptable plens starts bt lens O LSE ws ws_bytes B Lq H Hkv D page groups pp max_pages num_pages "
             "dtype").split()
    call = caller(lib.fa_paged_prefix_decode, names,
                  [M, 2 * M, 3 * M, 2048, 2048, 4 * M, 5 * M, 6 * M, 7 * M, 8 * M, 9 * M, 10 * M, 11 * M, 1 << 40, 5, 1, 4, 2, 64,
                   16, 2, 20, 10, 200, 0])
    for kw in (dict(Q=None), dict(K=2 * M + 8), dict(V=None), dict(kst=2040), dict(vst=2052), dict(ptable=None),
               dict(plens=5 * M + 2), dict(starts=None), dict(starts=6 * M + 1), dict(bt=None), dict(lens=None), dict(O=None),
               dict(LSE=10 * M + 4), dict(ws=None), dict(B=0), dict(Lq=0), dict(H=5), dict(groups=0), dict(groups=1 << 21),
               dict(pp=0), dict(max_pages=0), dict(num_pages=0), dict(pp=1 << 30)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=80), dict(dtype=2), dict(page=24), dict(Lq=65)):
        assert call(**dict(kw, kst=1 << 20, vst=1 << 20)) == UNSUPPORTED, kw
    # 2^31 units of 128 keys
    assert call(B=1 << 12, Hkv=64, H=64, kst=1 << 20, vst=1 << 20, page=16, pp=1 << 26) == UNSUPPORTED
    assert call(ws_bytes=64) == SMALL
    size = lib.fa_paged_prefix_decode_workspace_size
    sizes = [5, 1, 4, 2, 64, 16, 2, 20, 10]
    assert size(*sizes) > lib.fa_paged_decode_workspace_size(5, 1, 4, 2, 64, 16, 10, 0)
    for i, bad in ((0, 0), (1, 65), (2, 5), (4, 80), (5, 20), (6, 0), (7, 0), (8, 0)):
        assert size(*(bad if x == i else v for x, v in enumerate(sizes))) == 0


def test_tensors_on_the_host_are_refused(lib):
    q, kv = torch.zeros(1, 2, 4, 64, dtype=torch.float16), torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    i, t = torch.zeros(1, 3, dtype=torch.int32), fa.rope_table(64, device="cpu")
    for call in (lambda: fa.rope_fwd(q, q, t), lambda: fa.rope_bwd(q, None, t), lambda: fa.rope_fwd(None, q, t),
                 lambda: fa.paged_append(q, q, q, kv, kv, i, i, t), lambda: fa.paged_prefix_decode(q, kv, kv, i, i, i, i)):
        with pytest.raises(TypeError):
            call()
