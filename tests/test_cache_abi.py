"""Host-side checks of the window and paged-cache entry points (no GPU): every bad argument is
refused before anything reaches the device."""

import os

import pytest

from tiled_attention_fa_gb300 import _lib

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from tiled_attention_fa_gb300 import build
        build.build(quiet=True)
    return _lib.load()


def caller(fn, names, good):
    def call(**kw):
        a = list(good)
        for key, val in kw.items():
            a[names.index(key)] = val
        return fn(*a, None)
    return call


INVALID, UNSUPPORTED, SMALL = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED, _lib.FA_ERR_SCRATCH_TOO_SMALL


def test_window(lib):
    fwd = caller(lib.fa_window_fwd, "Q K V O LSE B Lq Lk H Hkv D window sinks dtype".split(),
                 [FAKE] * 5 + [1, 100, 200, 4, 2, 64, 50, 4, 0])
    bwd = caller(lib.fa_window_bwd, "Q K V dO LSE Delta dQ dK dV acc bytes zero B Lq Lk H Hkv D window sinks dtype".split(),
                 [FAKE] * 10 + [1 << 40, 1, 1, 100, 200, 4, 2, 64, 50, 4, 0])
    for call in (fwd, bwd):
        for kw in (dict(Q=None), dict(K=FAKE + 8), dict(LSE=None), dict(window=0), dict(sinks=-1), dict(Lk=99),
                   dict(H=3), dict(B=0)):
            assert call(**kw) == INVALID, kw
        assert call(D=96) == UNSUPPORTED and call(dtype=5) == UNSUPPORTED
    assert bwd(acc=None) == INVALID and bwd(dK=None) == INVALID
    size = lib.fa_window_bwd_workspace_size
    assert size(1, 100, 200, 4, 2, 64, 50, 0) == lib.fa_bwd_workspace_size(1, 100, 4, 64)
    need = size(1, 1000, 1000, 4, 2, 64, 50, 4)
    assert need > lib.fa_bwd_workspace_size(1, 1000, 4, 64) and bwd(Lq=1000, Lk=1000, bytes=need - 1) == SMALL
    assert size(1, 100, 99, 4, 2, 64, 50, 0) == 0 and size(1, 100, 100, 4, 2, 64, 0, 0) == 0


def test_paged_decode(lib):
    names = ("Q K V kst vst table lens O LSE w wst ws ws_bytes B Lq H Hkv D page max_pages num_pages window sinks "
             "dtype").split()
    call = caller(lib.fa_paged_decode, names,
                  [FAKE, FAKE, FAKE, 16 * 2 * 64, 16 * 2 * 64, FAKE, FAKE, FAKE, FAKE, None, 0, FAKE, 1 << 40, 2, 1, 4,
                   2, 64, 16, 10, 30, 0, 0, 0])
    for kw in (dict(Q=None), dict(V=FAKE + 8), dict(table=None), dict(lens=FAKE + 2), dict(O=None), dict(ws=None),
               dict(kst=16 * 2 * 64 - 8), dict(vst=16 * 2 * 64 + 4), dict(window=-1), dict(sinks=-1), dict(max_pages=0),
               dict(num_pages=0), dict(H=5), dict(B=0), dict(w=FAKE, wst=100), dict(w=FAKE + 4, wst=160),
               dict(max_pages=1 << 30)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=80), dict(dtype=2), dict(page=24), dict(page=8), dict(Lq=65)):
        kw = dict(kw, kst=1 << 20, vst=1 << 20)
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws_bytes=0) == SMALL
    size = lib.fa_paged_decode_workspace_size
    assert size(2, 1, 4, 2, 64, 16, 10, 1) - size(2, 1, 4, 2, 64, 16, 10, 0) == 2 * 2 * 2 * 2 * 128 * 4
    assert size(0, 1, 4, 2, 64, 16, 10, 0) == 0 and size(2, 1, 4, 2, 80, 16, 10, 0) == 0
    assert size(2, 65, 4, 2, 64, 16, 10, 0) == 0


def test_paged_write(lib):
    names = "K V kc vc kst vst table start counts w wst nw B L Hkv D page max_pages num_pages dtype".split()
    call = caller(lib.fa_paged_write, names,
                  [FAKE] * 4 + [2048, 2048, FAKE, FAKE, None, None, 0, None, 2, 7, 2, 64, 16, 10, 30, 0])
    for kw in (dict(K=None), dict(vc=FAKE + 8), dict(start=None), dict(counts=FAKE + 1), dict(nw=FAKE), dict(w=FAKE, wst=5),
               dict(kst=2040), dict(L=0), dict(max_pages=0)):
        assert call(**kw) == INVALID, kw
    assert call(D=96, kst=1 << 20, vst=1 << 20) == UNSUPPORTED and call(page=17) == UNSUPPORTED


def test_paged_write_weights_share_no_memory(lib):
    """weights rows of 160, new_weights [2, 2, 7]; every call below is refused."""
    M = 1 << 20
    names = "K V kc vc kst vst table start counts w wst nw B L Hkv D page max_pages num_pages dtype".split()
    call = caller(lib.fa_paged_write, names, [M, 2 * M, 3 * M, 4 * M, 2048, 2048, 5 * M, 6 * M, None, 7 * M, 160, 8 * M, 2, 7, 2,
                                              64, 16, 10, 30, 0])
    for kw in (dict(nw=7 * M), dict(nw=7 * M + 636 * 4), dict(nw=7 * M - 24 * 4), dict(w=8 * M), dict(wst=1 << 40)):
        assert call(**kw) == INVALID, kw


def test_key_weights(lib):
    names = "Q K LSE W ws ws_bytes B Lq Lk H Hkv D causal window sinks dtype".split()
    call = caller(lib.fa_key_weights, names, [FAKE] * 5 + [1 << 30, 1, 50, 70, 4, 2, 64, 1, 0, 0, 0])
    for kw in (dict(Q=None), dict(W=FAKE + 4), dict(ws=None), dict(Lk=49), dict(window=-1), dict(sinks=-1),
               dict(window=5, causal=0), dict(H=3)):
        assert call(**kw) == INVALID, kw
    assert call(D=32) == UNSUPPORTED and call(dtype=9) == UNSUPPORTED
    assert call(ws_bytes=0) == SMALL and lib.fa_key_weights_workspace_size() > 0


def test_key_weights_steps_fit_an_int(lib):
    """2^46 steps of 128 x 128 over at most 2^10 SMs: a CTA's share would not fit its counter."""
    L = 1 << 30
    assert lib.fa_key_weights(FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, 1, L, L, 1, 1, 64, 0, 0, 0, 0, None) == UNSUPPORTED


def test_paged_evict(lib):
    names = ("K V kst vst table lens w wst dst keep sinks recent kept new_lens nw B Hkv D page max_pages dst_pages "
             "num_pages dtype").split()
    call = caller(lib.fa_paged_evict, names,
                  [FAKE, FAKE, 2048, 2048, FAKE, FAKE, FAKE, 160, FAKE + 64, 32, 4, 8, FAKE, FAKE, FAKE, 2, 2, 64, 16, 10,
                   2, 30, 0])
    for kw in (dict(K=None), dict(table=None), dict(w=None), dict(w=FAKE + 4), dict(wst=159), dict(dst=None),
               dict(dst=FAKE), dict(keep=0), dict(keep=33), dict(sinks=-1), dict(recent=-1), dict(recent=29), dict(kept=None),
               dict(new_lens=None), dict(nw=None), dict(dst_pages=0), dict(kst=2040)):
        assert call(**kw) == INVALID, kw
    assert call(D=32) == UNSUPPORTED and call(page=48, kst=1 << 20, vst=1 << 20) == UNSUPPORTED
    assert call(B=1 << 15, Hkv=2) == UNSUPPORTED


def test_paged_evict_outputs_share_no_memory(lib):
    """Outputs on inputs or on one another (B 2, Hkv 2, tables of 10 and 2 pages of 16, rows of 160).
    Every call below is refused; none may reach a device, the buffers are not there."""
    M = 1 << 20
    kv, table, lens, w, dst, kept, new_lens, nw = (x * M for x in range(1, 9))
    names = ("K V kst vst table lens w wst dst keep sinks recent kept new_lens nw B Hkv D page max_pages dst_pages "
             "num_pages dtype").split()
    call = caller(lib.fa_paged_evict, names,
                  [kv, kv, 2048, 2048, table, lens, w, 160, dst, 32, 4, 8, kept, new_lens, nw, 2, 2, 64, 16, 10, 2, 30, 0])
    for kw in (dict(nw=w), dict(nw=w + 639 * 4 // 16 * 16), dict(nw=w - 127 * 4 // 16 * 16), dict(w=nw), dict(kept=lens),
               dict(kept=table + 19 * 4), dict(kept=dst - 127 * 4), dict(kept=w), dict(new_lens=table), dict(new_lens=dst + 12),
               dict(new_lens=lens + 4), dict(new_lens=lens - 4), dict(new_lens=kept), dict(new_lens=nw + 127 * 4),
               dict(kept=nw), dict(nw=kept + 127 * 4 // 16 * 16), dict(new_lens=w + 639 * 4), dict(new_lens=lens, nw=w),
               dict(wst=1 << 40)):
        assert call(**kw) == INVALID, kw


@pytest.mark.parametrize("B,L,H,Hkv,D,window,sinks", [
    (4, 8192, 32, 8, 128, 64, 8192),            # every key a sink: causal
    (1, 32768, 8, 8, 128, 64, 32704),           # nothing hidden: causal
    (1, 131072, 32, 8, 128, 128, 4096),
    (1, 1 << 20, 8, 8, 64, 1, 1 << 19),         # 4,096 sink tiles of up to 8,191 far Q tiles
    (2, 4096, 8, 8, 128, 64, 4),
])
def test_window_backward_workspace_is_bounded(lib, B, L, H, Hkv, D, window, sinks):
    """Beyond the dQ accumulator: two fp32 parts of dK and dV a sink tile, or eight units an SM of at
    most 256; nothing where no key is hidden."""
    extra = lib.fa_window_bwd_workspace_size(B, L, L, H, Hkv, D, window, sinks) - lib.fa_bwd_workspace_size(B, L, H, D)
    if window + sinks >= L:
        assert extra == 0
    else:
        tiles = B * Hkv * -(-sinks // 128)
        assert 0 < extra <= (2 * tiles + 8 * 256) * 2 * min(sinks, 128) * D * 4


def test_tensors_on_the_host_are_refused(lib):
    """The calls on torch tensors check their arguments before they touch the device."""
    import torch

    import tiled_attention_fa_gb300 as fa
    q, kv = torch.zeros(1, 2, 4, 64, dtype=torch.float16), torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    i = torch.zeros(1, 3, dtype=torch.int32)
    for call in (lambda: fa.window_fwd(q, q, q, 4), lambda: fa.window_attention_backward(q, q, q, q, q, q, 4),
                 lambda: fa.window_bwd(q, q, q, q, q, q, 4), lambda: fa.paged_decode(q, kv, kv, i, i),
                 lambda: fa.paged_write(q, q, kv, kv, i, i), lambda: fa.key_weights(q, q, q),
                 lambda: fa.paged_evict(kv, kv, i, i, q, i, 4), lambda: fa.paged_decode(None, kv, kv, i, i),
                 lambda: fa.key_weights([1.0], q, q)):
        with pytest.raises(TypeError):
            call()


def test_window_workspace_is_sized_on_its_device(lib, monkeypatch):
    """How the work is cut depends on the SMs of the device that runs the call."""
    import contextlib

    import torch

    import tiled_attention_fa_gb300 as fa
    from tiled_attention_fa_gb300 import api
    current = []

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "window_workspace_size", lambda *a: 4000 if current == ["cpu"] else 16)
    assert fa.alloc_window_workspace(1, 9, 9, 1, 1, 64, 4, 0, "cpu").numel() == 1000
