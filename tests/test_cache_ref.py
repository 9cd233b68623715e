"""The 64-bit references of the window, paged-cache and eviction operators, pinned on the CPU:
against straight loops, the library oracle's plain attention, and differences."""

import numpy as np
import pytest

from oracle import fa_oracle as orc
from tests import cache_ref as ref


def rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("Lq,Lk,window,sinks", [(5, 5, 2, 0), (4, 9, 3, 2), (3, 7, 1, 0), (6, 6, 50, 1), (2, 8, 2, 8)])
def test_window_mask_by_definition(Lq, Lk, window, sinks):
    m = ref.seen(np.arange(Lk - Lq, Lk), Lk, window, sinks)
    for i in range(Lq):
        a = i + Lk - Lq
        for j in range(Lk):
            assert m[i, j] == (j <= a and (j > a - window or j < sinks))
    assert m.any(axis=1).all()


def test_a_window_of_every_key_is_causal_attention():
    q, k, v = rand(1, 6, 4, 8), rand(1, 9, 2, 8, seed=1), rand(1, 9, 2, 8, seed=2)
    O, lse, _ = ref.forward(q, k, v, ref.seen(np.arange(3, 9), 9, 9, 0), "bf16")
    ro, rl = orc.forward(q, k, v, True)
    np.testing.assert_allclose(O, ro, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, rl, rtol=1e-12, atol=1e-12)


def test_backward_against_differences():
    q, k, v, do = (rand(1, n, h, 4, seed=s) for s, (n, h) in enumerate([(5, 4), (7, 2), (7, 2), (5, 4)]))
    mask = ref.seen(np.arange(2, 7), 7, 3, 1)
    grads, _ = ref.backward(q, k, v, do, mask, "fp16")
    f = lambda a, b, c: float((ref.forward(a, b, c, mask, "fp16")[0] * do).sum())  # noqa: E731
    h = 1e-6
    for which, (x, g) in enumerate(zip((q, k, v), grads)):
        for idx in np.ndindex(*x.shape):
            args = [q.copy(), k.copy(), v.copy()]
            args[which][idx] += h
            up = f(*args)
            args[which][idx] -= 2 * h
            assert abs((up - f(*args)) / (2 * h) - g[idx]) < 1e-7 * max(1, abs(g[idx])) + 1e-8


def test_key_weights_sum_to_the_visible_rows():
    q, k = rand(2, 6, 4, 8), rand(2, 8, 2, 8, seed=1)
    mask = ref.seen(np.arange(2, 8), 8)
    lse = ref.forward(q, k, rand(2, 8, 2, 8, seed=2), mask, "bf16")[1]
    W = ref.key_weights(q, k, lse, mask)
    np.testing.assert_allclose(W.sum(-1), 6 * 2)      # every query of both heads gives 1 in all
    lse[0, 1, 3] = -np.inf                             # an empty row gives nothing
    np.testing.assert_allclose(ref.key_weights(q, k, lse, mask).sum(-1)[0], [11, 12])


def test_paged_decode_of_one_page_order_is_plain_attention():
    kc, vc = rand(6, 4, 2, 8), rand(6, 4, 2, 8, seed=1)
    q = rand(2, 1, 4, 8, seed=2)
    table, lens = np.array([[3, 0, 5], [1, 4, 2]]), np.array([9, 0])
    O, lse, _, W = ref.paged_decode(q, kc, vc, table, lens, "bf16", weights=np.zeros((2, 2, 12)))
    k = np.concatenate([kc[3], kc[0], kc[5]])[None, :9]
    v = np.concatenate([vc[3], vc[0], vc[5]])[None, :9]
    ro, rl = orc.forward(q[:1], k, v, False)
    np.testing.assert_allclose(O[:1], ro, atol=1e-12)
    np.testing.assert_allclose(lse[:1], rl, atol=1e-12)
    assert not O[1].any() and np.isneginf(lse[1]).all()
    np.testing.assert_allclose(W[0].sum(-1), 2.0)      # two heads of each group
    assert not W[0, :, 9:].any() and not W[1].any()


def test_survivors():
    w = np.array([1.0, 5.0, 2.0, 5.0, 0.0, 7.0, 1.0, 0.5])
    assert ref.survivors(w, 8, 4, 1, 2) == [0, 5, 6, 7]
    assert ref.survivors(w, 8, 5, 0, 1) == [1, 2, 3, 5, 7]
    assert ref.survivors(w, 8, 2, 0, 0) == [1, 5]      # 7.0, and the first of the two fives
    assert ref.survivors(w, 3, 4, 1, 2) == [0, 1, 2]
    w[2] = np.nan
    assert ref.survivors(w, 8, 1, 0, 0) == [2]
