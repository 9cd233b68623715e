"""64-bit references of the window, paged-cache, key-weight and eviction operators, written from
their definitions (numpy, whole score matrices), with element-wise bounds on how far a kernel that
rounds where these kernels round can be from them.

Roundings counted (u = half a step of the 16-bit type, 2^-8 bf16 / 2^-11 fp16):
  P and dS are rounded to the 16-bit type before their products: u relative; in fp16 a value
    below 2^-14 is rounded to a multiple of 2^-24 instead, at most 2^-25 absolute.  Forward P is
    exp(s - m) with m the row max or up to 2^8 below it, so l >= 1 and the absolute part is at
    most 2^-25 per visible key after the division by l.
  O, dQ, dK, dV (and the O behind Delta) are rounded once at the store: u relative.
  fp32 work (scores, exponentials, sums): a score is a sum of at most 128 exact products in fp32,
    off by at most 128 * 2^-24 of sum |q k| / sqrt(D); with |q|, |k| of N(0, 1) entries that sum
    stays below 16, so a probability moves by at most 2^-13 relative.  FP32 = 2^-12 covers that,
    the exponential (2^-22) and the sums (at most 2^16 terms added in blocks).
"""

import numpy as np

U16 = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"fp16": 2.0 ** -25, "bf16": 0.0}
FP32 = 2.0 ** -12


def seen(pos, n, window=0, sinks=0):
    """[len(pos), n] bool: query at position a sees key j iff j <= a and (no window, or
    j > a - window, or j < sinks)."""
    a, j = np.asarray(pos)[:, None], np.arange(n)[None, :]
    m = j <= a
    if window:
        m &= (j > a - window) | (j < sinks)
    return m


def unit(q, k, mask):
    """Probabilities [Lq, Lk] and LSE [Lq] of one head; a row that sees nothing has P = 0, LSE = -inf."""
    s = (q @ k.T) / np.sqrt(q.shape[1])
    s = np.where(mask, s, -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    safe = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - safe[:, None])
    l = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = safe + np.log(l)
    return e / np.where(l > 0, l, 1.0)[:, None], lse


def unit_forward(q, k, v, mask, dt):
    """O, LSE and the bound on O of one head."""
    P, lse = unit(q, k, mask)
    O, pv = P @ v, P @ np.abs(v)
    u = U16[dt]
    bound = (u + FP32) * pv + SUB[dt] * (mask @ np.abs(v)) + u * np.abs(O) + 1e-7
    return O, lse, bound


def forward(q, k, v, mask, dt):
    """BSHD O, LSE [B, H, Lq] and the bound on O; one mask for every head."""
    B, Lq, H, D = q.shape
    g = H // k.shape[2]
    O, bound, lse = np.zeros((B, Lq, H, D)), np.zeros((B, Lq, H, D)), np.zeros((B, H, Lq))
    for b in range(B):
        for h in range(H):
            O[b, :, h], lse[b, h], bound[b, :, h] = unit_forward(q[b, :, h], k[b, :, h // g], v[b, :, h // g], mask, dt)
    return O, lse, bound


def backward(q, k, v, do, mask, dt):
    """(dQ, dK, dV) and their bounds, BSHD, summed over the query heads of a K/V head."""
    B, Lq, H, D = q.shape
    g = H // k.shape[2]
    c = 1 / np.sqrt(D)
    u, sub = U16[dt], SUB[dt]
    out = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    err = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for b in range(B):
        for h in range(H):
            Q, K, V, dO = q[b, :, h], k[b, :, h // g], v[b, :, h // g], do[b, :, h]
            P, _ = unit(Q, K, mask)
            O, pv = P @ V, P @ np.abs(V)
            delta = (O * dO).sum(1)
            dP = dO @ V.T
            dS = P * (dP - delta[:, None])
            e_o = (u + FP32) * pv + sub * (mask @ np.abs(V)) + u * np.abs(O)
            e_d = (np.abs(dO) * e_o).sum(1)
            e_s = (P * (e_d[:, None] + FP32 * (np.abs(dO) @ np.abs(V).T + np.abs(delta)[:, None]))
                   + u * np.abs(dS) + sub * mask)
            e_p = (u + FP32) * P + sub * mask
            out[0][b, :, h] = dS @ K * c
            out[1][b, :, h // g] += dS.T @ Q * c
            out[2][b, :, h // g] += P.T @ dO
            err[0][b, :, h] = e_s @ np.abs(K) * c
            err[1][b, :, h // g] += e_s.T @ np.abs(Q) * c
            err[2][b, :, h // g] += e_p.T @ np.abs(dO)
    return out, [e + u * np.abs(o) + 1e-7 for o, e in zip(out, err)]


def key_weights(q, k, lse, mask):
    """[B, Hkv, Lk]: sum over the group's heads and the queries of exp(s - LSE); a query whose LSE
    is -inf adds nothing."""
    B, Lq, H, D = q.shape
    Hkv = k.shape[2]
    W = np.zeros((B, Hkv, k.shape[1]))
    for b in range(B):
        for h in range(H):
            kh = h * Hkv // H
            s = (q[b, :, h] @ k[b, :, kh].T) / np.sqrt(D)
            live = np.isfinite(lse[b, h])
            safe = np.where(live, lse[b, h], 0.0)
            with np.errstate(over="ignore"):
                W[b, kh] += np.where(mask & live[:, None], np.exp(s - safe[:, None]), 0.0).sum(0)
    return W


def gather(cache, table, n):
    """The first n rows [n, Hkv, D] of a sequence whose pages are ``table``."""
    page = cache.shape[1]
    return np.stack([cache[table[t // page], t % page] for t in range(n)]) if n else cache[:0, 0]


def paged_decode(q, kc, vc, table, lens, dt, window=0, sinks=0, weights=None):
    """O [B, Lq, H, D], LSE [B, H, Lq], bound on O, and the updated weights (or None)."""
    B, Lq, H, D = q.shape
    Hkv = kc.shape[2]
    g = H // Hkv
    O, bound = np.zeros((B, Lq, H, D)), np.zeros((B, Lq, H, D))
    lse = np.full((B, H, Lq), -np.inf)
    W = None if weights is None else weights.copy()
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        k, v = gather(kc, table[b], n), gather(vc, table[b], n)
        mask = seen(np.arange(n - Lq, n), n, window, sinks)
        for h in range(H):
            O[b, :, h], lse[b, h], bound[b, :, h] = unit_forward(q[b, :, h], k[:, h // g], v[:, h // g], mask, dt)
            if W is not None:
                W[b, h // g, :n] += unit(q[b, :, h], k[:, h // g], mask)[0].sum(0)
    return O, lse, bound, W


def survivors(w, n, keep, sinks, recent):
    """Kept slots of one sequence and K/V head, ascending: everything when n <= keep, else the first
    `sinks`, the last `recent` and the heaviest of the others (NaN heaviest, ties to the lower index)."""
    if n <= keep:
        return list(range(n))
    first, last = list(range(sinks)), list(range(n - recent, n))
    mid = range(sinks, n - recent)
    key = lambda j: (0 if np.isnan(w[j]) else 1, 0.0 if np.isnan(w[j]) else -float(w[j]), j)  # noqa: E731
    return sorted(first + sorted(mid, key=key)[: keep - sinks - recent] + last)
