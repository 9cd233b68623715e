"""The cache and window operators as measured workloads: what each case is, its inputs, one pass
through it in plain torch operations or through the library, and its result in 64 bits.

Operators (all on fp16 / bf16, grouped K/V heads, head dim 64 or 128):
  window   causal attention in which query i at position a = i + Lk - Lq sees key j iff j <= a and
           (j > a - window or j < sinks); forward, or forward and backward
  decode   a few new tokens against a paged key/value cache, optionally after writing them into
           the cache and with the keys' attention weights accumulated
  weights  the attention weight every key of a prompt has received, from the forward's LSE
  evict    the `keep` survivors of every sequence and K/V head by accumulated weight, moved into
           other pages
"""

import math

import numpy as np
import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A prompt's chunk of 200 queries against the 1,000 keys before and in it: the smallest
        # prefill call, where launch and pipeline latency count.
        dict(name="window_chunk", op="window", B=1, Lq=200, Lk=1200, H=32, Hkv=8, D=128, dtype="bf16",
             window=1024, sinks=4, train=False),
        # A whole prompt with a window, the ordinary prefill of a served model.
        dict(name="window_prompt_8k", op="window", B=1, Lq=8192, Lk=8192, H=32, Hkv=8, D=128, dtype="bf16",
             window=1024, sinks=4, train=False),
        # Training with small heads, an odd length and a window that is no multiple of a tile.
        dict(name="window_train_odd", op="window", B=3, Lq=777, Lk=777, H=8, Hkv=8, D=64, dtype="fp16",
             window=200, sinks=1, train=True),
        # The training step of the grouped-head configuration (B4 H32/8 L4096) with a window.
        dict(name="window_train_4k", op="window", B=4, Lq=4096, Lk=4096, H=32, Hkv=8, D=128, dtype="bf16",
             window=1024, sinks=4, train=True),
        # One user, a short context, one token: nothing but latency.
        dict(name="decode_short", op="decode", B=1, Lq=1, H=32, Hkv=8, D=128, dtype="bf16", page=16, lo=500,
             hi=500, window=0, sinks=0, step=False, empty=0),
        # A full batch of long contexts of unequal length, two of its slots unused.
        dict(name="decode_batch_16k", op="decode", B=16, Lq=1, H=32, Hkv=8, D=128, dtype="bf16", page=64,
             lo=8000, hi=16384, window=0, sinks=0, step=False, empty=2),
        # Four drafted tokens a sequence checked at once, with the window the prompt had.
        dict(name="decode_draft_window", op="decode", B=8, Lq=4, H=32, Hkv=8, D=128, dtype="fp16", page=32,
             lo=2000, hi=32768, window=4096, sinks=4, step=False, empty=0),
        # A whole step: write the token, attend, accumulate the weights; one K/V head per query head.
        dict(name="decode_step_d64", op="decode", B=8, Lq=1, H=32, Hkv=32, D=64, dtype="fp16", page=128,
             lo=900, hi=4096, window=0, sinks=0, step=True, empty=0),
        # The weights of a whole prompt, before its cache is first cut down.
        dict(name="weights_prompt_4k", op="weights", B=1, Lq=4096, Lk=4096, H=32, Hkv=8, D=128, dtype="bf16",
             window=0, sinks=0),
        # The same of a short prompt of odd length with small heads.
        dict(name="weights_odd", op="weights", B=2, Lq=1001, Lk=1001, H=8, Hkv=2, D=64, dtype="fp16",
             window=0, sinks=0),
        # One long sequence cut down to a budget.
        dict(name="evict_one_32k", op="evict", B=1, Hkv=8, D=128, dtype="bf16", page=16, lo=32768, hi=32768,
             keep=2048, sinks=4, recent=256),
        # A batch of unequal sequences, some of them shorter than the budget.
        dict(name="evict_batch", op="evict", B=16, Hkv=8, D=128, dtype="bf16", page=64, lo=3000, hi=12000,
             keep=4096, sinks=4, recent=1000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "decode", "decode", "decode", "weights", "evict"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 8])
    if op in ("window", "weights"):
        while True:
            B = rng.choice([1, 1, 2, 3, 4])
            Lq = _log_int(rng, 64, 8192)
            Lk = Lq if rng.random() < 0.6 else Lq + _log_int(rng, 1, 4096)
            window = _log_int(rng, 32, 4096) if op == "window" or rng.random() < 0.3 else 0
            sinks = rng.choice([0, 1, 4, 64]) if window else 0
            c = dict(op=op, B=B, Lq=Lq, Lk=Lk, H=H, Hkv=Hkv, D=D, dtype=dtype, window=window, sinks=sinks)
            if op == "window":
                c["train"] = Lq == Lk and rng.random() < 0.5
            # the plain forms hold whole score matrices
            if B * H * Lq * Lk <= 2.2e9 and work(c)["flops"] <= 8e11:
                return c
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        while True:
            B = _log_int(rng, 1, 64)
            hi = _log_int(rng, 16, 32768)
            lo = max(8, int(hi * rng.choice([0.25, 0.5, 1.0])))
            Lq = rng.choice([1, 1, 1, 2, 5])
            window, sinks = rng.choice([(0, 0), (0, 0), (0, 0), (1024, 4), (500, 0)])
            step = rng.random() < 0.4
            empty = 0 if step or B < 4 else rng.choice([0, 1])
            if B * hi * Hkv * D <= 3e8 and B * hi * H * Lq <= 2e8:
                return dict(op=op, B=B, Lq=Lq, H=H, Hkv=Hkv, D=D, dtype=dtype, page=page, lo=min(lo, hi), hi=hi,
                            window=window, sinks=sinks, step=step, empty=empty)
    while True:
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 256, 32768)
        keep = max(8, int(hi * rng.uniform(0.05, 0.9)))
        sinks = rng.choice([0, 4])
        recent = int((keep - sinks) * rng.uniform(0.0, 0.6))
        if B * hi * Hkv * D <= 3e8:
            return dict(op=op, B=B, Hkv=Hkv, D=D, dtype=dtype, page=page, lo=max(1, hi // 3), hi=hi, keep=keep,
                        sinks=sinks, recent=recent)


def _pairs(Lq, Lk, window, sinks):
    """Visible (query, key) pairs of one head."""
    a = np.arange(Lk - Lq, Lk, dtype=np.int64)
    if not window:
        return int((a + 1).sum())
    first = np.maximum(a - window + 1, 0)
    return int((a + 1 - first).sum() + np.minimum(first, sinks).sum())


def work(case):
    c = case
    if c["op"] == "window":
        n = c["B"] * c["H"] * _pairs(c["Lq"], c["Lk"], c["window"], c["sinks"])
        q, kv = c["B"] * c["Lq"] * c["H"] * c["D"] * 2, c["B"] * c["Lk"] * c["Hkv"] * c["D"] * 2
        lse = c["B"] * c["H"] * c["Lq"] * 4
        if not c["train"]:
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * c["D"] * n}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * c["D"] * n}
    if c["op"] == "weights":
        n = c["B"] * c["H"] * _pairs(c["Lq"], c["Lk"], c["window"], c["sinks"])
        return {"bytes": c["B"] * (c["Lq"] * c["H"] + c["Lk"] * c["Hkv"]) * c["D"] * 2
                + c["B"] * c["H"] * c["Lq"] * 4 + c["B"] * c["Hkv"] * c["Lk"] * 4,
                "flops": 2 * c["D"] * n}
    if c["op"] == "decode":
        mean = (c["lo"] + c["hi"]) / 2
        if c["window"]:
            mean = min(mean, c["window"] + c["sinks"] + c["Lq"])
        keys = (c["B"] - c["empty"]) * mean
        b = keys * c["Hkv"] * c["D"] * 4 + 4 * c["B"] * c["Lq"] * c["H"] * c["D"]
        if c["step"]:
            b += keys * c["Hkv"] * 8
        return {"bytes": b, "flops": 4 * keys * c["Lq"] * c["H"] * c["D"]}
    mean = (c["lo"] + c["hi"]) / 2
    kept = min(c["keep"], mean)
    return {"bytes": c["B"] * c["Hkv"] * (4 * mean + kept * (c["D"] * 8 + 8)),
            "flops": c["B"] * c["Hkv"] * mean}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    if c["op"] in ("window", "weights"):
        s = dict(case=c, q=rand(c["B"], c["Lq"], c["H"], c["D"]), k=rand(c["B"], c["Lk"], c["Hkv"], c["D"]))
        if c["op"] == "weights":
            s["lse"] = _lse(_scores(s["q"], s["k"], _seen(c["Lq"], c["Lk"], c["window"], c["sinks"])))
            return s
        s["v"] = rand(c["B"], c["Lk"], c["Hkv"], c["D"])
        if c["train"]:
            s["do"] = rand(c["B"], c["Lq"], c["H"], c["D"])
        return s

    # A pool of pages in use by other sequences too: every sequence's pages lie anywhere in it.
    B, page = c["B"], c["page"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    wide = -(-c["hi"] // page)
    spare = -(-c.get("keep", 0) // page)
    order = torch.randperm(B * (wide + spare), generator=g, device="cuda").to(torch.int32).view(B, wide + spare)
    s = dict(case=c, k=rand(order.numel(), page, c["Hkv"], c["D"]), v=rand(order.numel(), page, c["Hkv"], c["D"]),
             table=order[:, :wide].contiguous())
    if c["op"] == "decode":
        if c["empty"]:
            lens[B - c["empty"]:] = 0
        s.update(q=rand(B, c["Lq"], c["H"], c["D"]), lens=lens)
        if c["step"]:
            s.update(k_new=rand(B, c["Lq"], c["Hkv"], c["D"]), v_new=rand(B, c["Lq"], c["Hkv"], c["D"]),
                     start=lens - c["Lq"],
                     weights=torch.rand(B, c["Hkv"], wide * page, generator=g, device="cuda") * 4)
        return s
    # Accumulated weights are heavy-tailed, and many keys have never been looked at.
    w = torch.exp(2 * torch.randn(B, c["Hkv"], wide * page, generator=g, device="cuda") - 3)
    w[torch.rand(w.shape, generator=g, device="cuda") < 0.1] = 0
    s.update(lens=lens, weights=w, dst=order[:, wide:].contiguous())
    return s


# ------------------------------------------------------------------ plain forms

def _seen(Lq, Lk, window, sinks):
    """[Lq, Lk]: which keys each query sees."""
    a = torch.arange(Lk - Lq, Lk, device="cuda")[:, None]
    j = torch.arange(Lk, device="cuda")[None, :]
    seen = j <= a
    return seen & ((j > a - window) | (j < sinks)) if window else seen


def _heads(x, Hkv):
    """[B, L, H, D] -> [B, Hkv, H / Hkv, L, D] in 32 bits."""
    B, L, H, D = x.shape
    return x.float().view(B, L, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)


def _back(x, dtype):
    """[B, Hkv, g, L, D] -> [B, L, H, D]."""
    B, Hkv, g, L, D = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, L, Hkv * g, D).to(dtype)


def _scores(q, k, seen):
    s = _heads(q, k.shape[2]) @ _heads(k, k.shape[2]).transpose(-1, -2)
    return s.mul_(1 / math.sqrt(q.shape[-1])).masked_fill_(~seen, -math.inf)


def _lse(s):
    """[B, Hkv, g, Lq, Lk] -> [B, H, Lq]; -inf where a row sees nothing."""
    m = s.amax(-1)
    safe = m.masked_fill(m == -math.inf, 0)
    lse = safe + (s - safe[..., None]).exp_().sum(-1).log()
    return lse.flatten(1, 2)


def _window_plain(s, c):
    q, k, v = s["q"], s["k"], s["v"]
    Hkv = k.shape[2]
    p = _scores(q, k, _seen(c["Lq"], c["Lk"], c["window"], c["sinks"]))
    lse = _lse(p)
    p = p.sub_(lse.view(p.shape[:-1])[..., None]).exp_()
    vh = _heads(v, Hkv)
    o = p @ vh
    if not c["train"]:
        return _back(o, q.dtype), lse
    do, scale = _heads(s["do"], Hkv), 1 / math.sqrt(c["D"])
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    ds = (do @ vh.transpose(-1, -2)).sub_((o * do).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ _heads(k, Hkv)) * scale
    dk = (ds.transpose(-1, -2) @ _heads(q, Hkv)).sum(2, keepdim=True) * scale
    return _back(o, q.dtype), lse, _back(dq, q.dtype), _back(dk, q.dtype), _back(dv, q.dtype)


def _decode_plain(s, c):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    B, Lq, page = c["B"], c["Lq"], c["page"]
    if c["step"]:
        at = s["start"].long()[:, None] + torch.arange(Lq, device="cuda")
        pages, rows = torch.gather(table, 1, at // page), at % page
        s["k"][pages, rows] = s["k_new"]
        s["v"][pages, rows] = s["v_new"]
        s["weights"].scatter_(2, at[:, None, :].expand(B, c["Hkv"], Lq), 0.0)
    n = table.shape[1] * page
    k = s["k"][table].reshape(B, n, c["Hkv"], c["D"])
    v = s["v"][table].reshape(B, n, c["Hkv"], c["D"])
    a = lens[:, None, None] - Lq + torch.arange(Lq, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")
    seen = j <= a
    if c["window"]:
        seen = seen & ((j > a - c["window"]) | (j < c["sinks"]))
    p = _scores(q, k, seen[:, None, None])
    lse = _lse(p)
    to = lse.view(p.shape[:-1])[..., None]
    p = p.sub_(to.masked_fill(to == -math.inf, 0)).exp_()
    o = _back(p @ _heads(v, c["Hkv"]), q.dtype)
    if not c["step"]:
        return o, lse
    s["weights"] += p.sum((2, 3))
    return o, lse, s["weights"], s["k"], s["v"]


def _weights_plain(s, c):
    p = _scores(s["q"], s["k"], _seen(c["Lq"], c["Lk"], c["window"], c["sinks"]))
    return p.sub_(s["lse"].view(p.shape[:-1])[..., None]).exp_().sum((2, 3))


def _evict_plain(s, c):
    w, keep, page = s["weights"], c["keep"], c["page"]
    B, Hkv, n = w.shape
    lens = s["lens"].long()[:, None, None]
    j = torch.arange(n, device="cuda")
    rank = torch.where((j < c["sinks"]) | (j >= lens - c["recent"]), math.inf, w)
    rank = rank.masked_fill(j >= lens, -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    t = torch.arange(keep, device="cuda")
    kept = torch.where(t < lens, best, n).sort(dim=-1).values
    live = kept < n
    src = torch.where(live, kept, 0)
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    sp, sr = s["table"].long()[b, src // page], src % page
    dp, dr = s["dst"].long()[b, t // page], t % page
    dr = dr.expand_as(src)
    s["k"][dp, dr, h] = torch.where(live[..., None], s["k"][sp, sr, h], s["k"][dp, dr, h])
    s["v"][dp, dr, h] = torch.where(live[..., None], s["v"][sp, sr, h], s["v"][dp, dr, h])
    new_w = torch.zeros(B, Hkv, s["dst"].shape[1] * page, device="cuda")
    new_w[..., :keep] = torch.where(live, torch.gather(w, 2, src), 0.0)
    kept = torch.where(live, kept, -1).to(torch.int32)
    return kept, s["lens"].clamp(max=keep), new_w, s["k"], s["v"]


def run(state):
    s = state
    c = s["case"]
    if own:
        import tiled_attention_fa_gb300 as fa
        if c["op"] == "window":
            o, lse = fa.window_fwd(s["q"], s["k"], s["v"], c["window"], c["sinks"])
            if not c["train"]:
                return o, lse
            dq, dk, dv, _ = fa.window_attention_backward(s["q"], s["k"], s["v"], o, lse, s["do"], c["window"],
                                                         c["sinks"])
            return o, lse, dq, dk, dv
        if c["op"] == "weights":
            return fa.key_weights(s["q"], s["k"], s["lse"], causal=True, window=c["window"], sinks=c["sinks"])
        if c["op"] == "decode":
            if not c["step"]:
                return fa.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], window=c["window"],
                                       sinks=c["sinks"])
            fa.paged_write(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["start"], weights=s["weights"])
            o, lse = fa.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], window=c["window"],
                                     sinks=c["sinks"], weights=s["weights"])
            return o, lse, s["weights"], s["k"], s["v"]
        kept, lens, w = fa.paged_evict(s["k"], s["v"], s["table"], s["lens"], s["weights"], s["dst"], c["keep"],
                                       sinks=c["sinks"], recent=c["recent"])
        return kept, lens, w, s["k"], s["v"]
    if c["op"] == "window":
        return _window_plain(s, c)
    if c["op"] == "weights":
        return _weights_plain(s, c)
    if c["op"] == "decode":
        return _decode_plain(s, c)
    return _evict_plain(s, c)


# ------------------------------------------------------------------ 64 bits

def _rows64(q, k, v, pos, window, sinks, lse=None):
    """One head in 64 bits: q [Lq, D] at positions pos, k, v [Lk, D] (v may be None).
    O, LSE and the probabilities, by the two-pass softmax."""
    x = torch.einsum("id,jd->ij", q, k) / math.sqrt(q.shape[1])
    j = torch.arange(k.shape[0], device=q.device)
    hide = j[None] > pos[:, None]
    if window:
        hide |= (j[None] <= pos[:, None] - window) & (j[None] >= sinks)
    x[hide] = -math.inf
    if lse is None:
        lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return (None if v is None else p @ v), lse, p


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "evict":
        w, lens = s["weights"].double().cpu().numpy(), s["lens"].cpu().numpy()
        new_w = np.zeros((c["B"], c["Hkv"], s["dst"].shape[1] * c["page"]))
        for b in range(c["B"]):
            n = int(lens[b])
            for h in range(c["Hkv"]):
                mid = np.arange(c["sinks"], max(n - c["recent"], c["sinks"]))
                best = mid[np.argsort(-w[b, h, mid], kind="stable")][: max(c["keep"] - c["sinks"] - c["recent"], 0)]
                kept = np.arange(n) if n <= c["keep"] else np.sort(
                    np.concatenate([np.arange(c["sinks"]), best, np.arange(n - c["recent"], n)]))
                new_w[b, h, : len(kept)] = w[b, h, kept]
        return None, None, new_w, None, None
    g = c["H"] // c["Hkv"]
    q = s["q"].double()
    if c["op"] == "decode":
        B, Lq = c["B"], c["Lq"]
        o = torch.zeros(B, Lq, c["H"], c["D"], dtype=torch.float64, device="cuda")
        lse = torch.full((B, c["H"], Lq), -math.inf, dtype=torch.float64, device="cuda")
        w = s["weights"].double() if c["step"] else None
        for b in range(B):
            n = int(s["lens"][b])
            if n == 0:
                continue
            k = s["k"][s["table"][b].long()].flatten(0, 1)[:n].double()
            v = s["v"][s["table"][b].long()].flatten(0, 1)[:n].double()
            if c["step"]:
                k[n - Lq:], v[n - Lq:] = s["k_new"][b].double(), s["v_new"][b].double()
                w[b, :, n - Lq: n] = 0
            pos = torch.arange(n - Lq, n, device="cuda")
            for h in range(c["H"]):
                o[b, :, h], lse[b, h], p = _rows64(q[b, :, h], k[:, h // g], v[:, h // g], pos, c["window"], c["sinks"])
                if c["step"]:
                    w[b, h // g, :n] += p.sum(0)
        return (o, lse, w, None, None) if c["step"] else (o, lse)
    k = s["k"].double()
    pos = torch.arange(c["Lk"] - c["Lq"], c["Lk"], device="cuda")
    if c["op"] == "weights":
        w = torch.zeros(c["B"], c["Hkv"], c["Lk"], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            for h in range(c["H"]):
                _, _, p = _rows64(q[b, :, h], k[b, :, h // g], None, pos, c["window"], c["sinks"],
                                  s["lse"][b, h].double())
                w[b, h // g] += p.sum(0)
        return w
    v = s["v"].double()
    o, lse = torch.zeros_like(q), torch.zeros(c["B"], c["H"], c["Lq"], dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(c["B"]):
        for h in range(c["H"]):
            kb, vb, qb = k[b, :, h // g], v[b, :, h // g], q[b, :, h]
            ob, lse[b, h], p = _rows64(qb, kb, vb, pos, c["window"], c["sinks"])
            o[b, :, h] = ob
            if c["train"]:
                dob = s["do"][b, :, h].double()
                dv[b, :, h // g] += p.T @ dob
                dp = dob @ vb.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(c["D"])
                dq[b, :, h] = ds @ kb
                dk[b, :, h // g] += ds.T @ qb
    return (o, lse, dq, dk, dv) if c["train"] else (o, lse)
