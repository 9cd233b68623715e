"""Rotary positions, the rotating append to a paged cache and decoding behind a shared prefix as
measured workloads: what each case is, its inputs, one pass through it in plain torch operations or
through the library, and its result in 64 bits.

Operators (all on fp16 / bf16, grouped K/V heads, head dim 64 or 128):
  rope     queries and keys turned by their positions, on one axis (text) or several (rows and
           columns of an image; time, height and width of a video): the pair (x, y) of a head's
           dims number i becomes (x cos t - y sin t, x sin t + y cos t) with
           t = position[axis of pair i] * base^(-2i / rotary dims); its backward pass turns the
           gradients by -t
  append   a step's new queries, keys and values: the queries turned, the keys turned on their way
           into the pages of a cache, the values into theirs, the new slots' weights reset
  prefix   new tokens of a batch whose sequences share long prefixes (one, or one a group of
           sequences): softmax over the prefix's keys and the sequence's own, both in pages
"""

import math

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The queries and keys of a prompt's chunk, out of the fused projection: the smallest call.
        dict(name="rope_chunk", op="rope", B=1, L=200, H=32, Hkv=8, D=128, rotary=128, axes=1, pairs="halves",
             dtype="bf16", train=False),
        # A whole prompt.
        dict(name="rope_prompt_8k", op="rope", B=1, L=8192, H=32, Hkv=8, D=128, rotary=128, axes=1, pairs="halves",
             dtype="bf16", train=False),
        # Image patches in training: rows and columns, half of each small head turned, odd length.
        dict(name="rope_image_train", op="rope", B=3, L=777, H=8, Hkv=8, D=64, rotary=32, axes=2, pairs="neighbours",
             dtype="fp16", train=True),
        # Video and text in training, at the grouped-head configuration (B4 H32/8 L4096).
        dict(name="rope_video_train", op="rope", B=4, L=4096, H=32, Hkv=8, D=128, rotary=128, axes=3, pairs="halves",
             dtype="bf16", train=True),
        # One user's next token: nothing but latency.
        dict(name="append_one", op="append", B=1, L=1, H=32, Hkv=8, D=128, rotary=128, axes=1, pairs="halves",
             dtype="bf16", page=16, lo=500, hi=500, ragged=False, weights=False),
        # The next token of a large batch, in a cache that is evicted by weight.
        dict(name="append_batch", op="append", B=256, L=1, H=32, Hkv=8, D=128, rotary=128, axes=1, pairs="halves",
             dtype="bf16", page=64, lo=100, hi=2000, ragged=False, weights=True),
        # Prompts with pictures, of unequal length in a padded batch.
        dict(name="append_prompts", op="append", B=4, L=2047, H=32, Hkv=8, D=128, rotary=128, axes=3, pairs="halves",
             dtype="bf16", page=128, lo=0, hi=3000, ragged=True, weights=False),
        # A few users of one assistant, short turns behind its instructions.
        dict(name="prefix_chat", op="prefix", B=8, Lq=1, H=32, Hkv=8, D=128, dtype="bf16", page=16, groups=1,
             plo=2001, phi=2001, lo=1, hi=100, empty=0),
        # Drafted tokens checked, four a sequence.
        dict(name="prefix_draft", op="prefix", B=20, Lq=4, H=32, Hkv=8, D=128, dtype="fp16", page=32, groups=1,
             plo=6001, phi=6001, lo=50, hi=800, empty=0),
        # Several documents, each with its own readers, small heads of their own, unused slots.
        dict(name="prefix_groups", op="prefix", B=40, Lq=1, H=16, Hkv=16, D=64, dtype="fp16", page=64, groups=5,
             plo=1000, phi=9000, lo=16, hi=500, empty=3),
        # One long document asked many questions at once.
        dict(name="prefix_document_32k", op="prefix", B=64, Lq=1, H=32, Hkv=8, D=128, dtype="bf16", page=64, groups=1,
             plo=32768, phi=32768, lo=100, hi=1000, empty=0),
        # Samples of one prompt, as many as a server runs at once.
        dict(name="prefix_samples", op="prefix", B=256, Lq=1, H=32, Hkv=8, D=128, dtype="bf16", page=128, groups=1,
             plo=16384, phi=16384, lo=64, hi=512, empty=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append", "prefix", "prefix", "prefix"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 7, 8])
    if op != "prefix":
        axes = rng.choice([1, 1, 2, 3])
        rotary = rng.choice([D, D, D // 2, D // 4])
        c = dict(op=op, H=H, Hkv=Hkv, D=D, rotary=rotary, axes=axes, pairs=rng.choice(["halves", "halves", "neighbours"]),
                 dtype=dtype)
    if op == "rope":
        while True:
            c.update(B=rng.choice([1, 1, 2, 3, 4]), L=_log_int(rng, 1, 16384), train=rng.random() < 0.5)
            if c["B"] * c["L"] * (H + Hkv) * D <= 8.3e7:
                return c
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        while True:
            L = 1 if rng.random() < 0.6 else _log_int(rng, 2, 4096)
            B = _log_int(rng, 1, 256)
            hi = _log_int(rng, 16, 4096)
            if B * L * (H + 2 * Hkv) * D <= 4e7 and B * (hi + L) * Hkv * D <= 4e8:
                c.update(B=B, L=L, page=page, lo=rng.choice([0, hi // 2, hi]), hi=hi, ragged=L > 1 and rng.random() < 0.5,
                         weights=rng.random() < 0.3)
                return c
    while True:
        B = _log_int(rng, 2, 256)
        Lq = rng.choice([1, 1, 1, 2, 5])
        groups = 1 if rng.random() < 0.6 else min(B, rng.randint(2, 8))
        phi = _log_int(rng, 64, 32768)
        plo = max(1, int(phi * rng.choice([0.25, 0.5, 1.0])))
        hi = _log_int(rng, 8, 2000)
        lo = max(Lq, int(hi * rng.choice([0.1, 0.5, 1.0])))
        empty = rng.choice([0, 0, 1]) if B >= 4 else 0
        if (lo <= hi and B * hi * Hkv * D <= 1.2e8 and groups * phi * Hkv * D <= 3e8
                and B * H * Lq * (phi + hi) <= 1.3e8):
            return dict(op=op, B=B, Lq=Lq, H=H, Hkv=Hkv, D=D, dtype=dtype, page=page, groups=groups, plo=plo, phi=phi,
                        lo=lo, hi=hi, empty=empty)


def _group_sizes(c):
    """Sequences of each group: unequal, and none of them empty."""
    G, B = c["groups"], c["B"]
    cut = [round(B * (i / G) ** 1.3) for i in range(G + 1)]
    for i in range(1, G + 1):
        cut[i] = min(max(cut[i], cut[i - 1] + 1), B - (G - i))
    return [b - a for a, b in zip(cut, cut[1:])]


def work(case):
    c = case
    D = c["D"]
    if c["op"] == "rope":
        n = c["B"] * c["L"] * (c["H"] + c["Hkv"]) * D * (2 if c["train"] else 1)
        return {"bytes": 4 * n + (4 * c["axes"] * c["B"] * c["L"] if c["axes"] > 1 else 0), "flops": 3 * n}
    if c["op"] == "append":
        tokens = c["B"] * c["L"]
        new = tokens * (0.5 if c["ragged"] else 1.0)  # those of a padded batch that count, in the mean
        b = 4 * D * (tokens * c["H"] + 2 * new * c["Hkv"]) + (4 * new * c["Hkv"] if c["weights"] else 0)
        return {"bytes": b + 4 * c["axes"] * tokens, "flops": 3 * D * (tokens * c["H"] + new * c["Hkv"])}
    live, rows = c["B"] - c["empty"], c["Lq"] * c["H"]
    prefix, mine = (c["plo"] + c["phi"]) / 2, (c["lo"] + c["hi"]) / 2
    return {"bytes": 4 * c["Hkv"] * D * (c["groups"] * prefix + live * mine) + c["B"] * rows * (4 * D + 4),
            "flops": 4 * D * live * rows * (prefix + mine)}


# ------------------------------------------------------------------ inputs

def _axes(c):
    """The axis of each pair: sections of a quarter for time and half of the rest each for height and
    width, or halves for two axes."""
    n = c["rotary"] // 2
    sections = {1: [n], 2: [n // 2, n - n // 2], 3: [n // 4, (n - n // 4) // 2, n - n // 4 - (n - n // 4) // 2]}
    return sections[c["axes"]]


def _positions(c, B, L, g):
    """[axes, B, L]: text counts up; an image or a video fills a grid, behind some text."""
    start = torch.randint(0, 100000, (B, 1), generator=g, device="cuda")
    i = torch.arange(L, device="cuda")[None]
    if c["axes"] == 1:
        return (start + i)[None].to(torch.int32)
    side = max(1, int(math.sqrt(L / (1 if c["axes"] == 2 else 4))))
    w, h, t = i % side, i // side % side, i // (side * side)
    at = [h, w] if c["axes"] == 2 else [t, h, w]
    return torch.stack([start + a for a in at]).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]
    B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)

    if c["op"] != "prefix":
        # The projection's output, one tensor: queries, keys and values are parts of each token's row.
        L = c["L"]
        s = dict(case=c, qkv=rand(B, L, H + 2 * Hkv, D), positions=None)
        if own:
            import tiled_attention_fa_gb300 as fa
            s["table"] = fa.rope_table(D, rotary=c["rotary"], sections=_axes(c))
        else:
            i = torch.arange(c["rotary"] // 2, dtype=torch.float64)
            s["freq"] = (10000.0 ** (-2.0 * i / c["rotary"])).cuda()
            s["axis"] = torch.tensor([a for a, count in enumerate(_axes(c)) for _ in range(count)]).cuda()
        if c["op"] == "rope":
            if c["axes"] > 1:
                s["positions"] = _positions(c, B, L, g)
            if c["train"]:
                s["dq"], s["dk"] = rand(B, L, H, D), rand(B, L, Hkv, D)
            return s
        # A cache's rotary positions are its slots only for text that was never cut.
        s["positions"] = _positions(c, B, L, g)
        s["counts"] = ints(1, L, B) if c["ragged"] else None
        page, wide = c["page"], -(-(c["hi"] + L) // c["page"])
        s["table_kv"] = torch.randperm(B * wide, generator=g, device="cuda").to(torch.int32).view(B, wide)
        s.update(k=rand(B * wide, page, Hkv, D), v=rand(B * wide, page, Hkv, D), start=ints(c["lo"], c["hi"], B))
        if c["weights"]:
            s["weights"] = torch.rand(B, Hkv, wide * page, generator=g, device="cuda") * 4
        return s

    # Prefixes' and sequences' pages lie anywhere in one pool.
    page, G = c["page"], c["groups"]
    pwide, wide = -(-c["phi"] // page), -(-c["hi"] // page)
    order = torch.randperm(G * pwide + B * wide, generator=g, device="cuda").to(torch.int32)
    plens, lens = ints(c["plo"], c["phi"], G), ints(c["lo"], c["hi"], B)
    if c["empty"]:
        lens[B - c["empty"]:] = 0
    sizes = _group_sizes(c)
    starts = torch.tensor([sum(sizes[:i]) for i in range(G + 1)], dtype=torch.int32, device="cuda")
    return dict(case=c, q=rand(B, c["Lq"], H, D), k=rand(order.numel(), page, Hkv, D), v=rand(order.numel(), page, Hkv, D),
                ptable=order[: G * pwide].view(G, pwide).contiguous(), plens=plens, starts=starts,
                table=order[G * pwide:].view(B, wide).contiguous(), lens=lens, sizes=sizes, host_plens=plens.tolist())


# ------------------------------------------------------------------ plain forms

def _angles(s, L):
    """cos and sin [B or 1, L, 1, pairs] in 32 bits, of angles in 64."""
    positions = s["positions"]
    if positions is None:
        positions = torch.arange(L, device="cuda", dtype=torch.int32)[None, None]
    at = positions.double()[s["axis"]].permute(1, 2, 0) * s["freq"]
    return at.cos().float()[:, :, None], at.sin().float()[:, :, None]


def _turn(x, cos, sin, c):
    """x [B, L, heads, D] turned."""
    R = c["rotary"]
    f = x.float()
    if c["pairs"] == "halves":
        a, b = f[..., : R // 2], f[..., R // 2: R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = f[..., 0:R:2], f[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, f[..., R:]], -1).to(x.dtype)


def _rope_plain(s, c):
    H, Hkv = c["H"], c["Hkv"]
    cos, sin = _angles(s, c["L"])
    out = [_turn(s["qkv"][:, :, :H], cos, sin, c), _turn(s["qkv"][:, :, H: H + Hkv], cos, sin, c)]
    if c["train"]:
        out += [_turn(s["dq"], cos, -sin, c), _turn(s["dk"], cos, -sin, c)]
    return tuple(out)


def _append_plain(s, c):
    B, L, H, Hkv, page = c["B"], c["L"], c["H"], c["Hkv"], c["page"]
    q, k, v = s["qkv"].split([H, Hkv, Hkv], 2)
    cos, sin = _angles(s, L)
    q, k = _turn(q, cos, sin, c), _turn(k, cos, sin, c)
    j = torch.arange(L, device="cuda")[None]
    at = s["start"].long()[:, None] + j
    pages, rows = torch.gather(s["table_kv"].long(), 1, at // page), at % page
    if s["counts"] is not None:
        live = j < s["counts"][:, None]
        pages, rows, k, v = pages[live], rows[live], k[live], v[live]
    s["k"][pages, rows] = k
    s["v"][pages, rows] = v
    if not c["weights"]:
        return q, s["k"], s["v"]
    to = at.clone()
    if s["counts"] is not None:
        to = torch.where(live, at, at[:, :1])  # (the first token counts)
    s["weights"].scatter_(2, to[:, None, :].expand(B, Hkv, L), 0.0)
    return q, s["k"], s["v"], s["weights"]


def _prefix_plain(s, c):
    B, Lq, H, Hkv, D, page = c["B"], c["Lq"], c["H"], c["Hkv"], c["D"], c["page"]
    g = H // Hkv
    q = s["q"].float().view(B, Lq, Hkv, g, D).permute(2, 0, 3, 1, 4)  # [Hkv, B, g, Lq, D]
    scale = 1 / math.sqrt(D)
    n = s["table"].shape[1] * page
    own_k = s["k"][s["table"].long()].reshape(B, n, Hkv, D).float().permute(2, 0, 1, 3)
    own_v = s["v"][s["table"].long()].reshape(B, n, Hkv, D).float().permute(2, 0, 1, 3)
    x = torch.matmul(q.reshape(Hkv, B, g * Lq, D), own_k.transpose(-1, -2)).view(Hkv, B, g, Lq, n) * scale
    a = s["lens"].long()[:, None] - Lq + torch.arange(Lq, device="cuda")
    seen = torch.arange(n, device="cuda") <= a[..., None]
    x = x.masked_fill_(~seen[None, :, None], -math.inf)
    lse = torch.empty(Hkv, B, g, Lq, device="cuda")
    o = torch.empty(Hkv, B, g, Lq, D, device="cuda")
    b0 = 0
    for i, size in enumerate(s["sizes"]):
        m = s["host_plens"][i]
        at = s["ptable"][i].long()
        kp = s["k"][at].flatten(0, 1)[:m].float().permute(1, 0, 2)  # [Hkv, m, D]
        vp = s["v"][at].flatten(0, 1)[:m].float().permute(1, 0, 2)
        part = slice(b0, b0 + size)
        b0 += size
        y = torch.matmul(q[:, part].reshape(Hkv, -1, D), kp.transpose(-1, -2)).mul_(scale).view(Hkv, size, g, Lq, m)
        z = x[:, part]
        top = torch.maximum(y.amax(-1), z.amax(-1))[..., None]
        y, z = y.sub_(top).exp_(), (z - top).exp_()
        den = y.sum(-1) + z.sum(-1)
        lse[:, part] = top[..., 0] + den.log()
        sum_o = torch.matmul(y.view(Hkv, -1, m), vp).view(Hkv, size, g, Lq, D)
        sum_o += torch.matmul(z.reshape(Hkv, size, g * Lq, n), own_v[:, part]).view(Hkv, size, g, Lq, D)
        o[:, part] = sum_o / den[..., None]
    pad = (a < 0)[None, :, None]  # a query before its sequence's first key is padding
    o.masked_fill_(pad[..., None], 0.0)
    lse.masked_fill_(pad, -math.inf)
    return (o.permute(1, 3, 0, 2, 4).reshape(B, Lq, H, D).to(s["q"].dtype),
            lse.permute(1, 0, 2, 3).reshape(B, H, Lq))


def run(state):
    s = state
    c = s["case"]
    if own:
        import tiled_attention_fa_gb300 as fa
        if c["op"] == "prefix":
            return fa.paged_prefix_decode(s["q"], s["k"], s["v"], s["ptable"], s["plens"], s["table"], s["lens"],
                                          group_starts=s["starts"])
        H, Hkv = c["H"], c["Hkv"]
        q, k = s["qkv"][:, :, :H], s["qkv"][:, :, H: H + Hkv]
        neighbours = c["pairs"] == "neighbours"
        if c["op"] == "rope":
            out = fa.rope_fwd(q, k, s["table"], s["positions"], interleaved=neighbours)
            if c["train"]:
                out = out + fa.rope_bwd(s["dq"], s["dk"], s["table"], s["positions"], interleaved=neighbours)
            return out
        v = s["qkv"][:, :, H + Hkv:]
        w = s.get("weights")
        q = fa.paged_append(q, k, v, s["k"], s["v"], s["table_kv"], s["start"], s["table"], s["positions"],
                            counts=s["counts"], interleaved=neighbours, weights=w)
        return (q, s["k"], s["v"]) if w is None else (q, s["k"], s["v"], w)
    if c["op"] == "rope":
        return _rope_plain(s, c)
    if c["op"] == "append":
        return _append_plain(s, c)
    return _prefix_plain(s, c)


# ------------------------------------------------------------------ 64 bits

def _spun(x, c, positions, sign=1.0):
    """x [B, L, heads, D] in 64 bits, its pairs as complex numbers times e^(i t)."""
    B, L, heads, D = x.shape
    R, n = c["rotary"], c["rotary"] // 2
    turn = torch.zeros(B, L, n, dtype=torch.float64, device=x.device)
    p = 0
    for axis, count in enumerate(_axes(c)):
        for _ in range(count):
            at = torch.arange(L, device=x.device) if positions is None else positions[axis]
            turn[:, :, p] = at.to(torch.float64) * math.exp(-math.log(10000.0) * p / n)
            p += 1
    spin = torch.polar(torch.ones_like(turn), sign * turn)
    y = x.double().clone()
    for h in range(heads):
        rot = y[:, :, h, :R]
        if c["pairs"] == "halves":
            z = torch.complex(rot[..., :n].contiguous(), rot[..., n:].contiguous()) * spin
            y[:, :, h, :R] = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(rot.reshape(B, L, n, 2).contiguous()) * spin
            y[:, :, h, :R] = torch.view_as_real(z).reshape(B, L, R)
    return y


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        out = [_spun(s["qkv"][:, :, :H], c, s["positions"]), _spun(s["qkv"][:, :, H: H + Hkv], c, s["positions"])]
        if c["train"]:
            out += [_spun(s["dq"], c, s["positions"], -1.0), _spun(s["dk"], c, s["positions"], -1.0)]
        return tuple(out)
    if c["op"] == "append":
        q = _spun(s["qkv"][:, :, :H], c, s["positions"])
        k = _spun(s["qkv"][:, :, H: H + Hkv], c, s["positions"])
        pool = s["k"].double()
        start, table, page = s["start"].tolist(), s["table_kv"].tolist(), c["page"]
        counts = s["counts"].tolist() if c["ragged"] else [c["L"]] * c["B"]
        for b in range(c["B"]):
            slots = range(start[b], start[b] + counts[b])
            flat = torch.tensor([table[b][t // page] * page + t % page for t in slots], device="cuda")
            pool.view(-1, Hkv, D)[flat] = k[b, : counts[b]]
        return (q, pool, None, None) if c["weights"] else (q, pool, None)
    B, Lq = c["B"], c["Lq"]
    g = H // Hkv
    o = torch.zeros(B, Lq, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Lq), -math.inf, dtype=torch.float64, device="cuda")
    if B * H > 10000:
        return None
    b = 0
    for i, size in enumerate(s["sizes"]):
        m = int(s["plens"][i])
        kp = s["k"][s["ptable"][i].long()].reshape(-1, Hkv, D)[:m].double()
        vp = s["v"][s["ptable"][i].long()].reshape(-1, Hkv, D)[:m].double()
        for b in range(b, b + size):
            n = int(s["lens"][b])
            k = torch.cat([kp, s["k"][s["table"][b].long()].reshape(-1, Hkv, D)[:n].double()])
            v = torch.cat([vp, s["v"][s["table"][b].long()].reshape(-1, Hkv, D)[:n].double()])
            for x in range(Lq):
                if n - Lq + x < 0:
                    continue
                sees = m + n - Lq + x + 1
                qx = s["q"][b, x].double().view(Hkv, g, D)
                z = torch.einsum("hgd,jhd->hgj", qx, k[:sees]) / math.sqrt(D)
                lse[b, :, x] = torch.logsumexp(z, -1).flatten()
                o[b, x] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, -1), v[:sees]).reshape(H, D)
        b += 1
    return o, lse
