"""Decoding behind shared prefixes against the 64-bit reference (tests/cache_ref.py) over the joined
keys of each sequence.  Slots that no query may use hold NaN."""

import numpy as np
import pytest
import torch

import tiled_attention_fa_gb300 as fa
from tests import cache_ref as ref
from tests.helpers import to64
from tests.test_gpu_window import within
from tiled_attention_fa_gb300 import _lib
from tiled_attention_fa_gb300.inputs import storage_dtype

pytestmark = pytest.mark.gpu


def setup(Lq, H, Hkv, D, dtype, page, plens, sizes, lens, seed, joint=False):
    """Pools with prefixes' and own keys in pages in random order, NaN in every other slot; tables with
    -1 where no page is needed."""
    g = torch.Generator().manual_seed(seed)
    dt = storage_dtype(dtype)
    B, G = len(lens), len(plens)
    PP, P = (max(1, -(-max(x) // page)) for x in (plens, lens))
    pages = G * PP + B * P + 2
    kv = torch.randn(pages, 2, page, Hkv, D, generator=g).to(dt)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    ptable, table = order[: G * PP].view(G, PP).clone(), order[G * PP: G * PP + B * P].view(B, P).clone()
    use = torch.zeros(pages, page, dtype=torch.bool)
    for t, ns in ((ptable, plens), (table, lens)):
        for row, n in zip(t, ns):
            for j in range(t.shape[1]):
                left = min(max(n - j * page, 0), page)
                if left:
                    use[row[j], :left] = True
                else:
                    row[j] = -1
    kv.permute(0, 2, 1, 3, 4)[~use] = float("nan")
    q = torch.randn(B, Lq, H, D, generator=g).to(dt)
    kv = kv.cuda()
    k, v = (kv[:, 0], kv[:, 1]) if joint else (kv[:, 0].contiguous(), kv[:, 1].contiguous())
    starts = np.concatenate([[0], np.cumsum(sizes)])
    as_int = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    return q.cuda(), k, v, ptable.cuda(), as_int(plens), table.cuda(), as_int(lens), as_int(starts)


def expected(q, k, v, ptable, plens, table, lens, starts, dtype):
    q, k, v = to64(q), to64(k), to64(v)
    ptable, table, plens, lens, starts = (x.cpu().numpy() for x in (ptable, table, plens, lens, starts))
    B, Lq, H, D = q.shape
    g = H // k.shape[2]
    O, bound, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((B, H, Lq), -np.inf)
    for b in range(B):
        grp = [i for i in range(len(plens)) if starts[i] <= b < starts[i + 1]]
        m, n = (int(plens[grp[0]]) if grp else 0), int(lens[b])
        parts = ([(ptable[grp[0]], m)] if m > 0 else []) + [(table[b], n)]
        if n <= 0:
            continue
        kb, vb = (np.concatenate([ref.gather(x, t, c) for t, c in parts]) for x in (k, v))
        own = np.arange(n - Lq, n)
        mask = ref.seen(m + own, m + n) & (own >= 0)[:, None]
        for h in range(H):
            O[b, :, h], lse[b, h], bound[b, :, h] = ref.unit_forward(q[b, :, h], kb[:, h // g], vb[:, h // g], mask, dtype)
    return O, lse, bound


def check(Lq, H, Hkv, D, dtype, page, plens, sizes, lens, seed=0, joint=False):
    args = setup(Lq, H, Hkv, D, dtype, page, plens, sizes, lens, seed, joint)
    q, k, v, ptable, pl, table, ln, starts = args
    o, lse = fa.paged_prefix_decode(q, k, v, ptable, pl, table, ln, starts)
    torch.cuda.synchronize()
    fa.check_device_error()
    O, L, bound = expected(*args, dtype)
    within(to64(o), O, bound, "O")
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(to64(lse)), empty)
    within(np.where(empty, 0, to64(lse)), np.where(empty, 0, L), np.full(L.shape, ref.FP32), "LSE")
    return args, o, lse


CASES = [
    # Lq, H, Hkv, D, dtype, page, plens, sizes, lens
    (1, 1, 1, 64, "fp16", 16, [1], [1], [1]),
    (1, 8, 8, 128, "bf16", 16, [500], [2], [3, 200]),
    (1, 32, 8, 128, "bf16", 64, [1000], [5], [1, 0, 77, 300, 129]),
    (4, 8, 2, 128, "fp16", 32, [300], [12], [4, 9, 2, 100] * 3),        # 192 rows: two tiles; two tokens of four
    (1, 7, 1, 64, "bf16", 128, [129], [40], [5] * 40),                  # 18 tokens a tile, rows left over
    (2, 6, 2, 64, "fp16", 256, [700], [50], list(range(50))),           # 21 tokens a tile, three tiles
    (1, 4, 4, 64, "bf16", 16, [128, 0, 2000, 31], [3, 2, 1, 4], [20, 1, 5, 60, 3, 400, 1, 2, 3, 4]),
    (3, 16, 4, 128, "bf16", 16, [257, 640], [40, 3], [7] * 43),         # groups of one and of several tiles
    (1, 128, 1, 128, "fp16", 64, [400], [3], [30, 1, 2]),               # a token fills a tile
    (25, 5, 1, 64, "bf16", 32, [333], [2], [25, 60]),                   # 125 rows a sequence
    (1, 8, 2, 128, "fp16", 64, [5000], [1], [10]),
]


@pytest.mark.parametrize("Lq,H,Hkv,D,dtype,page,plens,sizes,lens", CASES)
def test_prefix(cuda_lib, Lq, H, Hkv, D, dtype, page, plens, sizes, lens):
    check(Lq, H, Hkv, D, dtype, page, plens, sizes, lens, seed=sum(plens) + D)


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_long_prefix_in_many_parts(cuda_lib, D, dtype):
    check(1, 4, 1, D, dtype, 16, [20001], [40], [1 + 7 * i for i in range(40)], seed=1, joint=True)


@pytest.mark.parametrize("Lq,H,Hkv,D,dtype,page", [(1, 16, 16, 64, "fp16", 64), (1, 8, 2, 128, "bf16", 16), (3, 10, 2, 64, "bf16", 32),
                                                   (4, 32, 4, 128, "fp16", 128), (8, 8, 1, 128, "bf16", 64)])
def test_long_own_keys(cuda_lib, Lq, H, Hkv, D, dtype, page):
    """Own keys of many tiles (a sequence's tiles then go to both softmax groups in turn), 1 to 64 rows."""
    lens = [Lq + (i * 977) % 2000 for i in range(20)]
    check(Lq, H, Hkv, D, dtype, page, [700, 90], [15, 5], lens, seed=12)


def test_many_groups(cuda_lib):
    """More groups than threads that scan them; sequences before the first and behind the last."""
    sizes = [(5 * i) % 3 for i in range(400)]
    plens = [(37 * i * i) % 300 if i % 4 else 0 for i in range(400)]
    lens = [1 + (i * 13) % 40 for i in range(sum(sizes) + 5)]
    args = list(setup(1, 2, 1, 64, "fp16", 16, plens, sizes, lens, 3))
    args[7] = args[7] + 3
    o, lse = fa.paged_prefix_decode(*args)
    torch.cuda.synchronize()
    fa.check_device_error()
    O, L, bound = expected(*args, "fp16")
    within(to64(o), O, bound, "O")
    within(to64(lse), L, np.full(L.shape, ref.FP32), "LSE")


def test_no_groups_given_is_one(cuda_lib):
    args, o, lse = check(1, 8, 2, 64, "bf16", 32, [321], [9], [5] * 9, seed=4)
    got = fa.paged_prefix_decode(*args[:7])
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_rising_scores(cuda_lib):
    """Each tile's scores lie above the last one's, in the prefix and on into the own keys."""
    args = setup(1, 4, 2, 64, "fp16", 16, [1500], [3], [200] * 3, 8)
    q, k, v, ptable, _, table, _, _ = args
    k.zero_(), v.nan_to_num_(), q.zero_()
    q[..., 0] = 8.0
    k[ptable[0].long(), :, :, 0] = (torch.arange(ptable.shape[1] * 16) / 16.0).view(-1, 16, 1).to(k.dtype).cuda()
    for b in range(3):
        at = table[b].long()
        k[at, :, :, 0] = (94 + torch.arange(len(at) * 16) / 16.0).view(-1, 16, 1).to(k.dtype).cuda()
    o, lse = fa.paged_prefix_decode(*args)
    torch.cuda.synchronize()
    O, L, bound = expected(*args, "fp16")
    within(to64(o), O, bound, "O")
    # scores up to 107, scaled in fp32 (2^-22 relative)
    within(to64(lse), L, ref.FP32 + np.abs(L) * 2.0 ** -20, "LSE")


def test_not_numbers(cuda_lib):
    """NaN in a query stays in its row; NaN in a prefix's key reaches its group's rows alone; scores of
    -inf weigh nothing."""
    args = setup(1, 4, 2, 64, "bf16", 16, [200, 150], [3, 2], [9] * 5, 5)
    q, k, v, ptable, plens, table, lens, starts = args
    clean = fa.paged_prefix_decode(*args)
    q2 = q.clone()
    q2[1, 0, 2, 7] = float("nan")
    o, lse = fa.paged_prefix_decode(q2, *args[1:])
    bad = torch.zeros(5, 4, 1, dtype=torch.bool, device="cuda")
    bad[1, 2] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.isnan(o[1, 0, 2]).all()
    assert torch.equal(lse[~bad], clean[1][~bad])
    k2 = k.clone()
    k2[ptable[1, 3].long(), 5, 1] = float("nan")                       # key 53 of group 1, K/V head 1
    o, lse = fa.paged_prefix_decode(q, k2, *args[2:])
    bad.zero_()
    bad[3:, 2:] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(o).all(-1).transpose(1, 2), bad)
    k3, q3 = k.clone(), q.abs() + 0.1
    k3[ptable[0, :8].long()] = float("-inf")                           # a whole tile of -inf scores
    o, lse = fa.paged_prefix_decode(q3, k3, *args[2:])
    torch.cuda.synchronize()
    fa.check_device_error()
    k64 = to64(k3)
    with np.errstate(invalid="ignore"):
        O, L, bound = expected(q3, torch.from_numpy(np.maximum(k64, -1e4)), *args[2:], "bf16")
    within(to64(o)[:3], O[:3], bound[:3], "O")
    within(to64(lse)[:3], L[:3], np.full(L[:3].shape, ref.FP32), "LSE")


def test_wrong_tables_lengths_and_groups_stay_in_bounds(cuda_lib):
    q, k, v, ptable, plens, table, lens, starts = setup(1, 4, 2, 64, "fp16", 16, [100, 90], [2, 3], [30] * 5, 6)
    k.nan_to_num_(), v.nan_to_num_()
    for kw in (dict(plens=[10 ** 9, -7]), dict(lens=[10 ** 9, -5, 3, 0, 2 ** 31 - 1]), dict(starts=[5, 0, 5]), dict(starts=[0, 5, -9]),
               dict(starts=[-3, 2, 10 ** 6]), dict(starts=[0, 5, 0])):
        a = dict(plens=plens, lens=lens, starts=starts)
        a.update({x: torch.tensor(y, dtype=torch.int32, device="cuda") for x, y in kw.items()})
        o, lse = fa.paged_prefix_decode(q, k, v, ptable, a["plens"], table, a["lens"], a["starts"])
        assert torch.isfinite(o).all()
    wrong, wrong2 = ptable.clone(), table.clone()
    wrong[0, 1], wrong[1, 0], wrong2[2, 1] = 10 ** 9, -(10 ** 9), 10 ** 8
    o, _ = fa.paged_prefix_decode(q, k, v, wrong, plens, wrong2, lens, starts)
    # 200 groups of all 400 sequences each: more items than there is room for
    many = torch.tensor([0, 400] * 200 + [0], dtype=torch.int32, device="cuda")
    o2, _ = fa.paged_prefix_decode(q[:1].expand(400, -1, -1, -1).contiguous(), k, v, ptable[:1].expand(400, -1).contiguous(),
                                   torch.full((400,), 100, dtype=torch.int32, device="cuda"),
                                   table[:1].expand(400, -1).contiguous(), lens[:1].expand(400).contiguous(), many)
    torch.cuda.synchronize()
    fa.check_device_error()
    assert torch.isfinite(o).all() and o2.shape == (400, 1, 4, 64)     # (what starts that fall give is unspecified)


def test_same_as_the_whole_table(cuda_lib):
    """paged_decode over tables that list the prefix's pages first, for a prefix of whole pages: the same
    function, off by what both may round."""
    Lq, H, Hkv, D, page, n = 2, 8, 2, 128, 32, 640
    args = setup(Lq, H, Hkv, D, "bf16", page, [n], [6], [40, 3, 100, 7, 2, 66], 9)
    q, k, v, ptable, plens, table, lens, starts = args
    o, lse = fa.paged_prefix_decode(*args)
    whole = torch.cat([ptable.expand(6, -1), table], 1).contiguous()
    o2, lse2 = fa.paged_decode(q, k, v, whole, lens + n)
    torch.cuda.synchronize()
    _, _, bound = expected(*args, "bf16")
    within(to64(o), to64(o2), 2 * bound, "O")
    within(to64(lse), to64(lse2), np.full(lse.shape, 2 * ref.FP32), "LSE")


def test_steps_behind_a_prefix(cuda_lib):
    """As it is used: a prefix appended once, then every sequence's tokens appended (turned by their
    positions behind it) and attended to, captured as one graph and replayed."""
    from tests import rope_ref
    from tests.test_gpu_rope import freqs
    B, H, Hkv, D, page, n, steps = 5, 8, 2, 64, 16, 150, 4
    g = torch.Generator().manual_seed(2)
    P, PP = 1, -(-n // page)
    kc, vc = (torch.full((PP + B * P, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    order = torch.randperm(PP + B * P, generator=g).to(torch.int32).cuda()
    ptable, bt = order[None, :PP].contiguous(), order[PP:].view(B, P).contiguous()
    table = fa.rope_table(D)
    qkv0 = torch.randn(1, n, H + 2 * Hkv, D, generator=g).bfloat16()
    toks = torch.randn(steps, B, 1, H + 2 * Hkv, D, generator=g).bfloat16()
    fa.paged_append(*qkv0.cuda().split([H, Hkv, Hkv], 2), kc, vc, ptable, torch.zeros(1, dtype=torch.int32, device="cuda"), table)
    plens = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens, pos = start + 1, torch.full((1, B, 1), n, dtype=torch.int32, device="cuda")
    tok = toks[0].cuda()

    def step():
        q = fa.paged_append(*tok.split([H, Hkv, Hkv], 2), kc, vc, bt, start, table, pos)
        return fa.paged_prefix_decode(q, kc, vc, ptable, plens, bt, lens)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = step()
    # the turned values as they are stored
    whole = torch.cat([qkv0.expand(B, -1, -1, -1), toks[:, :, 0].transpose(0, 1)], 1)
    at = np.broadcast_to(np.arange(n + steps), (1, B, n + steps))
    turned = fa.rope_fwd(*whole.cuda().split([H, Hkv, Hkv], 2)[:2], table)
    for x, y in zip(whole.split([H, Hkv, Hkv], 2), turned):
        within(to64(y), *rope_ref.turned(to64(x), at, freqs(D), [0] * 32, D, False, "bf16"), "turned")
    O, _, bound = ref.forward(to64(turned[0]), to64(turned[1]), to64(whole[:, :, H + Hkv:]),
                              ref.seen(np.arange(n + steps), n + steps), "bf16")
    for i in range(steps):
        tok.copy_(toks[i])
        start.fill_(i), lens.fill_(i + 1), pos.fill_(n + i)
        graph.replay()
        torch.cuda.synchronize()
        within(to64(o), O[:, n + i: n + i + 1], bound[:, n + i: n + i + 1], f"O at {i}")
    fa.check_device_error()


@pytest.mark.parametrize("Lq,H,D,page,plens,sizes,hi", [(1, 32, 128, 64, [9000], [64], 700), (4, 32, 128, 16, [3001], [12], 300),
                                                        (1, 16, 64, 32, [4000, 1500, 700], [20, 9, 11], 200)])
def test_many_runs_under_load_give_the_same_bits(Lq, H, D, page, plens, sizes, hi):
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(Lq, hi + 1, (sum(sizes),), generator=g).tolist()
    args = setup(Lq, H, 8, D, "bf16", page, plens, sizes, lens, 10)
    outs = torch.stack([fa.paged_prefix_decode(*args)[0] for _ in range(40)])
    torch.cuda.synchronize()
    fa.check_device_error()
    assert not [i for i, o in enumerate(outs) if not torch.equal(o, outs[0])]


def test_two_calls_at_once(cuda_lib):
    """Two streams, eager and captured, each with a workspace of its own."""
    cases = [setup(1, 8, 2, 64, "fp16", 32, [900], [40], [31] * 40, s) for s in (1, 2)]
    want = [fa.paged_prefix_decode(*a) for a in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, outs = [], []
    for a in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(fa.paged_prefix_decode(*a))
        graphs.append(gr)
    for _ in range(20):
        eager = []
        for gr, a, s in zip(graphs, cases, streams):
            with torch.cuda.stream(s):
                gr.replay()
                eager.append(fa.paged_prefix_decode(*a))
        torch.cuda.synchronize()
        for got in (outs, eager):
            for x, y in zip(got, want):
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    fa.check_device_error()


def test_workspace_and_stream(cuda_lib):
    args, o, lse = check(1, 8, 2, 64, "fp16", 16, [300], [5], [9] * 5, seed=11)
    q, k, v, ptable, _, table = args[:6]
    n = fa.paged_prefix_decode_workspace_size(5, 1, 8, 2, 64, 16, 1, ptable.shape[1], table.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fa.paged_prefix_decode(*args, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    for t in got:
        owner = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert owner == [side.cuda_stream]
    with pytest.raises(_lib.FAError) as e:
        fa.paged_prefix_decode(*args, workspace=ws[: n - 16])
    assert e.value.status == _lib.FA_ERR_SCRATCH_TOO_SMALL


def test_refusals(cuda_lib):
    q, k, v, ptable, plens, table, lens, starts = args = setup(1, 4, 2, 64, "fp16", 16, [40, 20], [1, 1], [9, 3], 1)
    fa.paged_prefix_decode(*args)
    for err, i, x in ((TypeError, 3, ptable.long()), (TypeError, 0, q.bfloat16()), (ValueError, 4, plens[:1]),
                      (ValueError, 5, table[:1]), (ValueError, 6, lens[:1]), (ValueError, 7, starts[:2]), (ValueError, 7, None),
                      (TypeError, 7, [0, 1, 2]), (ValueError, 3, ptable[0]), (ValueError, 1, k[:, :, :, :32])):
        with pytest.raises(err):
            fa.paged_prefix_decode(*args[:i], x, *args[i + 1:])
    with pytest.raises(_lib.FAError) as e:
        fa.paged_prefix_decode(q.expand(2, 70, 4, 64).contiguous(), *args[1:])
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    fa.check_device_error()
