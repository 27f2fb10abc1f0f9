"""Appending to a paged cache, attention over it, beam selection and reordering
on the GPU against float64."""
import pytest
import torch

import gated_delta_rule_linear_gb300 as la
import servelib as ref
from layerlib import hold

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def up(*ts):
    return [None if t is None else t.cuda() for t in ts]


def rand(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def spectrum(sections):
    return torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / max(s, 1)) for s in sections])


# ------------------------------------------------------------------ append

def check_append(gen, new, past, H, Hk, d, sections, page, dtype, interleaved=False, own_pos=False, cu=None, with_q=True,
                 spoil=None):
    """One append of new[s] tokens behind past[s] ones, everything else left as it was."""
    total = sum(new) + 3 if cu is not None or any(m != 1 for m in new) else len(new)
    lens = [a + b for a, b in zip(new, past)]
    if cu is None and total != len(new):
        cu = [sum(new[:i]) for i in range(len(new) + 1)]
    q, k, v = rand(gen, total, H, d, dtype=dtype) if with_q else None, *(rand(gen, total, Hk, d, dtype=dtype) for _ in range(2))
    table, pages = ref.make_tables([max(x, 1) for x in lens], page, gen)
    if spoil:
        spoil(table, lens)
    kc, vc = (rand(gen, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    freq = spectrum(sections) if sections else None
    pos = torch.randint(-3000, 100000, (total, len(sections)), generator=gen).to(torch.int32) if own_pos else None
    where = ref.places(cu, lens, total)
    pos_used = pos if own_pos else ints([[w[1] if w else 0] for w in where])
    gk, gv = up(kc, vc)
    out = torch.full((total, H, d), 7.0, dtype=dtype, device="cuda") if with_q else None
    got = la.cache_append(*up(q, k, v), gk, gv, *up(table, ints(lens)), freq=freq.cuda() if sections else None,
                          pos=pos.cuda() if own_pos else None, sections=sections or None, interleaved=interleaved,
                          cu_seqlens=ints(cu).cuda() if cu is not None else None, q_out=out)
    wk, sk = ref.turned(k, pos_used, freq, sections, interleaved)
    want_k, bound_k, want_v = kc.double(), torch.zeros_like(kc, dtype=torch.float64), vc.clone()
    for t, w in enumerate(where):
        at = w and ref.row_of(table, pages, page, *w)
        if at:
            want_k[at] = wk[t]
            bound_k[at] = ref.turn_bound(wk[t], sk[t], dtype)
            want_v[at] = v[t]
    hold(gk, want_k, bound_k, "k_cache")
    assert torch.equal(gv.cpu(), want_v)
    if with_q:
        assert got is out
        wq, sq = ref.turned(q, pos_used, freq, sections, interleaved)
        bound = ref.turn_bound(wq, sq, dtype)
        for t, w in enumerate(where):
            if w is None:
                wq[t], bound[t] = 7.0, 0.0
        hold(got, wq, bound, "q")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,past,H,Hk,d,sections,page", [
    ([1] * 5, [0, 7, 15, 16, 40], 4, 2, 128, [64], 16), ([1], [0], 1, 1, 64, [32], 1), ([3, 0, 70, 1], [5, 9, 0, 31], 3, 3, 96, [24], 20),
    ([1] * 4, [3, 2, 1, 0], 2, 1, 10, [3], 4), ([300, 200], [1, 70000], 8, 8, 256, [128], 64), ([2, 5], [0, 3], 2, 1, 7, [1, 0, 2], 3),
    ([33, 1, 1], [0, 12, 6], 2, 2, 128, [], 8),
])
def test_append(new, past, H, Hk, d, sections, page, interleaved, dtype):
    gen = torch.Generator().manual_seed(sum(new) + d)
    check_append(gen, new, past, H, Hk, d, sections, page, dtype, interleaved, own_pos=len(sections) > 1)
    check_append(gen, new, past, H, Hk, d, sections, page, dtype, interleaved, own_pos=bool(sections), with_q=False)


def test_append_of_padded_and_crossing_bounds():
    gen = torch.Generator().manual_seed(1)
    # the unused end of a batch holds zeros, or repeats the last bound; bounds outside [0, total]; overlapping ones
    for cu in ([0, 4, 9, 0, 0], [0, 4, 9, 9, 9], [-5, 4, 9, 100, 100], [0, 5, 2, 8, 8]):
        check_append(gen, [4, 5, 0, 0], [9, 3, 20, 5], 2, 1, 64, [32], 8, BF, cu=cu)
    lens = [2 ** 31 - 1, -(2 ** 31), 7]  # of three tokens each: no places, but for the last
    kc = rand(gen, 9, 8, 1, 64, dtype=BF).cuda()
    vc, k = kc.clone(), rand(gen, 9, 1, 64, dtype=BF).cuda()
    table = torch.arange(9, dtype=torch.int32).reshape(3, 3).cuda()
    before = kc.clone()
    la.cache_append(None, k, k, kc, vc, table, ints(lens).cuda(), cu_seqlens=ints([0, 3, 6, 9]).cuda())
    before[6, 4:7] = k[6:]
    assert torch.equal(kc, before) and torch.equal(vc, before)


def test_append_of_many_sequences():
    """More sequences than a block has threads, many of them empty, padded by zeros."""
    gen = torch.Generator().manual_seed(11)
    n = 1500
    new = [int(x) for x in torch.randint(0, 3, (n,), generator=gen)]
    cu = [sum(new[:i]) for i in range(n + 1)] + [0] * 500
    check_append(gen, new + [0] * 500, torch.randint(0, 40, (n + 500,), generator=gen).tolist(), 2, 1, 64, [32], 16, BF, cu=cu)


def test_append_without_places():
    gen = torch.Generator().manual_seed(2)

    def spoil(table, lens):
        lens[0], lens[1], lens[2] = 1, -4, 1000  # places in front of the cache and behind the table
        table[3, 0], table[4, 0] = -1, 10 ** 6
        lens[5] = 0

    check_append(gen, [3, 2, 4, 5, 1, 2], [4] * 6, 2, 2, 64, [32], 8, BF, spoil=spoil)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_from_a_fused_projection_into_interleaved_pools(dtype):
    """Strided inputs, and keys and values of two layers in one pool; unaligned rows go element by element."""
    gen = torch.Generator().manual_seed(3)
    n, H, Hk, d, page, pages = 9, 4, 2, 64, 16, 12
    for extra in (0, 1):
        fused = rand(gen, n, (H + 2 * Hk) * d + extra, dtype=dtype).cuda()
        q, k, v = (fused[:, a:b].unflatten(1, (-1, d)) for a, b in ((0, H * d), (H * d, (H + Hk) * d),
                                                                    ((H + Hk) * d, (H + 2 * Hk) * d)))
        pool = rand(gen, pages, 2, 2, page, Hk, d, dtype=dtype).cuda()
        before = pool.clone()
        table = torch.arange(n, dtype=torch.int32).reshape(n, 1).expand(n, 3).contiguous().cuda()[:, :1]
        lens = ints([1 + i for i in range(n)]).cuda()
        freq = spectrum([32]).cuda()
        got = la.cache_append(q, k, v, pool[:, 1, 0], pool[:, 1, 1], table, lens, freq=freq)
        pos = (lens.cpu() - 1)[:, None]
        wq, sq = ref.turned(q.cpu(), pos, freq.cpu(), [32], False)
        wk, sk = ref.turned(k.cpu(), pos, freq.cpu(), [32], False)
        hold(got, wq, ref.turn_bound(wq, sq, dtype), "q")
        at = torch.arange(n)
        hold(pool[at, 1, 0, at], wk, ref.turn_bound(wk, sk, dtype), "k")
        assert torch.equal(pool[at, 1, 1, at], v)
        pool[at, 1, :, at] = before[at, 1, :, at]
        assert torch.equal(pool, before)
        dense = q.contiguous()
        assert la.cache_append(dense, k, v, pool[:, 1, 0], pool[:, 1, 1], table, lens, freq=freq, q_out=dense) is dense
        assert torch.equal(dense, got)


# --------------------------------------------------------------- attention

def check_attn(q, kc, vc, table, lens, window=0, max_len=0, scale=None):
    d = q.shape[-1]
    o, lse = la.paged_attn(*up(q, kc, vc, table, ints(lens)), window=window, max_len=max_len, with_lse=True, scale=scale)
    want, wl, size, dots = ref.attention(q, kc, vc, table, lens, d ** -0.5 if scale is None else scale, window)
    L = max([min(x, window or x) for x in lens] + [0])
    hold(o, want, ref.attn_bound(want, size, dots, d, L, q.dtype), "o")
    empty = wl == -INF
    assert torch.equal(lse.cpu() == -INF, empty)
    hold(lse[~empty.cuda()], wl[~empty], ref.lse_bound(wl, dots, d, L)[~empty], "lse")
    return o, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,H,Hk,d,page,window", [
    ([1], 1, 1, 64, 16, 0), ([33], 8, 8, 64, 16, 0), ([0, 1, 2, 15, 16, 17, 63, 64, 65, 130], 4, 1, 128, 16, 0),
    ([700, 3, 0, 129], 16, 2, 128, 20, 0), ([513, 40], 6, 2, 256, 64, 0), ([300, 5, 90], 12, 1, 64, 7, 0),
    ([1000, 64, 1], 32, 1, 128, 1, 0), ([1000, 64, 1, 0], 4, 4, 128, 256, 100), ([257, 31], 8, 2, 256, 3, 1),
    ([64, 65, 66], 3, 3, 64, 64, 64), ([90, 77], 40, 2, 128, 16, 33), ([2000], 2, 1, 64, 100, 1999),
])
def test_attn(lens, H, Hk, d, page, window, dtype):
    gen = torch.Generator().manual_seed(len(lens) + H + d)
    table, pages = ref.make_tables(lens, page, gen)
    q = rand(gen, len(lens), H, d, dtype=dtype)
    kc, vc = (rand(gen, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    a, _ = check_attn(q, kc, vc, table, lens, window)
    b, _ = check_attn(q, kc, vc, table, lens, window, max_len=max(max(lens), 1))
    c, _ = check_attn(q, kc, vc, table, lens, window, max_len=1)  # a bound that does not hold costs time only
    assert a.shape == b.shape == c.shape


@pytest.mark.parametrize("n,Hk,top", [(1, 1, 20000), (1, 8, 9000), (3, 2, 5000), (40, 2, 900), (200, 1, 200), (1000, 1, 9)])
def test_attn_over_split_lengths(n, Hk, top):
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, top + 1, (n,), generator=gen).tolist()
    lens[0] = top
    table, pages = ref.make_tables(lens, 64, gen)
    q = rand(gen, n, 2 * Hk, 64, dtype=BF)
    kc, vc = (rand(gen, pages, 64, Hk, 64, dtype=BF) for _ in range(2))
    check_attn(q, kc, vc, table, lens)
    check_attn(q, kc, vc, table, lens, max_len=top, window=max(top // 3, 1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,H,Hk,d,page,window,top", [
    (130, 16, 8, 128, 16, 0, 70), (130, 8, 8, 256, 20, 0, 40), (130, 16, 8, 128, 64, 9, 200), (200, 16, 8, 128, 16, 0, 1),
    (70, 32, 32, 64, 16, 0, 90),
])
def test_attn_of_many_short_sequences(n, H, Hk, d, page, window, top, dtype):
    """Several parts for each CTA, of a unit or two, some of the sequences empty; without and with a longest length."""
    gen = torch.Generator().manual_seed(n + d)
    lens = torch.randint(0, top + 1, (n,), generator=gen).tolist()
    lens[0] = lens[-1] = lens[n // 2] = 0
    lens[1] = top
    table, pages = ref.make_tables(lens, page, gen)
    q = rand(gen, n, H, d, dtype=dtype)
    kc, vc = (rand(gen, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    check_attn(q, kc, vc, table, lens, window)
    check_attn(q, kc, vc, table, lens, window, max_len=top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_leaves_out_what_is_not_there(dtype):
    """Pages outside the pool, lengths behind the table; NaN and infinity behind the length, in front of the window,
    in pages that nobody has, and beside the heads of a page."""
    gen = torch.Generator().manual_seed(5)
    lens, page, Hk, d = [50, 49, 0, 80, 64], 16, 2, 128
    table, pages = ref.make_tables(lens, page, gen, width=5)
    q = rand(gen, len(lens), 4, d, dtype=dtype)
    kc, vc = (rand(gen, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    window = 37
    used = torch.zeros(pages, page, dtype=torch.bool)
    for s, L in enumerate(lens):
        for p in range(max(L - window, 0), L):
            used[int(table[s, p // page]), p % page] = True
    kc[~used], vc[~used] = NAN, INF
    check_attn(q, kc, vc, table, lens, window)
    table[0, 2], table[1, 1:], table[4] = -1, pages, -7  # a hole, a lost end, nothing at all
    check_attn(q, kc, vc, table, lens, window)
    lens[3], lens[1] = 10 ** 9, -5
    for p in range(80 - 37, 80):
        used[int(table[3, p // page]), p % page] = True
    o, lse = la.paged_attn(*up(q, kc, vc, table, ints(lens)), window=window, with_lse=True)
    want, wl, size, dots = ref.attention(q, kc, vc, table, lens, d ** -0.5, window)
    hold(o, want, ref.attn_bound(want, size, dots, d, window, dtype), "o")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_of_large_and_equal_scores(dtype):
    """Scores that overflow an exponential without their maximum, rising along the length; all scores equal."""
    gen = torch.Generator().manual_seed(6)
    L, page, d = 400, 16, 64
    table, pages = ref.make_tables([L], page, gen)
    q = rand(gen, 1, 2, d, dtype=dtype)
    kc, vc = (rand(gen, pages, page, 1, d, dtype=dtype) for _ in range(2))
    for i in range(L):
        kc[int(table[0, i // page]), i % page] *= 0.1 * i
    check_attn(q, kc, vc, table, [L], scale=1.0)
    check_attn(q, kc, vc, table, [L], scale=0.0)
    check_attn(q, kc, vc, table, [L], scale=-2.0)


def test_attn_offsets_past_32_bits():
    gen = torch.Generator().manual_seed(7)
    page, Hk, d = 64, 4, 128
    pages = (1 << 32) // (page * Hk * d) + 40  # 2^32 elements and more
    kc = torch.empty(pages, page, Hk, d, dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    lens = [150, 64]
    table = torch.full((2, 3), -1, dtype=torch.int32)
    table[0], table[1, 0] = ints([pages - 1, 3, pages - 20]), pages - 2
    small_k, small_v = (rand(gen, 4, page, Hk, d, dtype=BF) for _ in range(2))
    short = torch.full((2, 3), -1, dtype=torch.int32)
    short[0], short[1, 0] = ints([0, 1, 2]), 3
    for i, g in enumerate([pages - 1, 3, pages - 20, pages - 2]):
        kc[g], vc[g] = small_k[i].cuda(), small_v[i].cuda()
    q = rand(gen, 2, 8, d, dtype=BF)
    o, _ = la.paged_attn(*up(q), kc, vc, *up(table, ints(lens)))
    want, _ = la.paged_attn(*up(q, small_k, small_v, short, ints(lens)))
    assert torch.equal(o, want)
    k, v = (rand(gen, 2, Hk, d, dtype=BF).cuda() for _ in range(2))
    la.cache_append(None, k, v, kc, vc, *up(table, ints(lens)))
    assert torch.equal(kc[pages - 20, 149 - 128], k[0]) and torch.equal(vc[pages - 2, 63], v[1])


def test_attn_strides_streams_and_graphs():
    gen = torch.Generator().manual_seed(8)
    n, H, Hk, d, page = 6, 8, 2, 128, 32
    lens = [900, 1, 0, 333, 64, 2000]
    table, pages = ref.make_tables(lens, page, gen, width=70)
    fused = rand(gen, n, H * d + 16, dtype=BF).cuda()
    q = fused[:, :H * d].unflatten(1, (H, d))
    pool = rand(gen, pages, 2, page, Hk, d, dtype=BF).cuda()
    kc, vc = pool[:, 0], pool[:, 1]
    wide = torch.cat([table, table], 1).cuda()[:, :70]
    on = ints(lens).cuda()
    want, wl = la.paged_attn(q.contiguous(), kc.contiguous(), vc.contiguous(), table.cuda(), on, with_lse=True)
    got, lse = la.paged_attn(q, kc, vc, wide, on, with_lse=True)
    assert torch.equal(got, want) and torch.equal(lse, wl)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [[la.paged_attn(q, kc, vc, wide, on, stream=s)[0] for s in side] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for pair in outs for o in pair)
    # two captured calls, replayed on two streams beside eager ones, with other lengths than they were captured with
    graphs = []
    for _ in range(2):
        g, mine = torch.cuda.CUDAGraph(), on.clone()
        with torch.cuda.graph(g):
            o = la.paged_attn(q, kc, vc, wide, mine, max_len=2240)[0]
        graphs.append((g, mine, o))
    graphs[1][1].copy_(ints([5, 2000, 70, 0, 1, 640]))
    table_ok = torch.where(wide < 0, torch.zeros_like(wide), wide)
    wide.copy_(table_ok)
    first = la.paged_attn(q, kc, vc, wide, graphs[0][1])[0]
    second = la.paged_attn(q, kc, vc, wide, graphs[1][1])[0]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (g, _, _) in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        la.paged_attn(q, kc, vc, wide, on)
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2], first) and torch.equal(graphs[1][2], second)


# --------------------------------------------------------------- selection

def check_select(logits, scores, K, done=None, eos=0, gap=1e-5):
    c = ref.candidates(logits, scores, done, eos)
    assert ref.nearest(c, K) > gap  # no two beams' candidates that the sums' roundings could exchange
    want = ref.selection(c, K)
    best, parent, token = la.beam_select(*up(logits, scores), K, done=None if done is None else done.cuda(), eos=eos)
    assert torch.equal(parent.cpu(), want[1]) and torch.equal(token.cpu(), want[2])
    low = want[0] == -INF
    assert torch.equal(best.cpu() == -INF, low)
    hold(best[~low.cuda()], want[0][~low], ref.select_bound(want[0])[~low], "scores")


SELECT = [(1, 1, 1, 1), (1, 4, 3, 12), (2, 3, 50, 5), (3, 1, 4096, 1), (1, 2, 4097, 32), (2, 4, 32000, 4), (1, 8, 50257, 8),
          (4, 2, 10000, 2), (1, 32, 700, 32), (1, 3, 70001, 6), (1, 5, 8195, 17)]


def select_case(B, W, V, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return (3 * torch.randn(B, W, V, generator=gen)).to(dtype), torch.randn(B, W, generator=gen) - 9


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,W,V,K", SELECT)
def test_select(B, W, V, K, dtype):
    logits, scores = select_case(B, W, V, K, dtype, B + W + V + K)
    check_select(logits, scores, K)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_masked_done_and_worthless(dtype):
    logits, scores = select_case(3, 4, 9000, 6, dtype, 1)
    logits[torch.rand(logits.shape, generator=torch.Generator().manual_seed(2)) < 0.9] = -INF
    done = torch.zeros(3, 4, dtype=torch.bool)
    done[0, 1] = done[1] = True
    logits[0, 1] = NAN  # not read
    check_select(logits, scores, 6, done, eos=5)
    check_select(logits, scores, 6, done, eos=8999)
    check_select(logits, scores, 6, done, eos=0)
    # no token allowed, one token allowed, NaN, infinity, scores that are none
    logits, scores = select_case(6, 2, 300, 8, dtype, 3)
    logits[0], logits[1, :, 1:], logits[2, 0, 77], logits[3, 1, 5] = -INF, -INF, NAN, INF
    scores[4, 0], scores[4, 1], scores[5, 1] = -INF, NAN, INF
    check_select(logits, scores, 8)


def test_select_ties():
    """Equal logits, equal beams, both zeros, all equal: the lowest index first."""
    for V in (40, 5000, 12001):
        row = torch.randint(-4, 5, (V,), generator=torch.Generator().manual_seed(V)).float()
        for dtype in (BF, F32):
            logits = row.to(dtype).expand(2, 5, V).clone()
            logits[1] = 0.0
            logits[1, :, ::3] = -0.0
            scores = torch.zeros(2, 5)
            c = ref.candidates(logits, scores)
            want = ref.selection(c, 24)
            best, parent, token = la.beam_select(*up(logits, scores), 24)
            assert torch.equal(parent.cpu(), want[1]) and torch.equal(token.cpu(), want[2])


def test_select_first_step():
    """One beam with a score and the others without: all K from its row, of few parts or many; fewer tokens than K."""
    for W, V, K in ((4, 700, 32), (16, 2129, 32), (16, 20011, 16), (32, 5003, 32)):
        for dtype in (BF, F32):
            logits, scores = select_case(2, W, V, K, dtype, V + W)
            scores[:, 0] = 0.0
            scores[:, 1:] = -INF
            check_select(logits, scores, K)
            logits[1, :, 5:] = -INF
            check_select(logits, scores, K)


def test_select_rising_and_falling_rows():
    """Orders that put all of a row's best in one place."""
    for V in (4096, 20000):
        x = torch.arange(V, dtype=torch.float64) / 977
        logits = torch.stack([x, x.flip(0), x * 0.37, -x])[None].float()
        check_select(logits, torch.tensor([[-1.0, -2.1, -3.2, -4.3]]), 32, gap=1e-6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_masks_of_the_lowest_value(dtype):
    """Tokens masked by the type's lowest value instead of -infinity; rows of nothing else; the highest value."""
    logits, scores = select_case(4, 2, 3000, 6, dtype, 5)
    low = torch.finfo(dtype).min
    logits[0, :, 10:2900] = low
    logits[1, 0] = low
    logits[2] = low
    logits[2, 1, 7] = 0.0
    logits[3, 1, 100:103] = torch.finfo(dtype).max
    check_select(logits, scores, 6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_values_that_grow_along_the_row(dtype):
    """Sums whose later terms are far above the first ones, in every part of a row."""
    for V in (700, 2048, 13144):
        logits, scores = select_case(2, 4, V, 8, dtype, V)
        for period in (2, 128, 256, 1024):
            rising = (30.0 * ((torch.arange(V) // period) % 2)).to(dtype)
            check_select((logits + rising).to(dtype), scores, 8)


def test_select_rows_at_every_alignment():
    """Vocabularies and strides that put rows at any offset from 16 bytes; rows that are alike tie."""
    for dtype in (BF, F32):
        for V, ld in ((4099, 4099), (9001, 9003), (257, 259), (8, 9), (70005, 70005)):
            gen = torch.Generator().manual_seed(ld)
            store = (3 * torch.randn(6, ld, generator=gen)).to(dtype)
            store[3, :V] = store[1, :V]
            for first in (0, 1, 3):
                flat = torch.cat([torch.zeros(first, dtype=dtype), store.flatten()]).cuda()
                view = flat[first:].view(6, ld)[:, :V].unflatten(0, (2, 3))
                scores = torch.tensor([[0.0, -1.0, -2.0], [-1.0, -2.5, -1.0]])
                scores[1, 0] = scores[0, 1]
                K = min(8, V)
                best, parent, token = la.beam_select(view, scores.cuda(), K)
                c = ref.candidates(store[:, :V].unflatten(0, (2, 3)), scores)
                assert ref.nearest(c, K) > 1e-5
                want = ref.selection(c, K)
                assert torch.equal(parent.cpu(), want[1]) and torch.equal(token.cpu(), want[2])
                hold(best, want[0], ref.select_bound(want[0]), "scores")
        # a row and its copy at another alignment, in one request
        gen = torch.Generator().manual_seed(1)
        for V in (5001, 33333):
            row = (3 * torch.randn(V, generator=gen)).to(dtype)
            best, parent, token = la.beam_select(row.expand(1, 7, V).contiguous().cuda(), torch.zeros(1, 7).cuda(), 21)
            order = torch.sort(-row.double(), stable=True)[1][:4]
            assert token.cpu()[0].tolist() == [int(order[i // 7]) for i in range(21)]
            assert parent.cpu()[0].tolist() == [i % 7 for i in range(21)]


def test_select_strides_streams_and_graphs():
    gen = torch.Generator().manual_seed(4)
    padded = (3 * torch.randn(2, 4, 5008, generator=gen)).to(BF).cuda()
    scores = torch.randn(2, 4, generator=gen).cuda()
    for V in (5000, 5001):
        want = la.beam_select(padded[..., :V].contiguous(), scores, 4)
        got = la.beam_select(padded[..., :V], scores, 4)
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
        hold(got[0], want[0].double().cpu(), 2 * ref.select_bound(want[0].double().cpu()), "scores")
    want = la.beam_select(padded, scores, 8, eos=3)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [[la.beam_select(padded, scores, 8, eos=3, stream=s) for s in side] for _ in range(5)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = la.beam_select(padded, scores, 8, eos=3)
    outs.append([held])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for got in o for a, b in zip(got, want))


# -------------------------------------------------------------- reordering

def some_parents(gen, B, W):
    p = torch.randint(0, W, (B, W), generator=gen).to(torch.int32)
    stay = torch.rand(B, W, generator=gen) < 0.3
    return torch.where(stay, torch.arange(W, dtype=torch.int32), p)


@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8, 13, 16, 31, 32])
@pytest.mark.parametrize("shape,dtype", [((2, 64, 64), F32), ((5,), F32), ((3, 7), BF), ((33,), torch.int32)])
def test_states(W, shape, dtype):
    gen = torch.Generator().manual_seed(W)
    if dtype is BF:
        shape = (shape[0], shape[1] + 1)  # rows of multiples of 4 bytes
    B, layers = 3, 2
    rows = B * W + 4
    pool = (torch.randn(layers, rows, *shape, generator=gen) * 100).to(dtype)
    slots = torch.randperm(rows, generator=gen)[:B * W].to(torch.int32)
    parent = some_parents(gen, B, W)
    if W > 2:
        parent[0, 1], parent[1, 0], slots[W + 1], slots[2 * W + 2] = -1, W, -1, rows  # rows that stay, rows that are none
    want = pool.clone()
    at = [int(s) if 0 <= s < rows else None for s in slots]
    for i, j in zip(at, ref.moved(at, parent, W)):
        if i is not None:
            want[:, i] = pool[:, j]
    got = pool.cuda()
    assert la.beam_states(got, parent.cuda(), slots=slots.cuda(), layered=True) is got
    assert torch.equal(got.cpu(), want)
    one = pool[0].clone().cuda()
    la.beam_states(one, parent.cuda())
    plain = ref.moved(list(range(B * W)), parent, W)
    assert torch.equal(one.cpu()[:B * W], pool[0][plain]) and torch.equal(one.cpu()[B * W:], pool[0][B * W:])


def test_states_of_large_strided_rows():
    gen = torch.Generator().manual_seed(1)
    B, W = 2, 3
    pool = torch.randn(3, B * W + 1, 2, 100000, generator=gen).cuda()
    parent = some_parents(gen, B, W)
    want = pool.clone()
    order = ref.moved(list(range(B * W)), parent, W)
    want[:, :B * W, 1] = pool[:, order, 1]
    la.beam_states(pool[:, :, 1], parent.cuda(), layered=True)
    assert torch.equal(pool, want)


def check_cache(gen, B, W, lens, page, layers, Hk, d, dtype, parent, shared=True):
    flat = [x for x in lens for _ in range(W)]
    table, pages = ref.make_tables([x + 1 for x in flat], page, gen)
    if shared:  # full pages that earlier steps have made common to the beams
        for b, x in enumerate(lens):
            full = x // page
            table[b * W:(b + 1) * W, :full // 2] = table[b * W, :full // 2].clone()
    kc, vc = (rand(gen, layers, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    want_k, want_v, want_t = kc.clone(), vc.clone(), table.clone()
    order = ref.moved(list(range(B * W)), parent, W)
    for i, j in enumerate(order):
        full, fill = divmod(max(flat[i], 0), page)
        want_t[i, :full] = table[j, :full]
        mine, theirs = int(table[i, full]), int(table[j, full])
        want_k[:, mine, :fill], want_v[:, mine, :fill] = kc[:, theirs, :fill], vc[:, theirs, :fill]
    got = up(kc, vc, table)
    la.beam_cache(*got, *up(ints(flat), parent), layered=True)
    assert torch.equal(got[2].cpu(), want_t)
    assert torch.equal(got[0].cpu(), want_k) and torch.equal(got[1].cpu(), want_v)
    # what every beam reads now is what its parent had
    for i, j in enumerate(order):
        for p in range(max(flat[i], 0)):
            a, b = (int(t[s, p // page]) for t, s in ((got[2], i), (table, j)))
            assert torch.equal(got[0][:, a, p % page].cpu(), kc[:, b, p % page])


@pytest.mark.parametrize("W", [1, 2, 4, 7, 16, 32])
@pytest.mark.parametrize("dtype,Hk,d", [(BF, 2, 64), (F32, 1, 64), (BF, 1, 6)])
def test_cache(W, dtype, Hk, d):
    gen = torch.Generator().manual_seed(W)
    lens = [0, 5, 16, 37, 64]
    check_cache(gen, len(lens), W, lens, 16, 2, Hk, d, dtype, some_parents(gen, len(lens), W))
    check_cache(gen, len(lens), W, lens, 5, 1, Hk, d, dtype, torch.zeros(len(lens), W, dtype=torch.int32), shared=False)


def test_cache_of_what_is_not_there():
    """Lengths without an open page, pages outside the pool, parents outside the request: left as they are."""
    gen = torch.Generator().manual_seed(9)
    W, page = 3, 8
    table = torch.arange(9, dtype=torch.int32).reshape(3, 3).repeat_interleave(W, 0)
    table = table + torch.arange(9, dtype=torch.int32)[:, None] * 9
    table[4, 1], table[8, 1] = -1, 10 ** 6
    kc, vc = (rand(gen, 100, page, 1, 64) for _ in range(2))
    lens = [24] * 3 + [10] * 3 + [10] * 3
    parent = ints([[1, 0, 5], [1, 2, 0], [2, 2, -1]])
    got = up(kc, vc, table)
    la.beam_cache(*got, *up(ints(lens), parent))
    want_t, want_k, want_v = table.clone(), kc.clone(), vc.clone()
    want_t[0], want_t[1] = table[1], table[0]        # all pages full, no open one
    want_t[3, :1], want_t[4, :1], want_t[5, :1] = table[4, :1], table[5, :1], table[3, :1]
    want_t[6, :1], want_t[7, :1] = table[8, :1], table[8, :1]
    want_k[int(table[5, 1]), :2], want_v[int(table[5, 1]), :2] = kc[int(table[3, 1]), :2], vc[int(table[3, 1]), :2]
    assert torch.equal(got[2].cpu(), want_t) and torch.equal(got[0].cpu(), want_k) and torch.equal(got[1].cpu(), want_v)
    for far in (10 ** 9, -3):
        got = up(kc, vc, table)
        la.beam_cache(*got, *up(ints([far] * 9), ints([[0, 0, 0]] * 3)))
        want = table.clone()
        if far > 0:
            want = table[[0, 0, 0, 3, 3, 3, 6, 6, 6]]
        assert torch.equal(got[2].cpu(), want) and torch.equal(got[0].cpu(), kc)


def test_empty_calls():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    kc = z(2, 16, 1, 64)
    assert la.cache_append(z(0, 2, 64), z(0, 1, 64), z(0, 1, 64), kc, kc.clone(), i(0, 3), i(0)).shape == (0, 2, 64)
    assert la.paged_attn(z(0, 2, 64), kc, kc, i(0, 3), i(0))[0].shape == (0, 2, 64)
    assert float(la.paged_attn(z(3, 2, 64) + 1, kc, kc, i(3, 0), i(3) + 9)[0].abs().sum()) == 0
    none = z(0, 16, 1, 64)
    assert float(la.paged_attn(z(3, 2, 64) + 1, none, none, i(3, 2), i(3) + 9)[0].abs().sum()) == 0
    assert la.beam_select(z(0, 2, 9), z(0, 2, dtype=F32), 2)[0].shape == (0, 2)
    la.beam_states(z(4, 8, dtype=F32), i(0, 2))
    la.beam_cache(kc, kc.clone(), i(0, 3), i(0), i(0, 2))
    torch.cuda.synchronize()
