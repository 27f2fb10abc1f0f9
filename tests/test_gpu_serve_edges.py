"""Calls of the serving operators at the edges of what their header allows, on the GPU against float64."""
import math

import pytest
import torch

import gated_delta_rule_linear_gb300 as la
import servelib as ref
from layerlib import hold
from test_gpu_serve import BF, F32, NAN, check_attn, ints, rand, some_parents, up

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("n,H,Hk,d,dtype,pages,length", [
    # just below 2^36 (bfloat16), 2^35 and 2^34 (float32) places of all parts
    (31, 1, 1, 64, BF, 2047, 70), (4, 32, 2, 128, BF, 2047, 900), (2, 96, 2, 256, BF, 2047, 5),
    (15, 4, 1, 128, F32, 2047, 3000), (7, 4, 1, 256, F32, 2047, 40), (7, 8, 1, 256, F32, 2047, 400),
    (3, 16, 1, 256, F32, 2047, 40),
    # of larger tables no more than 2^31 - 2^16 places of a sequence count
    (1, 4, 2, 128, BF, 1 << 20, 2 ** 31 - 1), (2, 8, 1, 256, F32, 1 << 20, 700),
])
def test_attn_of_the_largest_tables(n, H, Hk, d, dtype, pages, length):
    """Tables of pages that are not there (of 2^20 places each), as large as the header allows them: no place, no result."""
    page = 1 << 20
    q = torch.ones(n, H, d, dtype=dtype, device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.full((n, H), 7.0, device="cuda")
    table = torch.full((n, pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), length, dtype=torch.int32, device="cuda")
    rc = la.la_paged_attn(q, None, None, o, lse, table, lens, n, H, Hk, d, page, 0, pages, pages, 0, 0, 0.125, H * d,
                          page * Hk * d, la.LA_F32 if dtype is F32 else 0, torch.cuda.current_stream().cuda_stream)
    assert rc == la.CONSTANTS["LA_OK"], la.la_last_error()
    assert torch.equal(o, torch.zeros_like(o)) and bool((lse == -ref.INF).all())


@pytest.mark.parametrize("dtype,lens,H,Hk,d,page,window", [
    # bfloat16, 9 to 16 heads a key head, and more, in blocks of 16
    (BF, [0, 1, 64, 65, 700], 18, 2, 256, 16, 0), (BF, [513, 40, 3], 16, 1, 256, 20, 0), (BF, [2000], 24, 2, 256, 64, 1500),
    (BF, [9000, 17], 17, 1, 256, 128, 0), (BF, [300, 70, 1], 10, 1, 64, 7, 33), (BF, [5000], 33, 1, 64, 64, 0),
    (BF, [4000, 0, 12], 13, 1, 128, 16, 0),
    # float32, 5 to 8 heads, and more, in blocks of 8
    (F32, [0, 1, 16, 17, 700], 10, 2, 256, 16, 0), (F32, [513, 40, 3], 8, 1, 256, 20, 0), (F32, [2000], 12, 2, 256, 3, 1500),
    (F32, [5000, 17], 9, 1, 256, 128, 0), (F32, [300, 70, 1], 7, 1, 64, 7, 33), (F32, [4000, 0, 12], 17, 1, 128, 16, 0),
])
def test_attn_of_blocks_of_heads(dtype, lens, H, Hk, d, page, window):
    """Key heads with more queries than fill a small block: full and ragged blocks, whole parts and split ones."""
    gen = torch.Generator().manual_seed(H + d)
    table, pages = ref.make_tables(lens, page, gen)
    q = rand(gen, len(lens), H, d, dtype=dtype)
    kc, vc = (rand(gen, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    check_attn(q, kc, vc, table, lens, window)
    check_attn(q, kc, vc, table, lens, window, max_len=max(lens))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,share", [(64, 12), (128, 12), (256, 12), (256, 6)])
def test_attn_of_blocks_of_heads_leaves_out_what_is_not_there(dtype, d, share):
    """NaN and infinity behind the length, in front of the window and in pages that nobody has."""
    gen = torch.Generator().manual_seed(d + share)
    lens, page, Hk, window = [50, 49, 0, 400, 64], 16, 2, 37
    table, pages = ref.make_tables(lens, page, gen)
    q = rand(gen, len(lens), Hk * share, d, dtype=dtype)
    kc, vc = (rand(gen, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    used = torch.zeros(pages, page, dtype=torch.bool)
    for s, L in enumerate(lens):
        for p in range(max(L - window, 0), L):
            used[int(table[s, p // page]), p % page] = True
    kc[~used], vc[~used] = NAN, ref.INF
    check_attn(q, kc, vc, table, lens, window)
    check_attn(q, kc, vc, table, lens, window, max_len=400)


@pytest.mark.parametrize("dtype,share,d,n,top", [(BF, 16, 256, 150, 90), (BF, 11, 64, 330, 90), (F32, 8, 256, 160, 60),
                                                 (F32, 6, 128, 160, 100)])
def test_attn_of_blocks_of_heads_of_many_short_sequences(dtype, share, d, n, top):
    """Several parts for each CTA, of a unit or two, some of the sequences empty."""
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, top + 1, (n,), generator=gen).tolist()
    lens[0], lens[1], lens[-1] = 0, top, 0
    table, pages = ref.make_tables(lens, 16, gen)
    q = rand(gen, n, 4 * share, d, dtype=dtype)
    kc, vc = (rand(gen, pages, 16, 4, d, dtype=dtype) for _ in range(2))
    check_attn(q, kc, vc, table, lens)
    check_attn(q, kc, vc, table, lens, max_len=top)


# --------------------------------------------------------------- selection

@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_short_rows_at_every_alignment(dtype):
    """Rows that end in the first 16 bytes of a part or right behind a part, the first one at any element of 16 bytes: all
    granules behind them are nobody's, and nothing of memory is asked for there."""
    for first in range(16 // dtype.itemsize):
        for V in (1, 2, 7, 9, 255, 256, 257, 513):
            gen = torch.Generator().manual_seed(first + V)
            flat = (3 * torch.randn(first + 2 * V, generator=gen)).to(dtype)
            logits, scores, K = flat[first:].view(1, 2, V), torch.tensor([[-1.0, -1.25]]), min(3, 2 * V)
            c = ref.candidates(logits, scores)
            assert ref.nearest(c, K) > 1e-5
            want = ref.selection(c, K)
            best, parent, token = la.beam_select(flat.cuda()[first:].view(1, 2, V), scores.cuda(), K)
            assert torch.equal(parent.cpu(), want[1]) and torch.equal(token.cpu(), want[2])
            hold(best, want[0], ref.select_bound(want[0]), "scores")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [702, 5029, 33012])
def test_select_scores_about_the_log_of_the_sum(V, dtype):
    """A beam of V equal logits whose score is log V rounded up in float32, against one that has ended: its best is what the
    rounding added, 2.2e-7 to 4.4e-7, the other's 0.45 or 1.55 times that. The sum is V, its log good to 1e-8."""
    gain = float(torch.tensor(math.log(V))) - math.log(V)
    assert 2e-7 < gain < 4.5e-7
    logits = torch.zeros(1, 2, V, dtype=dtype).cuda()
    for live in (0, 1):
        for other in (0.45 * gain, 1.55 * gain):
            scores, done = torch.full((1, 2), other), torch.ones(1, 2, dtype=torch.bool)
            scores[0, live], done[0, live] = math.log(V), False
            best, parent, token = la.beam_select(logits, scores.cuda(), 1, done=done.cuda(), eos=V // 2)
            want = (live, 0, gain) if other < gain else (1 - live, V // 2, other)
            assert (int(parent), int(token)) == want[:2]
            assert abs(float(best) - want[2]) < 1e-8


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [700, 5003, 50257, 160001])
def test_select_sums_of_one_large_and_many_equal_logits(V, dtype):
    """Roundings that are the same in every term, and do not average out. A term is off by 2^-22 (its exponential) and, at a
    distance a below the largest, by a (2^-23 + 2^-26): the difference, its product with log2 e and that constant. It is
    scaled to the row's largest once at most (expf, 2^-22), and summed in pairs over six levels of 2^-24; the score is
    rounded once."""
    gen = torch.Generator().manual_seed(V)
    rows = torch.linspace(4.9, 10.6, 24).to(dtype)
    logits = (-rows)[None, :, None].expand(1, -1, V).clone()
    at = torch.randint(0, V, (24,), generator=gen)
    logits[0, torch.arange(24), at] = 0.0
    a = rows.double()
    want = -torch.log1p((V - 1) * torch.exp(-a))
    bound = 2.0 ** -22 * 3.5 + a * (2.0 ** -23 + 2.0 ** -26) + 2.0 ** -24 * want.abs() + 1e-8
    best, parent, token = la.beam_select(logits[0][:, None].contiguous().cuda(), torch.zeros(24, 1).cuda(), 1)
    assert torch.equal(token.cpu()[:, 0], at.int()) and not bool(parent.any())
    hold(best[:, 0], want, bound, "scores")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_of_both_zeros(dtype):
    """Scores of +0 and -0 are equal, of ended beams and of beams with one token."""
    zeros = torch.tensor([[-0.0, 0.0, -0.0, 0.0, 0.0, -0.0]])
    one = torch.zeros(1, 6, 1, dtype=dtype)
    one[0, ::2] = -0.0
    done = torch.tensor([[True, False, True, False, True, True]])
    for d in (torch.ones(1, 6, dtype=torch.bool), None, done):
        for K in (1, 3, 6):
            best, parent, token = la.beam_select(one.cuda(), zeros.cuda(), K, done=None if d is None else d.cuda())
            assert parent.tolist() == [list(range(K))] and not bool(token.any()) and bool((best == 0).all())
    logits = torch.full((1, 6, 300), -1.0, dtype=dtype)
    best, parent, token = la.beam_select(logits.cuda(), zeros.cuda(), 6, done=torch.ones(1, 6, dtype=torch.bool).cuda(), eos=7)
    assert parent.tolist() == [list(range(6))] and token.tolist() == [[7] * 6] and bool((best == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,W,K", [(40, 6, 32), (60, 32, 32), (300, 12, 32), (3001, 8, 24)])
def test_select_of_equal_candidates_of_other_scores(V, W, K, dtype):
    """Beams with the same logits, multiples of 1/4, and whole scores: many candidates are equal, as a score more makes up for
    four quarters of a logit. They come in the order of w*V + v, also where one logit has nearly all of the sum, whose log
    has bits of any weight then."""
    for seed in range(24):
        gen = torch.Generator().manual_seed(seed)
        row = -0.25 * torch.randint(0, 60, (V,), generator=gen).double()
        if seed % 2:
            row -= 5.0 + seed / 4
            row[seed] = 0.0
        scores = torch.randint(0, 30, (W,), generator=gen).double()
        c = (scores[:, None] + row).flatten()  # without the log, which is one for all
        at = torch.sort(-c, stable=True)[1][:K]
        best, parent, token = la.beam_select(row.to(dtype).expand(1, W, V).contiguous().cuda(), scores[None].float().cuda(), K)
        assert parent.cpu()[0].tolist() == (at // V).tolist() and token.cpu()[0].tolist() == (at % V).tolist()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_of_ended_beams_without_a_score(dtype):
    """All their candidates are -infinity, eos like the others, and come in the order of the index; with the eos in front of,
    among and behind the first K tokens."""
    for V, K in ((349, 21), (5, 10), (9000, 32), (40, 1)):
        logits = torch.zeros(4, 3, V, dtype=dtype)
        scores = torch.tensor([[-ref.INF] * 3, [NAN, ref.INF, -ref.INF], [-ref.INF, -2.0, -ref.INF], [-1.0, NAN, -3.0]])
        done = torch.tensor([[True] * 3, [True] * 3, [True] * 3, [True, True, False]])
        for eos in (0, V // 2, V - 1):
            want = ref.selection(ref.candidates(logits, scores, done, eos), K)
            best, parent, token = la.beam_select(*up(logits, scores), K, done=done.cuda(), eos=eos)
            assert torch.equal(parent.cpu(), want[1]) and torch.equal(token.cpu(), want[2])
            assert torch.equal(best.cpu() == -ref.INF, want[0] == -ref.INF)


def test_numbers_that_an_int_does_not_hold_are_refused():
    """2^32 + 5 is not 5."""
    far = 2 ** 32 + 5
    logits, scores = torch.zeros(1, 2, 50, device="cuda"), torch.zeros(1, 2, device="cuda")
    done = torch.ones(1, 2, dtype=torch.bool, device="cuda")
    for kw in (dict(eos=far, done=done), dict(eos=5 - 2 ** 32, done=done), dict(K=far)):
        with pytest.raises(ValueError, match="below 2"):
            la.beam_select(logits, scores, **kw)
    q, cache = torch.zeros(1, 2, 64, dtype=BF, device="cuda"), torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda")
    table, lens = ints([[0, 1]]).cuda(), ints([30]).cuda()
    for kw in (dict(window=far), dict(max_len=far), dict(window=-(2 ** 40))):
        with pytest.raises(ValueError, match="below 2"):
            la.paged_attn(q, cache, cache, table, lens, **kw)
    for kw in (dict(window=-1), dict(max_len=-1)):
        with pytest.raises(la.LAError):
            la.paged_attn(q, cache, cache, table, lens, **kw)
    with pytest.raises(la.LAError):
        la.beam_select(logits, scores, eos=50, done=done)


# -------------------------------------------------------------- reordering

@pytest.mark.parametrize("layers", [0, 1])
@pytest.mark.parametrize("token", [0, 128])
def test_cache_of_no_layers_or_no_bytes(layers, token):
    """The table follows the parents; caches of no layers, or of tokens without bytes, stay as they are. (One layer of
    tokens with bytes: the copies of the open pages that the others leave out.)"""
    gen = torch.Generator().manual_seed(layers + token)
    B, W, page = 2, 4, 8
    lens = [5] * W + [21] * W
    table, pages = ref.make_tables([x + 1 for x in lens], page, gen)
    parent = some_parents(gen, B, W)
    kc, vc = (rand(gen, 1, pages, page, 1, 64, dtype=BF) for _ in range(2))
    want_t, want_k, want_v = table.clone(), kc.clone(), vc.clone()
    for i, j in enumerate(ref.moved(list(range(B * W)), parent, W)):
        full, fill = divmod(lens[i], page)
        want_t[i, :full] = table[j, :full]
        if layers and token:
            mine, theirs = int(table[i, full]), int(table[j, full])
            want_k[:, mine, :fill], want_v[:, mine, :fill] = kc[:, theirs, :fill], vc[:, theirs, :fill]
    gk, gv, gt, gl, gp = up(kc, vc, table, ints(lens), parent)
    rc = la.la_beam_cache(gk, gv, gt, gl, gp, B, W, page, pages, table.shape[1], table.shape[1], layers, token, page * 128,
                          pages * page * 128, torch.cuda.current_stream().cuda_stream)
    assert rc == la.CONSTANTS["LA_OK"], la.la_last_error()
    assert torch.equal(gt.cpu(), want_t) and torch.equal(gk.cpu(), want_k) and torch.equal(gv.cpu(), want_v)
    if layers == 0:
        none = torch.zeros(0, pages, page, 1, token // 2, dtype=BF, device="cuda")
        got = table.cuda()
        la.beam_cache(none, none.clone(), got, gl, gp, layered=True)
        assert torch.equal(got.cpu(), want_t)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 3)])
@pytest.mark.parametrize("order", ["layers inside pages", "pages inside layers", "one page", "one layer"])
def test_cache_in_strided_pools(order, dtype, d):
    """Keys and values of all layers in one pool, layers in front of or behind the pages, with room between them; what is not
    the open pages' stays as it is. d = 3: 4 bytes at a time."""
    gen = torch.Generator().manual_seed(len(order) + d)
    B, W, page, Hk = 2, 3, 4, 2
    layers = 1 if order == "one layer" else 3
    lens = [6] * W + [11] * W
    table, pages = ref.make_tables([x + 1 for x in lens], page, gen)
    if order == "one page":
        table, pages, lens = torch.zeros(B * W, 1, dtype=torch.int32), 1, [3] * (B * W)
        table[1:] = -1
    inside = order == "layers inside pages"
    pool = rand(gen, *((pages, layers + 1) if inside else (layers, pages + 2)), 2, page, Hk, d, dtype=dtype)
    view = lambda p: (p[:, :layers].transpose(0, 1) if inside else p[:, :pages]).unbind(2)  # noqa: E731
    parent = some_parents(gen, B, W)
    want, want_t = pool.clone(), table.clone()
    wk, wv = view(want)
    kc, vc = view(pool)
    for i, j in enumerate(ref.moved(list(range(B * W)), parent, W)):
        full, fill = divmod(lens[i], page)
        want_t[i, :full] = table[j, :full]
        mine, theirs = int(table[i, full]), int(table[j, full])
        if mine >= 0 and theirs >= 0:
            wk[:, mine, :fill], wv[:, mine, :fill] = kc[:, theirs, :fill], vc[:, theirs, :fill]
    got = pool.cuda()
    gk, gv = view(got)
    gt = table.cuda()
    la.beam_cache(gk, gv, gt, *up(ints(lens), parent), layered=True)
    assert torch.equal(gt.cpu(), want_t) and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("inside", [False, True])
def test_states_in_strided_pools(inside):
    gen = torch.Generator().manual_seed(3)
    B, W, layers = 3, 5, 4
    pool = rand(gen, *((B * W + 2, layers + 1) if inside else (layers, B * W + 2)), 6, 10)
    view = lambda p: p[:, :layers].transpose(0, 1) if inside else p[:, :B * W]  # noqa: E731
    parent = some_parents(gen, B, W)
    want = pool.clone()
    view(want)[:, :B * W] = view(pool)[:, ref.moved(list(range(B * W)), parent, W)]
    got = pool.cuda()
    la.beam_states(view(got), parent.cuda(), layered=True)
    assert torch.equal(got.cpu(), want)


def test_pools_that_overlap_are_refused():
    one = torch.zeros(1, 8, 4, 2, 64, dtype=BF, device="cuda")
    parent, lens = ints([[0, 0]]).cuda(), ints([1, 1]).cuda()
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        la.beam_states(one.expand(3, -1, -1, -1, -1), parent, layered=True)
    with pytest.raises(ValueError, match="overlap"):
        la.beam_cache(one.expand(3, -1, -1, -1, -1), one.expand(3, -1, -1, -1, -1), table, lens, parent, layered=True)
    flat = torch.zeros(4096, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="overlap"):  # layers closer than a page
        la.beam_states(flat.as_strided((2, 4, 64), (32, 256, 1)), parent, layered=True)
    with pytest.raises(ValueError, match="dense"):
        la.beam_states(flat.as_strided((2, 4, 64), (1024, 256, 2)), parent, layered=True)
