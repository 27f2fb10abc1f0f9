"""Packed retention on the GPU against the float64 recurrences: forward,
backward, single tokens."""
import pytest
import torch

import gated_delta_rule_linear_gb300 as la
from layerlib import (HALF, gammas, hold, packed_bound, retention, retention_bwd, starts, state_bound)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LENS = [[1], [128], [129], [300], [0, 5, 0, 127, 1, 260, 0], [64, 65, 63, 1, 1, 2], [0, 0], [1100]]


def draw(lens, H, Hk, dk, dv, dtype, seed=0, extra=0):
    gen = torch.Generator().manual_seed(seed)
    N = sum(lens) + extra
    n = lambda *s: torch.randn(*s, generator=gen) * dk ** -0.5  # noqa: E731
    q, k, v, dO = n(N, Hk, dk), n(N, Hk, dk), n(N, H, dv), n(N, H, dv)
    S0, dS = n(len(lens), H, dk, dv), n(len(lens), H, dk, dv)
    return [t.to(dtype) for t in (q, k, v, dO)] + [S0, dS]


def cu(lens):
    return torch.tensor(starts(lens), dtype=torch.int32).cuda()


def up(*ts):
    return [None if t is None else t.cuda() for t in ts]


def done():
    assert la.la_stream_status(torch.cuda.current_stream().cuda_stream) == 0


def check_fwd(lens, H, Hk, dk, dv, dtype, decay=True, init=True, g=None, max_len=0, seed=0):
    q, k, v, _, S0, _ = draw(lens, H, Hk, dk, dv, dtype, seed)
    S0 = S0 if init else None
    g = gammas(H, decay) if g is None else g
    dq, dk_, dv_, dg, dS = up(q, k, v, g, S0)
    o, S = la.packed_fwd(dq, dk_, dv_, cu(lens), "linear" if g is None else "retnet", g=dg, S0=dS, max_len=max_len)
    done()
    want, Sw = retention(q, k, v, g, lens, S0)
    size, Ss = retention(q, k, v, g, lens, S0, positive=True)
    T = max(lens)
    hold(o, want, packed_bound(want, size, T, dtype), "o")
    hold(S, Sw, state_bound(Ss, T, dtype), "S_final")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward_lengths(lens, dtype):
    check_fwd(lens, 2, 2, 128, 128, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 2)])
def test_forward_heads(dk, dv, H, Hk, dtype):
    check_fwd([200, 7, 131], H, Hk, dk, dv, dtype, seed=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_without_state_or_decay(dtype):
    check_fwd([140, 260], 2, 1, 64, 128, dtype, decay=False, init=False, seed=2)
    check_fwd([140, 260], 2, 1, 64, 128, dtype, decay=False, init=True, seed=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_decays(dtype):
    # from none to none left: the powers under- and never overflow
    g = torch.tensor([0.0, -0.5, -5.0, -90.0, -1e4, float("-inf")])
    check_fwd([300, 1, 70], 6, 6, 64, 64, dtype, g=g, seed=3)


def test_slow_decay_over_a_long_sequence():
    # gamma^n over thousands of tokens: a rounded factor applied again and again would show
    g = torch.tensor([-2.0 ** -13])
    check_fwd([6000], 1, 1, 64, 64, BF, g=g, seed=4)
    check_fwd([6000], 1, 1, 64, 64, F32, g=g, seed=4)


@pytest.mark.parametrize("max_len", [0, 1, 5000, 1 << 30])
def test_max_len_is_a_hint(max_len):
    check_fwd([2500, 3, 0, 900], 2, 1, 64, 64, BF, max_len=max_len, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slots(dtype):
    # pool rows: used, twice the same, out of range on both sides, and an empty sequence's
    lens, H, dk, dv = [130, 5, 40, 0, 17, 64], 2, 64, 128
    q, k, v, _, S0, _ = draw(lens, H, 1, dk, dv, dtype, 6)
    pool = torch.randn(7, H, dk, dv, generator=torch.Generator().manual_seed(9))
    slots = torch.tensor([4, -1, 7, 2, 4, 0], dtype=torch.int32)
    alive = [0, 3, 5]  # sequences that own their slot
    start = torch.stack([pool[slots[s]] if s in alive else torch.zeros(H, dk, dv) for s in range(6)])
    g = gammas(H)
    for alias in (True, False):
        dev = pool.cuda()
        dst = dev if alias else torch.full_like(dev, 7.0)
        o, S = la.packed_fwd(*up(q, k, v), cu(lens), "retnet", g=g.cuda(), S0=dev, S_final=dst, slots=slots.cuda())
        done()
        assert S is dst
        want, Sw = retention(q, k, v, g, lens, start)
        size, Ss = retention(q, k, v, g, lens, start, positive=True)
        hold(o, want, packed_bound(want, size, 130, dtype), "o")
        for s in alive:
            hold(S[slots[s]], Sw[s], state_bound(Ss[s], 130, dtype), f"state of {s}")
        for row in (1, 3, 5, 6):
            assert torch.equal(S[row].cpu(), pool[row] if alias else torch.full_like(pool[row], 7.0))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_a_fused_projection_and_rows_behind(dtype):
    # q, k, v read where a fused projection left them; rows behind the last sequence stay as they were,
    # and what they hold (NaN) reaches nothing
    lens, H, Hk, dk, dv, extra = [77, 140], 4, 2, 64, 128, 90
    q, k, v, _, S0, _ = draw(lens, H, Hk, dk, dv, dtype, 7, extra)
    N = sum(lens)
    for t in (q, k, v):
        t[N:] = float("nan")
    fused = torch.cat([t.reshape(len(t), -1) for t in (q, k, v)], 1).cuda()
    a, b = Hk * dk, 2 * Hk * dk
    fq, fk, fv = fused[:, :a].unflatten(1, (Hk, dk)), fused[:, a:b].unflatten(1, (Hk, dk)), fused[:, b:].unflatten(1, (H, dv))
    o = torch.full((N + extra, H, dv), 3.0, dtype=dtype, device="cuda")
    g = gammas(H)
    la.packed_fwd(fq, fk, fv, cu(lens), "retnet", g=g.cuda(), S0=S0.cuda(), o=o)
    done()
    assert (o[N:] == 3.0).all()
    want, _ = retention(q[:N], k[:N], v[:N], g, lens, S0)
    size, _ = retention(q[:N], k[:N], v[:N], g, lens, S0, positive=True)
    hold(o[:N], want, packed_bound(want, size, 140, dtype), "o")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_neighbours_nan_stays_there(dtype):
    lens, H = [100, 150, 60], 2
    q, k, v, _, S0, _ = draw(lens, H, H, 64, 64, dtype, 8)
    clean = la.packed_fwd(*up(q, k, v), cu(lens), "retnet", g=gammas(H).cuda(), S0=S0.cuda())
    for t in (q, k, v):
        t[100:250] = float("nan")
    S0[1] = float("inf")
    o, S = la.packed_fwd(*up(q, k, v), cu(lens), "retnet", g=gammas(H).cuda(), S0=S0.cuda())
    done()
    for s, rows in ((0, slice(0, 100)), (2, slice(250, 310))):
        assert torch.equal(o[rows], clean[0][rows]) and torch.equal(S[s], clean[1][s])


def check_bwd(lens, H, Hk, dk, dv, dtype, decay=True, states=True, g=None, max_len=0, seed=0):
    q, k, v, dO, S0, dS = draw(lens, H, Hk, dk, dv, dtype, seed)
    if not states:
        S0 = dS = None
    g = gammas(H, decay) if g is None else g
    got = la.packed_bwd(*up(q, k, v, dO), cu(lens), "linear" if g is None else "retnet", g=None if g is None else g.cuda(),
                        S0=None if S0 is None else S0.cuda(), dS_final=None if dS is None else dS.cuda(), max_len=max_len)
    done()
    want = retention_bwd(q, k, v, dO, g, lens, S0, dS)
    size = retention_bwd(q, k, v, dO, g, lens, S0, dS, positive=True)
    T = max(lens)
    for name, a, b, c in zip(("dq", "dk", "dv"), got, want, size):
        hold(a, b, packed_bound(b, c, T, dtype), name)
    hold(got[3], want[3], state_bound(size[3], T, dtype), "dS0")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_backward_lengths(lens, dtype):
    check_bwd(lens, 2, 2, 128, 128, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 2)])
def test_backward_heads(dk, dv, H, Hk, dtype):
    check_bwd([200, 7, 131], H, Hk, dk, dv, dtype, seed=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_without_states_or_decay(dtype):
    check_bwd([140, 260], 2, 1, 64, 128, dtype, decay=False, states=False, seed=2)
    check_bwd([140, 260], 2, 2, 128, 64, dtype, decay=False, seed=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_strong_decays(dtype):
    check_bwd([300, 1, 70], 6, 6, 64, 64, dtype, g=torch.tensor([0.0, -0.5, -5.0, -90.0, -1e4, float("-inf")]), seed=3)


@pytest.mark.parametrize("max_len", [0, 1, 3000])
def test_backward_of_long_sequences(max_len):
    check_bwd([2500, 3, 0, 900], 2, 1, 64, 64, BF, max_len=max_len, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_rows_of_no_sequence(H, Hk, dtype):
    # tokens in front of the first sequence and behind the last: read by nobody, written by nobody
    front, lens, back, dk, dv = 37, [150, 0, 90], 45, 64, 64
    q, k, v, dO, S0, dS = draw(lens, H, Hk, dk, dv, dtype, 23, front + back)
    rows = slice(front, front + sum(lens))
    for t in (q, k, v, dO):
        t[:front] = t[front + sum(lens):] = float("nan")
    c = cu(lens) + front
    g = gammas(H)
    N = len(q)
    args = up(q, k, v, dO)
    outs = [torch.full((N, Hk, dk), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
    outs += [torch.full((N, H, dv), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
    dS0 = torch.empty(3, H, dk, dv, device="cuda")
    mode = la.MODE_IDS["retnet"] | (la.LA_F32 if dtype == F32 else 0)
    ld = (Hk * dk, Hk * dk, H * dv)
    stream = torch.cuda.current_stream().cuda_stream
    dg, dS0_in, dS_in = up(g, S0, dS)
    assert la.la_packed_bwd(*args[:3], dg, args[3], dS0_in, dS_in, outs[0], outs[1], outs[2], dS0, c, 3, N, 0, H, Hk, dk,
                            dv, *ld, mode, stream) == 0
    assert la.la_packed_fwd(*args[:3], dg, outs[3], dS0_in, None, c, None, 3, N, 0, 3, H, Hk, dk, dv, *ld, mode, stream) == 0
    done()
    inner = [t[rows] for t in (q, k, v, dO)]
    want = retention_bwd(*inner, g, lens, S0, dS)[:3] + (retention(*inner[:3], g, lens, S0)[0],)
    size = retention_bwd(*inner, g, lens, S0, dS, positive=True)[:3] + (
        retention(*inner[:3], g, lens, S0, positive=True)[0],)
    for name, t, a, b in zip(("dq", "dk", "dv", "o"), outs, want, size):
        assert (t[:front] == 5.0).all() and (t[front + sum(lens):] == 5.0).all(), name
        hold(t[rows], a, packed_bound(a, b, 150, dtype), name)


def test_backward_against_differences():
    # the linear map's gradient against the forward itself, in float32: L = <dO, o> + <dS, S_final> is
    # linear in each input, so a step of any size is exact up to rounding
    lens, H = [37, 70], 2
    q, k, v, dO, S0, dS = draw(lens, H, 1, 64, 64, F32, 10)
    g = gammas(H).cuda()
    base = dict(zip("qkvS", up(q, k, v, S0)))

    def loss(**kw):
        x = {**base, **kw}
        o, S = la.packed_fwd(x["q"], x["k"], x["v"], cu(lens), "retnet", g=g, S0=x["S"])
        return (o.double() * dO.cuda()).sum() + (S.double() * dS.cuda()).sum()

    grads = la.packed_bwd(*up(q, k, v, dO), cu(lens), "retnet", g=g, S0=S0.cuda(), dS_final=dS.cuda())
    gen = torch.Generator().manual_seed(11)
    for name, grad in zip("qkvS", grads):
        step = torch.randn(base[name].shape, generator=gen).cuda()
        diff = loss(**{name: base[name] + step}) - loss(**{name: base[name] - step})
        want = 2 * (grad.double() * step).sum()
        # two losses of about 1e3 float32 products and sums each: 2^-24 of their absolute sums
        size = (grad.double().abs() * step.abs()).sum() + loss().abs()
        assert (diff - want).abs() <= 2.0 ** -14 * size, (name, diff, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("n,H,Hk", [(1, 1, 1), (5, 4, 2), (33, 3, 3)])
def test_step(n, H, Hk, dk, dv, dtype):
    q, k, v, _, _, _ = draw([n], H, Hk, dk, dv, dtype, 12)
    gen = torch.Generator().manual_seed(13)
    pool = torch.randn(n + 2, H, dk, dv, generator=gen)
    slots = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32)
    for g in (gammas(H), None):
        S = pool.cuda()
        o = la.packed_step(*up(q, k, v), S, "linear" if g is None else "retnet", g=None if g is None else g.cuda(),
                           slots=slots.cuda())
        done()
        want, Sw = retention(q, k, v, g, [1] * n, pool[slots.long()])
        size, Ss = retention(q, k, v, g, [1] * n, pool[slots.long()], positive=True)
        hold(o, want, HALF[dtype] * want.abs() + 2.0 ** -16 * size, "o")
        hold(S.cpu()[slots.long()], Sw, 2.0 ** -22 * Ss, "S")
        rest = [r for r in range(n + 2) if r not in slots.tolist()]
        assert torch.equal(S.cpu()[rest], pool[rest])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_padding_and_repeated_slots(dtype):
    # rows of one slot are one after the other; padding rows give zeros and touch nothing
    slots = torch.tensor([2, -1, 0, 2, 9, 0, 2], dtype=torch.int32)
    n, H, dk, dv = 7, 2, 64, 64
    q, k, v, _, _, _ = draw([n], H, 2, dk, dv, dtype, 14)
    pool = torch.randn(4, H, dk, dv, generator=torch.Generator().manual_seed(15))
    g, S = gammas(H), pool.cuda()
    o = la.packed_step(*up(q, k, v), S, "retnet", g=g.cuda(), slots=slots.cuda())
    done()
    for slot in (0, 2):
        rows = [i for i in range(n) if slots[i] == slot]
        args = (q[rows], k[rows], v[rows], g, [len(rows)], pool[slot:slot + 1])
        want, Sw = retention(*args)
        size, Ss = retention(*args, positive=True)
        hold(o[rows], want, HALF[dtype] * want.abs() + 2.0 ** -16 * size, f"o of slot {slot}")
        hold(S[slot], Sw[0], 2.0 ** -21 * Ss[0], f"S of slot {slot}")
    assert (o[[1, 4]] == 0).all()
    assert torch.equal(S[[1, 3]].cpu(), pool[[1, 3]])


def test_step_without_slots_and_with_strided_rows():
    n, H, d = 6, 2, 128
    q, k, v, _, S0, _ = draw([n], H, H, d, d, BF, 16)
    pool = torch.randn(n, H, d, d, generator=torch.Generator().manual_seed(17))
    fused = torch.cat([t.reshape(n, -1) for t in (q, k, v)], 1).cuda()
    parts = [fused[:, i * H * d:(i + 1) * H * d].unflatten(1, (H, d)) for i in range(3)]
    S, T = pool.cuda(), pool.cuda()
    o = la.packed_step(*parts, S, "linear")
    p = la.packed_step(*up(q, k, v), T, "linear", slots=torch.arange(n, dtype=torch.int32).cuda())
    done()
    assert torch.equal(o, p) and torch.equal(S, T)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_tokens(dtype):
    # a prompt through the forward, then single tokens: the same as the whole sequence
    n, H = 150, 2
    q, k, v, _, _, _ = draw([n], H, 1, 64, 128, dtype, 18)
    g = gammas(H)
    S = torch.zeros(3, H, 64, 128, device="cuda")
    slot = torch.tensor([1], dtype=torch.int32).cuda()
    dq, dk, dv = up(q, k, v)
    o = [la.packed_fwd(dq[:147], dk[:147], dv[:147], cu([147]), "retnet", g=g.cuda(), S0=S, S_final=S, slots=slot)[0]]
    for t in range(147, n):
        o.append(la.packed_step(dq[t:t + 1], dk[t:t + 1], dv[t:t + 1], S, "retnet", g=g.cuda(), slots=slot))
    done()
    want, Sw = retention(q, k, v, g, [n])
    size, Ss = retention(q, k, v, g, [n], positive=True)
    hold(torch.cat(o), want, packed_bound(want, size, n, dtype), "o")
    hold(S[1:2], Sw, state_bound(Ss, n, dtype), "S")
    assert (S[[0, 2]] == 0).all()


def test_streams_and_graphs():
    # two streams at once, and a captured call replayed on new inputs while an eager one uses the pool
    lens, H = [2000, 700, 1300], 2
    a = up(*draw(lens, H, 1, 64, 64, BF, 19)[:4])
    b = up(*draw(lens, H, 1, 64, 64, BF, 20)[:4])
    g, c = gammas(H).cuda(), cu(lens)

    def both(x):
        o, S = la.packed_fwd(*x[:3], c, "retnet", g=g)
        return [o, S, *la.packed_bwd(*x, c, "retnet", g=g)]

    ra, rb = both(a), both(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for s, x, want in ((s1, a, ra), (s2, b, rb)):
            with torch.cuda.stream(s):
                got.append((both(x), want))
    torch.cuda.synchronize()
    for r, want in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want))
    live = [t.clone() for t in a]
    graphs = []
    for _ in range(2):  # two graphs over the same library pool
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = both(live)
        graphs.append((gr, res))
    for x, want in ((b, rb), (a, ra)):
        for t, u in zip(live, x):
            t.copy_(u)
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
            eager = both(b)
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, res in graphs:
            assert all(torch.equal(p, q) for p, q in zip(res, want))
        assert all(torch.equal(p, q) for p, q in zip(eager, rb))
    done()


@pytest.mark.parametrize("lens,H,Hk", [([130, 70, 1], 64, 32), ([8200, 300], 1, 1)])
def test_captured_with_workspaces(lens, H, Hk):
    # calls that plan and split their work, captured: allocations, overlapping passes and head sums replayed
    a, b = (up(*draw(lens, H, Hk, 64, 64, BF, seed)[:4]) for seed in (32, 33))
    g, c = gammas(H).cuda(), cu(lens)

    def both(x):
        o, S = la.packed_fwd(*x[:3], c, "retnet", g=g)
        return [o, S, *la.packed_bwd(*x, c, "retnet", g=g)]

    want = {0: both(a), 1: both(b)}
    live = [t.clone() for t in a]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = both(live)
    for k, x in ((1, b), (0, a), (1, b)):
        for t, u in zip(live, x):
            t.copy_(u)
        graph.replay()
        eager = both(a)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(res, want[k]))
        assert all(torch.equal(p, q) for p, q in zip(eager, want[0]))
    done()


def test_a_stream_argument():
    lens, H = [300], 2
    x = up(*draw(lens, H, 2, 64, 64, BF, 21)[:3])
    g = gammas(H).cuda()
    want = la.packed_fwd(*x, cu(lens), "retnet", g=g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = la.packed_fwd(*x, cu(lens), "retnet", g=g, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_same_every_run():
    lens, H = [900, 33, 400], 4
    x = up(*draw(lens, H, 1, 128, 64, BF, 22)[:4])
    g = gammas(H).cuda()
    a = la.packed_bwd(*x, cu(lens), "retnet", g=g)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, la.packed_bwd(*x, cu(lens), "retnet", g=g)))


@pytest.mark.parametrize("H,Hk,dk,dv", [(1, 1, 64, 64), (2, 1, 64, 128)])
def test_backward_of_split_sequences(H, Hk, dk, dv):
    # long enough that all three passes go by segments
    check_bwd([8200, 0, 300], H, Hk, dk, dv, BF, seed=26)


def test_split_sequences_with_a_pool():
    lens, H, dk, dv = [3300, 40, 0, 2900], 2, 128, 64
    q, k, v, _, _, _ = draw(lens, H, 1, dk, dv, BF, 27)
    pool = torch.randn(6, H, dk, dv, generator=torch.Generator().manual_seed(28))
    slots = torch.tensor([5, 2, 0, 2], dtype=torch.int32)  # the last one names the second one's row
    g = gammas(H)
    start = torch.stack([pool[5], pool[2], pool[0], torch.zeros(H, dk, dv)])
    S = pool.cuda()
    o, _ = la.packed_fwd(*up(q, k, v), cu(lens), "retnet", g=g.cuda(), S0=S, S_final=S, slots=slots.cuda())
    done()
    want, Sw = retention(q, k, v, g, lens, start)
    size, Ss = retention(q, k, v, g, lens, start, positive=True)
    hold(o, want, packed_bound(want, size, 3300, BF), "o")
    hold(S[[5, 2, 0]], Sw[:3], state_bound(Ss[:3], 3300, BF), "S")
    assert torch.equal(S[[1, 3, 4]].cpu(), pool[[1, 3, 4]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths_that_are_not_what_they_should_be(dtype):
    # bounds outside the tokens are clamped, a decreasing one makes an empty sequence: [0,300), none, [100,700), none
    q, k, v, dO, _, _ = draw([700], 2, 1, 64, 64, dtype, 29)
    c = torch.tensor([-7, 300, 100, 2000, 650], dtype=torch.int32).cuda()
    g = gammas(2)
    args = up(q, k, v, dO)
    o, S = la.packed_fwd(*args[:3], c, "retnet", g=g.cuda())
    got = la.packed_bwd(*args, c, "retnet", g=g.cuda())
    done()
    part = (q[100:], k[100:], v[100:], g, [600])
    want, size = (retention(*part, positive=p)[0][200:] for p in (False, True))
    hold(o[300:], want, packed_bound(want, size, 600, dtype), "o")  # rows of one sequence only
    assert (S[[1, 3]] == 0).all() and all(t.shape for t in got)
    # the same long sequence several times over: more segments than there is room for
    n = 6000
    q, k, v, dO, _, _ = draw([n], 1, 1, 64, 64, dtype, 30)
    args = up(q, k, v, dO)
    again = torch.tensor([0, n, 0, n, 0, n], dtype=torch.int32).cuda()
    la.packed_fwd(*args[:3], again, "retnet", g=g[:1].cuda())
    la.packed_bwd(*args, again, "retnet", g=g[:1].cuda())
    done()
    check_fwd([1500, 1], 1, 1, 64, 64, dtype, seed=31)


def test_offsets_past_32_bits():
    # 2^24 tokens of 128 channels: the last sequence's elements lie behind 2^31
    n, tail, d = 1 << 24, 150, 128
    N = n + tail
    q, k, v, dO, S0, dS = draw([tail], 1, 1, d, d, BF, 24)
    big = [torch.zeros(N, 1, d, dtype=BF, device="cuda") for _ in range(4)]
    for t, x in zip(big, (q, k, v, dO)):
        t[n:] = x.cuda()
    step = n // 64
    c = torch.tensor([i * step for i in range(65)] + [N], dtype=torch.int32).cuda()
    g = gammas(1)
    o, S = la.packed_fwd(*big[:3], c, "retnet", g=g.cuda())
    args, size_args = (q, k, v, g, [tail]), dict(positive=True)
    want, Sw = retention(*args)
    size, Ss = retention(*args, **size_args)
    hold(o[n:], want, packed_bound(want, size, tail, BF), "o")
    hold(S[64:], Sw, state_bound(Ss, tail, BF), "S_final")
    assert (o[:n].view(-1, 1 << 20).float().abs().amax(1) == 0).all()
    del o
    got = la.packed_bwd(*big, c, "retnet", g=g.cuda())
    done()
    want = retention_bwd(q, k, v, dO, g, [tail])
    size = retention_bwd(q, k, v, dO, g, [tail], positive=True)
    for name, a, b, e in zip(("dq", "dk", "dv"), got, want, size):
        hold(a[n:], b, packed_bound(b, e, tail, BF), name)


def test_many_short_sequences():
    # more sequences than a CTA's threads, lengths 0 to 3, and a pool of states in another order
    gen = torch.Generator().manual_seed(25)
    lens = torch.randint(0, 4, (1500,), generator=gen).tolist()
    q, k, v, _, S0, _ = draw(lens, 1, 1, 64, 64, BF, 25)
    slots = torch.randperm(1600, generator=gen)[:1500].to(torch.int32)
    pool = torch.zeros(1600, 1, 64, 64)
    pool[slots.long()] = S0
    dev = pool.cuda()
    g = gammas(1)
    o, S = la.packed_fwd(*up(q, k, v), cu(lens), "retnet", g=g.cuda(), S0=dev, S_final=dev, slots=slots.cuda())
    done()
    want, Sw = retention(q, k, v, g, lens, S0)
    size, Ss = retention(q, k, v, g, lens, S0, positive=True)
    hold(o, want, packed_bound(want, size, 3, BF), "o")
    hold(S.cpu()[slots.long()], Sw, state_bound(Ss, 3, BF), "S")
