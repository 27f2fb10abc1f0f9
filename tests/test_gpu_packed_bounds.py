"""Packed retention on the GPU where a call's bounds are unusual: batches of many short
sequences, padded and decreasing cu_seqlens, values at the end of the range."""
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_linear_gb300 as la
from layerlib import gammas, hold, packed_bound, retention, retention_bwd, starts, state_bound

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cu(lens):
    return torch.tensor(starts(lens), dtype=torch.int32).cuda()


def up(*ts):
    return [None if t is None else t.cuda() for t in ts]


def done():
    assert la.la_stream_status(torch.cuda.current_stream().cuda_stream) == 0


def draw(N, n, H, Hk, dk, dv, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen) * dk ** -0.5  # noqa: E731
    q, k, v, dO = r(N, Hk, dk), r(N, Hk, dk), r(N, H, dv), r(N, H, dv)
    return [t.to(dtype) for t in (q, k, v, dO)] + [r(n, H, dk, dv), r(n, H, dk, dv)]


# A process of its own: the library's pool keeps what earlier calls took.
MEMORY = """
import torch
import gated_delta_rule_linear_gb300 as la

def used(lens, max_len, backward, H=16, d=128):
    N = sum(lens)
    q, k, v, o = (torch.zeros(N, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    g = torch.full((H,), -0.01, device="cuda")
    c = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    spare = [torch.empty_like(q) for _ in range(3)]  # room for the results, kept by torch
    del spare
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    if backward:
        la.packed_bwd(q, k, v, o, c, "retnet", g=g, with_dS0=False, max_len=max_len)
    else:
        la.packed_fwd(q, k, v, c, "retnet", g=g, with_state=False, max_len=max_len, o=o)
    torch.cuda.synchronize()
    assert la.la_stream_status(torch.cuda.current_stream().cuda_stream) == 0
    return before - torch.cuda.mem_get_info()[0]

used([300], 0, False)
used([300], 0, True)
print(used(LENS, MAX_LEN, BACKWARD))
"""


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("lens,max_len", [("[16] * 4096", 0), ("[60000] + [1] * 4095", 60000)])
def test_many_sequences_take_little_workspace(lens, max_len, backward):
    # No more states than the segments that a sequence was split into, however many sequences there are. 16 heads
    # of 128 x 128: a state of all heads is 1 MiB. Split sequences hold at most two segments for each of total / seg,
    # and seg is an SM's share of total * H * dv / 64 or more: 2 * 152 / 32 = 9.5 states a pass, three passes; plans
    # and allocation granularity (32 MiB a pool block) on top.
    code = MEMORY.replace("LENS", lens).replace("MAX_LEN", str(max_len)).replace("BACKWARD", str(backward))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert int(r.stdout) <= 128 << 20, r.stdout


def timed(fn):
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(5):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / 5


def test_unknown_lengths_cost_no_walk_over_all_sequences():
    # 4096 prompts of 8 tokens on a pool of states: without max_len the call has to allow for long sequences, and
    # finds none. That is a few launches more, not a second walk over the sequences.
    n, H, d = 4096, 16, 128
    q, k, v = (torch.zeros(8 * n, H, d, dtype=BF, device="cuda") for _ in range(3))
    o = torch.empty_like(v)
    g = torch.full((H,), -0.01, device="cuda")
    c = torch.arange(0, 8 * n + 1, 8, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous()
    pool = torch.zeros(n, H, d, d, device="cuda")
    known, unknown = (timed(lambda m=m: la.packed_fwd(q, k, v, c, "retnet", g=g, S0=pool, S_final=pool, slots=slots,
                                                      max_len=m, o=o)) for m in (8, 0))
    done()
    print(f"known {known:.3f} ms, unknown {unknown:.3f} ms")
    assert unknown <= 1.1 * known + 0.05, (known, unknown)


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 1)])
def test_few_split_sequences_among_many(H, Hk):
    # split sequences between hundreds of short and empty ones, forward on a pool and backward
    gen = torch.Generator().manual_seed(40)
    lens = torch.randint(0, 5, (400,), generator=gen).tolist()
    lens[3], lens[200], lens[399] = 2700, 5200, 3100
    N, n, dk, dv = sum(lens), len(lens), 64, 64
    q, k, v, dO, S0, dS = draw(N, n, H, Hk, dk, dv, BF, 41)
    slots = torch.randperm(n + 5, generator=gen)[:n].to(torch.int32)
    pool = torch.full((n + 5, H, dk, dv), 7.0)
    pool[slots.long()] = S0
    S, g = pool.cuda(), gammas(H)
    o, _ = la.packed_fwd(*up(q, k, v), cu(lens), "retnet", g=g.cuda(), S0=S, S_final=S, slots=slots.cuda())
    got = la.packed_bwd(*up(q, k, v, dO), cu(lens), "retnet", g=g.cuda(), S0=S0.cuda(), dS_final=dS.cuda())
    done()
    (want, Sw), (size, Ss) = (retention(q, k, v, g, lens, S0, positive=p) for p in (False, True))
    hold(o, want, packed_bound(want, size, 5200, BF), "o")
    hold(S.cpu()[slots.long()], Sw, state_bound(Ss, 5200, BF), "S")
    free = [r for r in range(n + 5) if r not in slots.tolist()]
    assert (S.cpu()[free] == 7.0).all()
    want, size = (retention_bwd(q, k, v, dO, g, lens, S0, dS, positive=p) for p in (False, True))
    for name, a, b, e in zip(("dq", "dk", "dv"), got, want, size):
        hold(a, b, packed_bound(b, e, 5200, BF), name)
    hold(got[3], want[3], state_bound(size[3], 5200, BF), "dS0")


def raw_bwd(args, g, c, n, dtype):
    """dq, dk, dv into buffers of fives."""
    q, k, v, dO = args
    (N, Hk, dk), (_, H, dv) = q.shape, v.shape
    outs = [torch.full((N, h, d), 5.0, dtype=dtype, device="cuda") for h, d in ((Hk, dk), (Hk, dk), (H, dv))]
    mode = la.MODE_IDS["retnet"] | (la.LA_F32 if dtype == F32 else 0)
    assert la.la_packed_bwd(q, k, v, g, dO, None, None, *outs, None, c, n, N, 0, H, Hk, dk, dv, Hk * dk, Hk * dk, H * dv,
                            mode, torch.cuda.current_stream().cuda_stream) == 0
    done()
    return outs


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(2, 2), (2, 1)])
def test_gradients_of_a_padded_batch(H, Hk, dtype):
    # a batch of fixed size with three sequences in use, the rest of cu_seqlens zero: empty sequences
    lens, back = [60, 0, 140], 25
    N = sum(lens) + back
    q, k, v, dO, _, _ = draw(N, 1, H, Hk, 64, 64, dtype, 42)
    c = torch.tensor([0, 60, 60, 200, 0, 0, 0], dtype=torch.int32).cuda()
    g = gammas(H)
    got = raw_bwd(up(q, k, v, dO), g.cuda(), c, 6, dtype)
    part = [t[:200] for t in (q, k, v, dO)]
    want, size = (retention_bwd(*part, g, lens, positive=p) for p in (False, True))
    for name, a, b, e in zip(("dq", "dk", "dv"), got, want, size):
        hold(a[:200], b, packed_bound(b, e, 140, dtype), name)
        assert (a[200:] == 5.0).all(), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(2, 2), (2, 1)])
def test_gradients_with_decreasing_bounds(H, Hk, dtype):
    # clamped into [0, 700]: [0, 300), none, [100, 700), none. Rows of one sequence are that sequence's.
    q, k, v, dO, _, _ = draw(700, 1, H, Hk, 64, 64, dtype, 43)
    g = gammas(H)
    got = raw_bwd(up(q, k, v, dO), g.cuda(), torch.tensor([-7, 300, 100, 2000, 650], dtype=torch.int32).cuda(), 4, dtype)
    for a, b, rows in ((0, 300, slice(0, 100)), (100, 700, slice(300, 700))):
        part = [t[a:b] for t in (q, k, v, dO)]
        want, size = (retention_bwd(*part, g, [b - a], positive=p) for p in (False, True))
        inner = slice(rows.start - a, rows.stop - a)
        for name, t, w, e in zip(("dq", "dk", "dv"), got, want, size):
            hold(t[rows], w[inner], packed_bound(w, e, 600, dtype)[inner], f"{name} of [{a}, {b})")
    # [400, 500) and [50, 250): the rows between them are nobody's
    got = raw_bwd(up(q, k, v, dO), g.cuda(), torch.tensor([400, 500, 50, 250], dtype=torch.int32).cuda(), 3, dtype)
    for a, b in ((400, 500), (50, 250)):
        part = [t[a:b] for t in (q, k, v, dO)]
        want, size = (retention_bwd(*part, g, [b - a], positive=p) for p in (False, True))
        for name, t, w, e in zip(("dq", "dk", "dv"), got, want, size):
            hold(t[a:b], w, packed_bound(w, e, 200, dtype), f"{name} of [{a}, {b})")
    for t in got:
        assert (t[:50] == 5.0).all() and (t[250:400] == 5.0).all() and (t[500:] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_of_tokens_that_do_not_see_each_other(dtype):
    # Tokens 10 and 20 hold values whose product is beyond float32, the others ones whose products with
    # them are of order one. Neither sees the other (10 comes first), so that every result is finite.
    n, H, d = 100, 2, 64
    g = gammas(H)
    for pair in ("qk", "vd"):  # q_10 . k_20, and dO_10 . v_20
        q, k, v, dO, _, _ = draw(n, 1, H, H, d, d, F32, 44)
        first, second = (q, k) if pair == "qk" else (dO, v)
        for t, far in ((first, 10), (second, 20)):
            scale = torch.full((n, 1, 1), 2.0 ** -70)
            scale[far] = 2.0 ** 70
            t *= scale
        q, k, v, dO = (t.to(dtype) for t in (q, k, v, dO))
        args = up(q, k, v, dO)
        o, S = la.packed_fwd(*args[:3], cu([n]), "retnet", g=g.cuda())
        got = la.packed_bwd(*args, cu([n]), "retnet", g=g.cuda())
        done()
        (want, Sw), (size, Ss) = (retention(q, k, v, g, [n], positive=p) for p in (False, True))
        hold(o, want, packed_bound(want, size, n, dtype), f"o, {pair}")
        hold(S, Sw, state_bound(Ss, n, dtype), f"S, {pair}")
        want, size = (retention_bwd(q, k, v, dO, g, [n], positive=p) for p in (False, True))
        for name, a, b, e in zip(("dq", "dk", "dv"), got, want, size):
            hold(a, b, packed_bound(b, e, n, dtype), f"{name}, {pair}")
        hold(got[3], want[3], state_bound(size[3], n, dtype), f"dS0, {pair}")
