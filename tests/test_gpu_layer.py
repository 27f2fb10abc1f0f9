"""Rotary positions and the block epilogue on the GPU against float64, and a
retention layer of all the layer operators together."""
import pytest
import torch

import gated_delta_rule_linear_gb300 as la
from layerlib import HALF, gammas, hold, packed_bound, retention, retention_bwd, starts

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def up(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ------------------------------------------------------------------ rotary

def turned(x, pos, freq, sections, interleaved, inverse, scale):
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    angle = (pos.double()[:, axis] * freq)[:, None]
    c, s = torch.cos(angle), torch.sin(angle) * (-1 if inverse else 1)
    P = len(axis)
    y = x.double().clone()
    a, b = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    u, w = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    size = x.double().abs()
    size[..., a] = size[..., b] = u.abs() + w.abs()
    return y * scale, size * abs(scale)


def spectrum(sections):
    return torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / max(s, 1)) for s in sections])


def hold_turned(got, x, *args):
    want, size = turned(x, *args)
    # cosine, sine and angle: 2^-21 together; products and sums: 2^-22
    hold(got, want, HALF[x.dtype] * want.abs() + 2.0 ** -20 * size, "rotary")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,Hk,d,sections,far", [
    (1, 1, 1, 64, [32], 10), (37, 4, 2, 128, [64], 4000000), (130, 3, 1, 128, [12, 10, 10], 500),
    (9, 2, 2, 96, [24, 24], 90), (5, 2, 1, 10, [3], 70), (6, 1, 1, 7, [1, 0, 2], 70), (700, 16, 16, 256, [128], 65536),
])
def test_rotary(N, H, Hk, d, sections, far, interleaved, dtype):
    gen = torch.Generator().manual_seed(N + d)
    q, k = torch.randn(N, H, d, generator=gen).to(dtype), torch.randn(N, Hk, d, generator=gen).to(dtype)
    pos = torch.randint(-far, far, (N, len(sections)), generator=gen).to(torch.int32)
    freq = spectrum(sections)
    for inverse in (False, True):
        a, b = la.rotary(*up(q, k, pos, freq), sections=sections, interleaved=interleaved, inverse=inverse,
                         scale_q=1.0, scale_k=0.25)
        hold_turned(a, q, pos, freq, sections, interleaved, inverse, 1.0)
        hold_turned(b, k, pos, freq, sections, interleaved, inverse, 0.25)
        only, none = la.rotary(*up(q, None, pos, freq), sections=sections, interleaved=interleaved, inverse=inverse)
        assert none is None and torch.equal(only, a)


def test_rotary_at_the_ends_of_int32():
    pos = torch.tensor([[-2 ** 31], [2 ** 31 - 1], [0], [10 ** 9]], dtype=torch.int32)
    freq = spectrum([32]) * torch.where(torch.arange(32) % 2 == 0, 1.0, -1.0)
    q = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(1))
    a, _ = la.rotary(*up(q, None, pos, freq))
    # the angle's float64 product is itself off by 2^31 radians 2^-53, and so is the turns' frequency
    want, size = turned(q, pos, freq, [32], False, False, 1.0)
    hold(a, want, HALF[F32] * want.abs() + (2.0 ** -20 + 2.0 ** -20) * size, "rotary")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_layouts(dtype):
    # rows of a fused projection, in place, and to and from the chunk kernels' head-major layout
    B, T, H, Hk, d = 2, 17, 3, 1, 64
    N, gen = B * T, torch.Generator().manual_seed(2)
    x = torch.randn(N, (H + Hk) * d, generator=gen).to(dtype).cuda()
    q, k = x[:, :H * d].unflatten(1, (H, d)), x[:, H * d:].unflatten(1, (Hk, d))
    pos = torch.randint(0, 999, (N, 1), generator=gen).to(torch.int32).cuda()
    freq = spectrum([32]).cuda()
    a, b = la.rotary(q, k, pos, freq)
    hold_turned(a, q.cpu(), pos.cpu(), freq.cpu(), [32], False, False, 1.0)
    hq, hk = la.rotary(q, k, pos, freq, T_out=T)
    major = lambda t: t.unflatten(0, (B, T)).transpose(1, 2).contiguous()  # noqa: E731
    assert torch.equal(hq, major(a)) and torch.equal(hk, major(b))
    iq, ik = la.rotary(major(q), major(k), pos, freq)
    assert torch.equal(iq, a) and torch.equal(ik, b)
    pq, pk = q.contiguous(), k.contiguous()
    la.rotary(pq, pk, pos, freq, q_out=pq, k_out=pk)
    assert torch.equal(pq, a) and torch.equal(pk, b)
    odd = torch.randn(N * d * 2 + 1, generator=gen).to(dtype).cuda()[1:].view(N, 2, d)  # not 16-byte aligned
    c, _ = la.rotary(odd, None, pos, freq)
    hold_turned(c, odd.cpu(), pos.cpu(), freq.cpu(), [32], False, False, 1.0)


# ---------------------------------------------------------------- epilogue

def block(x, w, gate, act, res, scale, w_next, eps):
    norm = lambda t: t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)  # noqa: E731
    t = norm(x)
    t = t if w is None else t * w
    if gate is not None:
        t = t * (torch.sigmoid(gate) if act == "sigmoid" else gate * torch.sigmoid(gate))
    t = t if scale is None else t * scale
    t = t if res is None else t + res
    return t, norm(t) * (1.0 if w_next is None else w_next)


def cases(N, G, d, dtype, gate, res, scale, nxt, w=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=r(N, G, d).to(dtype), w=1 + 0.2 * r(d) if w else None, gate=2 * r(N, G, d).to(dtype) if gate else None,
                res=r(N, G, d).to(dtype) if res else None, scale=0.5 + 0.2 * r(d) if scale else None,
                w_next=1 + 0.2 * r(d) if nxt else None), r(N, G, d).to(dtype), r(N, G, d).to(dtype)


SHAPES = [(1, 1, 1), (3, 1, 7), (5, 3, 64), (40, 4, 80), (33, 16, 128), (7, 1, 1000), (6, 2, 2048), (3, 1, 5001),
          (2, 1, 16384), (300, 5, 256), (2, 1, 16383), (9, 1, 4096)]
KINDS = [(False, False, False, False), (True, False, False, False), (False, True, True, True), (True, True, True, True),
         (True, False, True, True)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate,res,scale,nxt", KINDS)
@pytest.mark.parametrize("N,G,d", SHAPES)
def test_epilogue(N, G, d, gate, res, scale, nxt, dtype):
    for act in ("silu", "sigmoid") if gate else ("silu",):
        c, d_out, d_next = cases(N, G, d, dtype, gate, res, scale, nxt, w=N != 5, seed=N * d)
        eps = 1e-5
        dev = {n: None if t is None else t.cuda() for n, t in c.items()}
        out, after = la.epilogue(**dev, act=act, eps=eps)
        f = {n: None if t is None else t.double().requires_grad_() for n, t in c.items()}
        want, wnext = block(f["x"], f["w"], f["gate"], act, f["res"], f["scale"], f["w_next"], eps)
        # a float32 chain: the row sum has at most 41 roundings one after the other (32 loads, 9 levels),
        # the exponential 2^-20: 2^-17 of the terms of the last sum
        u = HALF[dtype]
        rest = torch.zeros_like(want) if c["res"] is None else c["res"].double().abs()
        terms = (want.detach() - (0 if c["res"] is None else c["res"].double())).abs() + rest
        hold(out, want.detach(), u * want.detach().abs() + 2.0 ** -17 * terms, "out")
        if nxt:
            r2 = (wnext.detach() / want.detach().where(want != 0, torch.ones_like(want))).abs()
            hold(after, wnext.detach(), u * wnext.detach().abs() + 2.0 ** -16 * (r2 * terms + wnext.detach().abs()), "next")
        else:
            assert after is None
        # backward, against autograd in float64; the terms of its last sums from the same graph on absolute values
        got = la.epilogue_bwd(dev["x"], d_out.cuda(), w=dev["w"], gate=dev["gate"], act=act, res=dev["res"],
                              scale=dev["scale"], w_next=dev["w_next"], d_next=d_next.cuda() if nxt else None, eps=eps)
        ends, seeds = [want], [d_out.double()]
        if nxt:
            ends, seeds = ends + [wnext], seeds + [d_next.double()]
        there = [(n, t) for n, t in f.items() if t is not None]
        grads = dict(zip([n for n, _ in there], torch.autograd.grad(ends, [t for _, t in there], seeds)))
        size = bwd_terms(f, act, d_out.double(), d_next.double() if nxt else None, want.detach(), wnext.detach(), eps)
        for n, t in f.items():
            if t is None:
                assert got["d" + n] is None
            else:
                half = u if t.dim() == 3 else HALF[F32]
                hold(got["d" + n], grads[n], half * grads[n].abs() + 2.0 ** -15 * size[n] + 1e-30, "d" + n)


def bwd_terms(f, act, d_out, d_next, out, nxt, eps):
    """Sums of the absolute values of the terms behind each gradient (the order of its rounding errors)."""
    z = {n: None if t is None else t.detach() for n, t in f.items()}
    x, one = z["x"], torch.ones_like(z["x"])
    w = one if z["w"] is None else z["w"].abs()
    sc = one if z["scale"] is None else z["scale"].abs()
    a = sl = one
    if z["gate"] is not None:
        s = torch.sigmoid(z["gate"])
        # the sums inside the slope, by their terms
        a, sl = (s, s) if act == "sigmoid" else ((z["gate"] * s).abs(), s * (1 + z["gate"].abs()))
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = (x * r).abs()
    tot = d_out.abs()
    size = {}
    if d_next is not None:
        r2 = 1 / torch.sqrt((out * out).mean(-1, keepdim=True) + eps)
        # out itself is a sum with the residual: its terms, not its value
        m = r2 * ((0 if z["res"] is None else z["res"].abs()) + sc * n * w * a)
        e = d_next.abs() * (1 if z["w_next"] is None else z["w_next"].abs())
        size["w_next"] = (d_next.abs() * m).sum((0, 1))
        tot = tot + r2 * (e + m * (e * m).mean(-1, keepdim=True))
    size["res"] = tot
    size["scale"] = (tot * n * w * a).sum((0, 1))
    size["gate"] = tot * sc * n * w * sl
    size["w"] = (tot * sc * a * n).sum((0, 1))
    e = tot * sc * a * w
    size["x"] = r * (e + n * (e * n).mean(-1, keepdim=True))
    return size


def test_epilogue_of_a_zero_row_and_of_far_gates():
    x = torch.zeros(3, 1, 64)
    x[1] = 1.0
    gate = torch.full((3, 1, 64), -200.0)
    gate[1, 0, ::2] = 200.0
    for dtype in (BF, F32):
        out, nxt = la.epilogue(x.to(dtype).cuda(), gate=gate.to(dtype).cuda(), with_next=True)
        want, wn = block(x.double(), None, gate.double(), "silu", None, None, None, 1e-5)
        hold(out, want, HALF[dtype] * want.abs() + 1e-30 + 2.0 ** -17 * want.abs(), "out")
        hold(nxt, wn, HALF[dtype] * wn.abs() + 2.0 ** -16 * wn.abs() + 1e-30, "next")
        got = la.epilogue_bwd(x.to(dtype).cuda(), torch.ones(3, 1, 64, dtype=dtype).cuda(), gate=gate.to(dtype).cuda())
        assert all(torch.isfinite(t).all() for t in got.values() if t is not None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_epilogue_layouts_and_aliases(dtype):
    B, T, G, d = 2, 19, 3, 128
    c, d_out, d_next = cases(B * T, G, d, dtype, True, True, True, True, seed=4)
    dev = {n: t.cuda() for n, t in c.items()}
    out, nxt = la.epilogue(**dev)
    major = dict(dev, x=dev["x"].unflatten(0, (B, T)).transpose(1, 2).contiguous())
    a, b = la.epilogue(**major)
    assert torch.equal(a, out) and torch.equal(b, nxt)
    p = la.epilogue_bwd(dev["x"], d_out.cuda(), d_next=d_next.cuda(), **{n: t for n, t in dev.items() if n != "x"})
    q = la.epilogue_bwd(major["x"], d_out.cuda(), d_next=d_next.cuda(), **{n: t for n, t in dev.items() if n != "x"})
    assert torch.equal(q["dx"].transpose(1, 2).reshape(B * T, G, d), p["dx"])
    assert all(torch.equal(p[n], q[n]) for n in p if n != "dx")
    for name, other in (("x", "gate"), ("gate", "res"), ("res", "x")):
        live = {n: t.clone() for n, t in dev.items()}
        a, b = la.epilogue(**live, out=live[name], next=live[other])
        assert torch.equal(a, out) and torch.equal(b, nxt)
    odd = {n: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape) for n, t in dev.items()}  # unaligned
    a, b = la.epilogue(**odd)
    u = HALF[dtype]
    hold(a, out.double().cpu(), 2 * u * out.double().cpu().abs() + 2.0 ** -16 * (out.double().cpu().abs() + c["res"].double().abs()), "out")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_epilogue_bwd_parts(dtype):
    # either end alone; the residual is not read without d_next; no tokens: zero sums
    c, d_out, d_next = cases(21, 2, 64, dtype, True, True, True, True, seed=5)
    dev = {n: t.cuda() for n, t in c.items()}
    x = dev.pop("x")
    zero = torch.zeros_like(d_out).cuda()
    both = la.epilogue_bwd(x, zero, d_next=d_next.cuda(), **dev)
    alone = la.epilogue_bwd(x, None, d_next=d_next.cuda(), **dev)
    assert all(torch.equal(both[n], alone[n]) for n in both)
    dev.pop("w_next")
    a = la.epilogue_bwd(x, d_out.cuda(), **dev)
    dev["res"] = torch.full_like(x, float("nan"))
    b = la.epilogue_bwd(x, d_out.cuda(), **dev)
    assert all(torch.equal(a[n], b[n]) for n in a if a[n] is not None)
    none = la.epilogue_bwd(x[:0], d_out[:0].cuda(), w=dev["w"], scale=dev["scale"])
    assert (none["dw"] == 0).all() and (none["dscale"] == 0).all() and none["dx"].numel() == 0


def test_epilogue_bwd_is_the_same_every_run_and_on_many_rows():
    c, d_out, _ = cases(5000, 4, 64, F32, True, False, False, False, seed=6)
    dev = {n: t.cuda() for n, t in c.items() if t is not None}
    a = la.epilogue_bwd(d_out=d_out.cuda(), **dev)
    for _ in range(3):
        b = la.epilogue_bwd(d_out=d_out.cuda(), **dev)
        assert all(torch.equal(a[n], b[n]) for n in a if a[n] is not None)
    f = {n: t.double().requires_grad_() for n, t in c.items() if t is not None}
    out, _ = block(f["x"], f["w"], f["gate"], "silu", None, None, None, 1e-5)
    (dw,) = torch.autograd.grad(out, f["w"], d_out.double())
    size = bwd_terms({**{n: None for n in c}, **f}, "silu", d_out.double(), None, out.detach(), None, 1e-5)["w"]
    hold(a["dw"], dw, 2.0 ** -15 * size, "dw")


def test_offsets_past_32_bits():
    # 2^24 rows of 128 channels: the last rows' elements lie behind 2^31
    n, tail, d = 1 << 24, 5, 128
    gen = torch.Generator().manual_seed(9)
    x, gate = (torch.randn(tail, 1, d, generator=gen).to(BF) for _ in range(2))
    big = [torch.zeros(n + tail, 1, d, dtype=BF, device="cuda") for _ in range(2)]
    for t, r in zip(big, (x, gate)):
        t[n:] = r.cuda()
    out, _ = la.epilogue(big[0], gate=big[1])
    want, _ = block(x.double(), None, gate.double(), "silu", None, None, None, 1e-5)
    hold(out[n:], want, HALF[BF] * want.abs() + 2.0 ** -17 * want.abs(), "out")
    dx = la.epilogue_bwd(big[0], big[1], gate=big[1])["dx"]
    alone = la.epilogue_bwd(x.cuda(), gate.cuda(), gate=gate.cuda())["dx"]
    assert torch.equal(dx[n:], alone)
    pos = torch.zeros(n + tail, 1, dtype=torch.int32, device="cuda")
    pos[n:, 0] = torch.arange(7, 7 + tail)
    freq = spectrum([64])
    turned_x, _ = la.rotary(big[0], None, pos, freq.cuda())
    hold_turned(turned_x[n:], x, pos[n:].cpu(), freq, [64], False, False, 1.0)


# ------------------------------------------------------------- a whole layer

@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_retention_layer(dtype):
    """rotary -> packed retention -> epilogue, forward and backward, each stage on what the one before it gave."""
    lens, H, Hk, d = [140, 1, 67], 4, 2, 64
    N, gen = sum(lens), torch.Generator().manual_seed(7)
    r = lambda *s: (torch.randn(*s, generator=gen)).to(dtype)  # noqa: E731
    q, k, v, gate, d_out = r(N, Hk, d), r(N, Hk, d), r(N, H, d), r(N, H, d), r(N, H, d)
    w, g, freq = 1 + 0.1 * torch.randn(d, generator=gen), gammas(H), spectrum([32])
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)[:, None]
    c = torch.tensor(starts(lens), dtype=torch.int32).cuda()
    dq, dk, dv, dgate, dw, dg, dfreq, dpos, dd = up(q, k, v, gate, w, g, freq, pos, d_out)
    rq, rk = la.rotary(dq, dk, dpos, dfreq, scale_k=d ** -0.5)
    o, _ = la.packed_fwd(rq, rk, dv, c, "retnet", g=dg, max_len=max(lens))
    y, _ = la.epilogue(o, w=dw, gate=dgate)
    e = la.epilogue_bwd(o, dd, w=dw, gate=dgate)
    gq, gk, gv, _ = la.packed_bwd(rq, rk, dv, e["dx"], c, "retnet", g=dg, max_len=max(lens))
    bq, bk = la.rotary(gq, gk, dpos, dfreq, inverse=True, scale_k=d ** -0.5)
    cpu = lambda t: t.cpu()  # noqa: E731
    hold_turned(rk, k, pos, freq, [32], False, False, d ** -0.5)
    args = (cpu(rq), cpu(rk), v, g, lens)
    want, size = retention(*args)[0], retention(*args, positive=True)[0]
    hold(o, want, packed_bound(want, size, 140, dtype), "o")
    out, _ = block(cpu(o).double(), w.double(), gate.double(), "silu", None, None, None, 1e-5)
    hold(y, out, HALF[dtype] * out.abs() + 2.0 ** -17 * out.abs() + 1e-30, "y")
    args = (cpu(rq), cpu(rk), v, cpu(e["dx"]), g, lens)
    for name, got, want, size in zip(("dq", "dk", "dv"), (gq, gk, gv), retention_bwd(*args),
                                     retention_bwd(*args, positive=True)):
        hold(got, want, packed_bound(want, size, 140, dtype), name)
    hold_turned(bk, cpu(gk), pos, freq, [32], False, True, d ** -0.5)
    hold_turned(bq, cpu(gq), pos, freq, [32], False, True, 1.0)
    assert la.la_stream_status(torch.cuda.current_stream().cuda_stream) == 0


def test_between_the_chunk_kernels():
    # head-major rotary in front of la_chunk_fwd, epilogue on its head-major o: the dense batch of the packed layer
    B, T, H, d = 2, 256, 2, 64
    gen = torch.Generator().manual_seed(8)
    q, k, v, gate = (torch.randn(B * T, H, d, generator=gen).to(BF).cuda() for _ in range(4))
    pos = torch.arange(T, dtype=torch.int32).repeat(B)[:, None].cuda()
    g, freq, w = gammas(H).cuda(), spectrum([32]).cuda(), (1 + 0.1 * torch.randn(d, generator=gen)).cuda()
    hq, hk = la.rotary(q, k, pos, freq, scale_k=d ** -0.5, T_out=T)
    ho, _ = la.chunk_fwd(hq, hk, v.unflatten(0, (B, T)).transpose(1, 2).contiguous(), "retnet", g=g)
    y, _ = la.epilogue(ho, w=w, gate=gate)
    rq, rk = la.rotary(q, k, pos, freq, scale_k=d ** -0.5)
    o, _ = la.packed_fwd(rq, rk, v, torch.tensor([0, T, 2 * T], dtype=torch.int32).cuda(), "retnet", g=g)
    want, size = (retention(rq.cpu(), rk.cpu(), v.cpu(), g.cpu(), [T, T], positive=p)[0] for p in (False, True))
    hold(o, want, packed_bound(want, size, T, BF), "packed")
    out, _ = block(ho.transpose(1, 2).reshape(B * T, H, d).double().cpu(), w.double().cpu(), gate.double().cpu(), "silu",
                   None, None, None, 1e-5)
    hold(y, out, HALF[BF] * out.abs() + 2.0 ** -17 * out.abs() + 1e-30, "y")
