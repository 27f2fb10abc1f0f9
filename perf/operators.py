"""Cases of the layer operators: rotary positions, packed retention (prompts,
training, single tokens) and the block epilogue.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the package's entry points. ``exact``
gives the same results from the definitions in 64 bits.

Sizes follow the package's own workloads (16 heads of 128, 4 x 16384 and
8 x 4096 tokens, 128 decode requests) and generic ragged batches around them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 64  # tokens of a chunk of the plain chunked form
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # prefill / evaluation of four documents of the package's longest training length
        {"name": "fwd 4x16384", "op": "packed_fwd", "n": 4, "total": 65536, "ragged": False, "lens": 0, "H": 16,
         "Hk": 16, "dk": 128, "dv": 128, "decay": True, "pool": False},
        # one engine step's prompts: ragged requests with shared query/key heads and a pool of states
        {"name": "fwd 48 prompts", "op": "packed_fwd", "n": 48, "total": 24011, "ragged": True, "lens": 7, "H": 16,
         "Hk": 4, "dk": 128, "dv": 128, "decay": True, "pool": True},
        # one short prompt on a small model: latency
        {"name": "fwd 1x300", "op": "packed_fwd", "n": 1, "total": 300, "ragged": False, "lens": 0, "H": 8, "Hk": 8,
         "dk": 64, "dv": 64, "decay": True, "pool": False},
        # the training step's backward pass at the package's RetNet shape
        {"name": "bwd 8x4096", "op": "packed_bwd", "n": 8, "total": 32768, "ragged": False, "lens": 0, "H": 16,
         "Hk": 16, "dk": 128, "dv": 128, "decay": True, "pool": False},
        # packed documents of different lengths, shared key heads, unequal head widths
        {"name": "bwd 24 documents", "op": "packed_bwd", "n": 24, "total": 12001, "ragged": True, "lens": 11, "H": 8,
         "Hk": 4, "dk": 64, "dv": 128, "decay": True, "pool": False},
        # decode: the package's 128 resident requests
        {"name": "step 128", "op": "packed_step", "n": 128, "H": 16, "Hk": 16, "dk": 128, "dv": 128, "dtype": "bf16",
         "decay": True},
        # decode of a few requests: latency
        {"name": "step 3 f32", "op": "packed_step", "n": 3, "H": 8, "Hk": 4, "dk": 64, "dv": 64, "dtype": "f32",
         "decay": True},
        # per-head norm and gate after the mixer, reading the chunk forward's head-major output
        {"name": "epilogue heads", "op": "epilogue", "N": 65536, "T": 16384, "G": 16, "d": 128, "dtype": "bf16",
         "gate": "silu", "res": False, "scale": False, "next": False},
        # the residual stream of a decode batch: post-norm, layer scale, residual, the next block's pre-norm
        {"name": "epilogue decode", "op": "epilogue", "N": 37, "T": 0, "G": 1, "d": 2048, "dtype": "f32",
         "gate": "none", "res": True, "scale": True, "next": True},
        # its training backward at 8 x 4096 tokens of 16 x 128 channels
        {"name": "epilogue bwd", "op": "epilogue_bwd", "N": 32768, "T": 0, "G": 1, "d": 2048, "dtype": "bf16",
         "gate": "sigmoid", "res": True, "scale": True, "next": True},
        # rotation of queries and keys of the long documents, far positions
        {"name": "rotary 4x16384", "op": "rotary", "N": 65536, "H": 16, "Hk": 16, "d": 128, "rot": 128, "axes": 1,
         "dtype": "bf16", "interleaved": True, "inverse": False, "far": 1000000},
        # gradient of a video clip's three-axis rotation, half of the channels turned
        {"name": "rotary video bwd", "op": "rotary", "N": 1001, "H": 8, "Hk": 2, "d": 128, "rot": 64, "axes": 3,
         "dtype": "f32", "interleaved": False, "inverse": True, "far": 300},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    return H, rng.choice([h for h in range(1, H + 1) if H % h == 0])


def draw(rng):
    op = rng.choice(["packed_fwd", "packed_fwd", "packed_bwd", "packed_bwd", "packed_step", "epilogue",
                     "epilogue_bwd", "rotary"])
    if op in ("packed_fwd", "packed_bwd"):
        H, Hk = _heads(rng)
        n = _log(rng, 1, 64)
        total = _log(rng, 1, 32768 if op == "packed_fwd" else 16384)
        return {"op": op, "n": n, "total": total, "ragged": True, "lens": rng.randrange(1 << 20), "H": H, "Hk": Hk,
                "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]), "decay": rng.random() < 0.8,
                "pool": op == "packed_fwd" and rng.random() < 0.5}
    if op == "packed_step":
        H, Hk = _heads(rng)
        return {"op": op, "n": _log(rng, 1, 128), "H": H, "Hk": Hk, "dk": rng.choice([64, 128]),
                "dv": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f32"]), "decay": rng.random() < 0.8}
    if op in ("epilogue", "epilogue_bwd"):
        heads = rng.random() < 0.5
        G = rng.choice([1, 2, 3, 4, 8, 16]) if heads else 1
        d = rng.choice([64, 80, 128, 256]) if heads else _log(rng, 33, 5000)
        N = _log(rng, 1, max(2, 32768 * 1024 // (G * d)))
        B = rng.choice([1, 2, 4])
        T = N if heads and rng.random() < 0.5 else 0
        return {"op": op, "N": N * B if T else N, "T": T, "G": G, "d": d, "dtype": rng.choice(["bf16", "f32"]),
                "gate": rng.choice(["none", "silu", "sigmoid"]), "res": rng.random() < 0.5,
                "scale": rng.random() < 0.5, "next": rng.random() < 0.5}
    H, Hk = _heads(rng)
    axes = rng.choice([1, 2, 3])
    d = rng.choice([64, 96, 128, 256])
    rot = rng.choice([d, d // 2])
    return {"op": op, "N": _log(rng, 1, 16384), "H": H, "Hk": Hk, "d": d, "rot": rot, "axes": axes,
            "dtype": rng.choice(["bf16", "f32"]), "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5,
            "far": _log(rng, 100, 4000000) if axes == 1 else _log(rng, 10, 4000)}


# ------------------------------------------------------- inputs of every case

def _lengths(case):
    n, total = case["n"], case["total"]
    if not case["ragged"]:
        return [total // n] * n
    rng = random.Random(case["lens"])
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _sections(case):
    """How many of the rot/2 pairs turn with each axis."""
    pairs, axes = case["rot"] // 2, case["axes"]
    rest = [pairs // axes] * (axes - 1)
    return [pairs - sum(rest)] + rest


def _plan(lens, dev):
    """Chunk table of the plain form: token of every chunk row (or the zero row behind the last token), rows in
    use, sequence, and offset of the chunk in its sequence."""
    L = torch.tensor(lens, dtype=torch.int64)
    nc = (L + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lens)), nc)
    first = torch.cumsum(nc, 0) - nc
    a0 = (torch.arange(int(nc.sum())) - first[seq]) * CHUNK
    rows = torch.clamp(L[seq] - a0, max=CHUNK)
    start = torch.cumsum(L, 0) - L
    r = torch.arange(CHUNK)
    idx = torch.where(r[None] < rows[:, None], (start[seq] + a0)[:, None] + r[None], torch.tensor(int(L.sum())))
    # where each token sits in the padded chunks
    back = torch.nonzero((r[None] < rows[:, None]).reshape(-1))[:, 0]
    return {"L": L.to(dev), "seq": seq.to(dev), "a0": a0.to(dev), "rows": rows.to(dev), "idx": idx.to(dev),
            "back": back.to(dev)}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)

    op, st = case["op"], {"case": case}
    if op.startswith("packed"):
        H, Hk, dk, dv, n = case["H"], case["Hk"], case["dk"], case["dv"], case["n"]
        dt = DT[case.get("dtype", "bf16")]
        N = n if op == "packed_step" else case["total"]
        st["q"], st["k"] = normal((N, Hk, dk), dk ** -0.5, dt), normal((N, Hk, dk), dk ** -0.5, dt)
        st["v"] = normal((N, H, dv), dk ** -0.5, dt)
        st["mode"] = "retnet" if case["decay"] else "linear"
        # the per-head decays 1 - 2^(-5-h) of the package's RetNet workload
        st["g"] = torch.tensor([math.log1p(-(2.0 ** (-5 - h))) for h in range(H)], device=DEV) if case["decay"] else None
        if op == "packed_step":
            st["slots"] = torch.randperm(n + 3, generator=gen, device=DEV)[:n].to(torch.int32)
            st["S"] = normal((n + 3, H, dk, dv), 0.1)
            return st
        lens = _lengths(case)
        st["lens"], st["max_len"] = lens, max(lens)
        st["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
        st["plan"] = _plan(lens, DEV)
        if op == "packed_bwd":
            st["S0"] = normal((n, H, dk, dv), 0.1)
            st["dO"] = normal((N, H, dv), dv ** -0.5, dt)
            st["dS"] = normal((n, H, dk, dv), 0.1)
        elif case["pool"]:  # the engine's pool of states: read and written at the requests' slots
            st["slots"] = torch.randperm(n + 3, generator=gen, device=DEV)[:n].to(torch.int32)
            st["S"] = normal((n + 3, H, dk, dv), 0.1)
        else:
            st["S"] = st["slots"] = None
        return st
    if op.startswith("epilogue"):
        N, G, d, T, dt = case["N"], case["G"], case["d"], case["T"], DT[case["dtype"]]
        shape = (N // T, G, T, d) if T else (N, G, d)
        st["x"] = normal(shape, 1.0, dt)
        st["w"] = 1.0 + normal((d,), 0.1)
        st["gate"] = normal((N, G, d), 1.0, dt) if case["gate"] != "none" else None
        st["res"] = normal((N, G, d), 1.0, dt) if case["res"] else None
        st["scale"] = 0.5 + normal((d,), 0.1) if case["scale"] else None
        st["w_next"] = 1.0 + normal((d,), 0.1) if case["next"] else None
        if op == "epilogue_bwd":
            st["d_out"] = normal((N, G, d), 1.0, dt)
            st["d_next"] = normal((N, G, d), 1.0, dt) if case["next"] else None
        return st
    N, H, Hk, d, rot, axes, dt = (case["N"], case["H"], case["Hk"], case["d"], case["rot"], case["axes"],
                                  DT[case["dtype"]])
    st["q"], st["k"] = normal((N, H, d), 1.0, dt), normal((N, Hk, d), 1.0, dt)
    st["pos"] = torch.randint(0, case["far"], (N, axes), generator=gen, device=DEV).to(torch.int32)
    st["sections"] = _sections(case)
    # one spectrum for each axis: base 10000, from 1 downwards
    st["freq"] = torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / max(s, 1)) for s in st["sections"]]).to(DEV)
    return st


# ------------------------------------------------------------ the plain forms

def _chunks(x, plan):
    """[N, H, d] -> [H, chunks, CHUNK, d], rows not in use zero."""
    x = torch.cat([x, x.new_zeros((1,) + x.shape[1:])])
    return x[plan["idx"]].permute(2, 0, 1, 3)


def _power(g, e):
    """exp(g e) for every head and exponent e (g None: ones)."""
    e = e.double()
    if g is None:
        return torch.ones_like(e).float()[None]
    return torch.exp(g.double().reshape(-1, *[1] * e.dim()) * e[None]).float()


def _decay_pass(x, y, z, g, S, plan, reverse):
    """out_i = sum_j gamma^|i-j| (x_i . y_j) z_j over j <= i (reverse: j >= i) of the same sequence, plus what the
    state that enters the sequence gives; also the state that leaves it. Chunked: products inside a chunk, and
    every chunk's contribution to every later chunk's entering state."""
    X, Y, Z = (_chunks(t, plan) for t in (x, y, z))
    i = torch.arange(CHUNK, device=x.device)
    rows, a0, L, seq = plan["rows"], plan["a0"], plan["L"], plan["seq"]
    end = a0 + rows
    away = (i[None] - i[:, None]) if reverse else (i[:, None] - i[None])
    inside = _power(g, away.clamp(min=0)) * (away >= 0)
    out = (X @ Y.transpose(-1, -2) * inside[:, None]) @ Z
    keep = (i[None] + 1).expand(len(rows), -1) if reverse else (rows[:, None] - 1 - i[None]).clamp(min=0)
    U = (Y * _power(g, keep)[..., None]).transpose(-1, -2) @ Z
    H, nc, a, b = U.shape
    U = U.reshape(H, nc, a * b)
    same = seq[:, None] == seq[None]
    if reverse:
        far, into = a0[None] - end[:, None], L[seq] - end
        gone, reach = a0, (rows[:, None] - 1 - i[None]).clamp(min=0)
    else:
        far, into = a0[:, None] - end[None], a0
        gone, reach = L[seq] - end, (i[None] + 1).expand(len(rows), -1)
    enter = (_power(g, far.clamp(min=0)) * (same & (far >= 0))) @ U
    leave = (_power(g, gone)[:, None] * (seq[None] == torch.arange(len(L), device=x.device)[:, None])) @ U
    leave = leave.reshape(H, len(L), a, b).transpose(0, 1)
    enter = enter.reshape(H, nc, a, b)
    if S is not None:
        S = S.transpose(0, 1)
        enter = enter + _power(g, into)[..., None, None] * S[:, seq]
        leave = leave + (_power(g, L)[..., None, None] * S).transpose(0, 1)
    out = out + _power(g, reach)[..., None] * (X @ enter)
    return out.permute(1, 2, 0, 3).reshape(nc * CHUNK, H, b)[plan["back"]], leave


def _wide(x, H):
    """Shared heads, once for every head that uses them."""
    return x.float().repeat_interleave(H // x.shape[1], 1)


def _plain_packed_fwd(st):
    c, S = st["case"], st["S"]
    q, k, v = _wide(st["q"], c["H"]), _wide(st["k"], c["H"]), st["v"].float()
    S0 = None if S is None else S[st["slots"].long()]
    o, S1 = _decay_pass(q, k, v, st["g"], S0, st["plan"], False)
    if S is None:
        S = S1
    else:
        S[st["slots"].long()] = S1
    return {"o": o.to(st["v"].dtype), "S": S}


def _plain_packed_bwd(st):
    c = st["case"]
    q, k, v, dO = _wide(st["q"], c["H"]), _wide(st["k"], c["H"]), st["v"].float(), st["dO"].float()
    t = lambda S: S.transpose(-1, -2)  # noqa: E731
    dq, _ = _decay_pass(dO, v, k, st["g"], t(st["S0"]), st["plan"], False)
    dk, _ = _decay_pass(v, dO, q, st["g"], t(st["dS"]), st["plan"], True)
    dv, dS0 = _decay_pass(k, q, dO, st["g"], st["dS"], st["plan"], True)
    dq, dk = (x.reshape(len(x), c["Hk"], -1, c["dk"]).sum(2) for x in (dq, dk))
    dt = st["v"].dtype
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dS0": dS0}


def _plain_packed_step(st):
    c, S, at = st["case"], st["S"], st["slots"].long()
    q, k, v = _wide(st["q"], c["H"]), _wide(st["k"], c["H"]), st["v"].float()
    gamma = 1.0 if st["g"] is None else torch.exp(st["g"])[None, :, None, None]
    new = gamma * S[at] + k[..., None] * v[..., None, :]
    S[at] = new
    return {"o": (q[..., None] * new).sum(-2).to(st["v"].dtype), "S": S}


EPS = 1e-5


def _tokens(x):
    """[B, G, T, d] -> [B T, G, d]."""
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3]) if x.dim() == 4 else x


def _like(y, x):
    """The way back of _tokens."""
    return y.reshape(x.shape[0], x.shape[2], x.shape[1], x.shape[3]).transpose(1, 2).contiguous() if x.dim() == 4 else y


def _gate(st):
    """Value and slope of the gate's activation."""
    if st["gate"] is None:
        return None, None
    a = st["gate"].float()
    s = 1.0 / (1.0 + torch.exp(-a))
    return (s, s * (1.0 - s)) if st["case"]["gate"] == "sigmoid" else (a * s, s * (1.0 + a * (1.0 - s)))


def _plain_epilogue(st):
    x = _tokens(st["x"]).float()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = n * st["w"]
    a, slope = _gate(st)
    out = y if a is None else y * a
    out = out if st["scale"] is None else out * st["scale"]
    out = out if st["res"] is None else out + st["res"].float()
    return x, n, y, a, slope, out


def _plain_epilogue_fwd(st):
    out, dt = _plain_epilogue(st)[-1], st["x"].dtype
    got = {"out": out.to(dt)}
    if st["w_next"] is not None:
        got["next"] = (out * torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS) * st["w_next"]).to(dt)
    return got


def _plain_epilogue_bwd(st):
    x, n, y, a, slope, out = _plain_epilogue(st)
    dt, total, got = st["x"].dtype, st["d_out"].float(), {}
    if st["w_next"] is not None:
        r = torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS)
        e, m = st["d_next"].float(), out * r
        got["dw_next"] = (e * m).sum((0, 1))
        e = e * st["w_next"]
        total = total + r * (e - m * (e * m).mean(-1, keepdim=True))
    if st["res"] is not None:
        got["dres"] = total.to(dt)
    if st["scale"] is not None:
        got["dscale"] = (total * (y if a is None else y * a)).sum((0, 1))
        total = total * st["scale"]
    if a is not None:
        got["dgate"] = (total * y * slope).to(dt)
        total = total * a
    got["dw"] = (total * n).sum((0, 1))
    e = total * st["w"]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    got["dx"] = _like((r * (e - n * (e * n).mean(-1, keepdim=True))).to(dt), st["x"])
    return got


def _axis_of_pair(st):
    return torch.repeat_interleave(torch.arange(len(st["sections"]), device=DEV),
                                   torch.tensor(st["sections"], device=DEV))


def _plain_rotary(st):
    c = st["case"]
    angle = st["pos"].double()[:, _axis_of_pair(st)] * st["freq"]  # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    sin = -sin if c["inverse"] else sin
    half, rot = c["rot"] // 2, c["rot"]

    def turn(x):
        f = x.float()
        if c["interleaved"]:
            a, b = f[..., 0:rot:2], f[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = f[..., :half], f[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, f[..., rot:]], -1).to(x.dtype)

    return {"q": turn(st["q"]), "k": turn(st["k"])}


PLAIN = {"packed_fwd": _plain_packed_fwd, "packed_bwd": _plain_packed_bwd, "packed_step": _plain_packed_step,
         "epilogue": _plain_epilogue_fwd, "epilogue_bwd": _plain_epilogue_bwd, "rotary": _plain_rotary}


def _own(st):
    import gated_delta_rule_linear_gb300 as la
    c = st["case"]
    op = c["op"]
    if op == "packed_fwd":
        o, S = la.packed_fwd(st["q"], st["k"], st["v"], st["cu"], st["mode"], g=st["g"], S0=st["S"], S_final=st["S"],
                             slots=st["slots"], max_len=st["max_len"])
        return {"o": o, "S": S}
    if op == "packed_bwd":
        dq, dk, dv, dS0 = la.packed_bwd(st["q"], st["k"], st["v"], st["dO"], st["cu"], st["mode"], g=st["g"],
                                        S0=st["S0"], dS_final=st["dS"], max_len=st["max_len"])
        return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0}
    if op == "packed_step":
        o = la.packed_step(st["q"], st["k"], st["v"], st["S"], st["mode"], g=st["g"], slots=st["slots"])
        return {"o": o, "S": st["S"]}
    if op == "epilogue":
        out, after = la.epilogue(st["x"], w=st["w"], gate=st["gate"], act=c["gate"], res=st["res"], scale=st["scale"],
                                 w_next=st["w_next"], eps=EPS)
        return {"out": out} if after is None else {"out": out, "next": after}
    if op == "epilogue_bwd":
        got = la.epilogue_bwd(st["x"], st["d_out"], w=st["w"], gate=st["gate"], act=c["gate"], res=st["res"],
                              scale=st["scale"], w_next=st["w_next"], d_next=st["d_next"], eps=EPS)
        return {name: t for name, t in got.items() if t is not None}
    q, k = la.rotary(st["q"], st["k"], st["pos"], st["freq"], sections=st["sections"], interleaved=c["interleaved"],
                     inverse=c["inverse"])
    return {"q": q, "k": k}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------ what a pass cannot avoid

def work(case):
    op = case["op"]
    if op.startswith("packed"):
        H, Hk, dk, dv, n = case["H"], case["Hk"], case["dk"], case["dv"], case["n"]
        state = n * H * dk * dv * 4
        if op == "packed_step":
            e = 2 if case["dtype"] == "bf16" else 4
            return {"bytes": 2 * state + n * e * (2 * Hk * dk + 2 * H * dv), "flops": 5 * n * H * dk * dv}
        N = case["total"]
        if op == "packed_fwd":
            states = state * (2 if case["pool"] else 1)
            return {"bytes": 2 * N * (2 * Hk * dk + 2 * H * dv) + states, "flops": 4 * N * H * dk * dv}
        return {"bytes": 2 * N * (4 * Hk * dk + 3 * H * dv) + 3 * state, "flops": 10 * N * H * dk * dv}
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("epilogue"):
        size = case["N"] * case["G"] * case["d"]
        gate, res, nxt = case["gate"] != "none", case["res"], case["next"]
        if op == "epilogue":
            return {"bytes": e * size * (2 + gate + res + nxt), "flops": size * (6 + 5 * gate + 5 * nxt)}
        # res is read only where the norm behind it is differentiated
        return {"bytes": e * size * (3 + 2 * gate + res + (res and nxt) + nxt), "flops": size * (12 + 8 * gate + 10 * nxt)}
    size = case["N"] * (case["H"] + case["Hk"])
    return {"bytes": 2 * e * size * case["d"] + 4 * case["N"] * case["axes"], "flops": 3 * size * case["rot"]}


# ------------------------------------------------- the definitions in 64 bits

def _order(st):
    """Sequences from the longest to the shortest: the ones still running are the first ones."""
    lens = st["lens"]
    order = sorted(range(len(lens)), key=lambda s: -lens[s])
    L = [lens[s] for s in order]
    start = st["cu"].long()[torch.tensor(order, device=DEV)]
    return order, L, start


def _running(L):
    """How many of the sequences (longest first) have a token t, for every t."""
    counts, m = [], len(L)
    for t in range(L[0] if L else 0):
        while m and L[m - 1] <= t:
            m -= 1
        counts.append(m)
    return counts


def _gammas(st, H):
    return torch.ones(H, dtype=torch.float64, device=DEV) if st["g"] is None else torch.exp(st["g"].double())


def _each_head(x, H):
    return x.double()[:, torch.arange(H, device=DEV) // (H // x.shape[1])]


def _exact_packed_fwd(st):
    c = st["case"]
    H = c["H"]
    q, k, v = _each_head(st["q"], H), _each_head(st["k"], H), st["v"].double()
    order, L, start = _order(st)
    gamma = _gammas(st, H)[None, :, None, None]
    rows = torch.tensor(order, device=DEV)
    if st["S"] is not None:
        rows = st["slots"].long()[rows]
        pool = st["S"].double()
    else:
        pool = torch.zeros((c["n"], H, c["dk"], c["dv"]), dtype=torch.float64, device=DEV)
    S = pool[rows]
    o = torch.zeros_like(v)
    for t, m in enumerate(_running(L)):
        tok = start[:m] + t
        S[:m].mul_(gamma).addcmul_(k[tok][..., None], v[tok][..., None, :])
        o[tok] = torch.einsum("nhk,nhkv->nhv", q[tok], S[:m])
    pool[rows] = S
    return {"o": o, "S": pool}


def _exact_packed_bwd(st):
    c = st["case"]
    H = c["H"]
    q, k, v, dO = _each_head(st["q"], H), _each_head(st["k"], H), st["v"].double(), st["dO"].double()
    order, L, start = _order(st)
    gamma = _gammas(st, H)[None, :, None, None]
    rows = torch.tensor(order, device=DEV)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    S, G = st["S0"].double()[rows], st["dS"].double()[rows]
    last = start + torch.tensor(L, device=DEV) - 1
    for t, m in enumerate(_running(L)):
        tok = start[:m] + t
        S[:m].mul_(gamma).addcmul_(k[tok][..., None], v[tok][..., None, :])
        dq[tok] = torch.einsum("nhkv,nhv->nhk", S[:m], dO[tok])
        tok = last[:m] - t
        G[:m].addcmul_(q[tok][..., None], dO[tok][..., None, :])
        dk[tok] = torch.einsum("nhkv,nhv->nhk", G[:m], v[tok])
        dv[tok] = torch.einsum("nhkv,nhk->nhv", G[:m], k[tok])
        G[:m].mul_(gamma)
    dS0 = torch.empty_like(G)
    dS0[rows] = G
    dq, dk = (x.reshape(len(x), c["Hk"], H // c["Hk"], c["dk"]).sum(2) for x in (dq, dk))
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0}


def _exact_packed_step(st):
    c, at = st["case"], st["slots"].long()
    q, k, v = _each_head(st["q"], c["H"]), _each_head(st["k"], c["H"]), st["v"].double()
    pool = st["S"].double()
    S = pool[at] * _gammas(st, c["H"])[None, :, None, None] + torch.einsum("nhk,nhv->nhkv", k, v)
    pool[at] = S
    return {"o": torch.einsum("nhk,nhkv->nhv", q, S), "S": pool}


def _exact_block(st, x, w, gate, res, scale, w_next):
    """The block's end as one differentiable expression."""
    norm = lambda t: t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)  # noqa: E731
    t = norm(x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3]) if x.dim() == 4 else x) * w
    if gate is not None:
        t = t * (torch.sigmoid(gate) if st["case"]["gate"] == "sigmoid" else gate * torch.sigmoid(gate))
    if scale is not None:
        t = scale * t
    if res is not None:
        t = res + t
    return t, None if w_next is None else norm(t) * w_next


def _exact_epilogue(st):
    names = ("x", "w", "gate", "res", "scale", "w_next")
    leaves = [None if st[n] is None else st[n].double() for n in names]
    if st["case"]["op"] == "epilogue":
        out, after = _exact_block(st, *leaves)
        return {"out": out} if after is None else {"out": out, "next": after}
    leaves = [None if t is None else t.requires_grad_() for t in leaves]
    out, after = _exact_block(st, *leaves)
    ends, seeds = [out], [st["d_out"].double()]
    if after is not None:
        ends, seeds = ends + [after], seeds + [st["d_next"].double()]
    there = [(n, t) for n, t in zip(names, leaves) if t is not None]
    grads = torch.autograd.grad(ends, [t for _, t in there], seeds)
    return {"d" + n: g for (n, _), g in zip(there, grads)}


def _exact_rotary(st):
    c = st["case"]
    parts, at = [], 0
    for axis, s in enumerate(st["sections"]):  # one turn e^{i pos f} for each pair of an axis
        parts.append(st["pos"][:, axis:axis + 1].double() * st["freq"][at:at + s])
        at += s
    angle = torch.cat(parts, 1)
    turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)[:, None]

    def one(x):
        y = x.double().clone()
        r = y[..., :c["rot"]]
        pairs = r.unflatten(-1, (-1, 2)) if c["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y[..., :c["rot"]] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return y

    return {"q": one(st["q"]), "k": one(st["k"])}


EXACT = {"packed_fwd": _exact_packed_fwd, "packed_bwd": _exact_packed_bwd, "packed_step": _exact_packed_step,
         "epilogue": _exact_epilogue, "epilogue_bwd": _exact_epilogue, "rotary": _exact_rotary}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
