"""Cases of the serving operators: appending to a paged cache, attention of one
token over it, beam selection, and the reordering of states and caches by beams.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits; angles and the candidates' scores in 64) or, with ``own`` set, through
the package's entry points. ``exact`` gives the same results from the
definitions in 64 bits.

Sizes follow the package's own workloads (16 heads of 128, 128 decode requests,
8 x 4096 tokens) and generic ragged batches around them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one engine step of 128 resident requests: one new token each
        {"name": "append 128 tokens", "op": "append", "n": 128, "total": 128, "lens": 3, "past": 1500, "H": 16, "Hk": 4,
         "d": 128, "rot": 128, "axes": 0, "page": 64, "interleaved": False, "dtype": "bf16"},
        # prompts of eight requests of 4096 tokens
        {"name": "append 8x4096", "op": "append", "n": 8, "total": 32768, "lens": 0, "past": 0, "H": 16, "Hk": 4,
         "d": 128, "rot": 128, "axes": 0, "page": 64, "interleaved": False, "dtype": "bf16"},
        # chunks of prompts with pictures in them (three-axis positions), half of the channels turned, float32
        {"name": "append chunks f32", "op": "append", "n": 11, "total": 2003, "lens": 5, "past": 700, "H": 8, "Hk": 8,
         "d": 128, "rot": 64, "axes": 3, "page": 20, "interleaved": True, "dtype": "f32"},
        # one request's first tokens on a small model: latency
        {"name": "attn 1x33", "op": "attn", "n": 1, "max_len": 33, "lens": 0, "H": 8, "Hk": 8, "d": 64, "page": 16,
         "window": 0, "dtype": "bf16"},
        # one engine step of 128 ragged requests
        {"name": "attn 128 ragged", "op": "attn", "n": 128, "max_len": 8192, "lens": 9, "H": 16, "Hk": 4, "d": 128,
         "page": 64, "window": 0, "dtype": "bf16"},
        # two requests over long documents: the work is in the length
        {"name": "attn 2x131072", "op": "attn", "n": 2, "max_len": 131072, "lens": 0, "H": 16, "Hk": 2, "d": 128,
         "page": 256, "window": 0, "dtype": "bf16"},
        # a full batch of long requests
        {"name": "attn 64x16384", "op": "attn", "n": 64, "max_len": 16384, "lens": 0, "H": 32, "Hk": 8, "d": 128,
         "page": 128, "window": 0, "dtype": "bf16"},
        # a layer with a sliding window, wide heads, float32, pages of an odd size
        {"name": "attn window f32", "op": "attn", "n": 37, "max_len": 5000, "lens": 4, "H": 8, "Hk": 2, "d": 256,
         "page": 20, "window": 1024, "dtype": "f32"},
        # one request of four beams
        {"name": "select 1x4", "op": "select", "B": 1, "W": 4, "V": 32000, "K": 4, "dtype": "f32", "masked": False,
         "done": False},
        # a batch of eight beams, an odd vocabulary, a grammar's forbidden tokens, beams that have ended
        {"name": "select 32x8", "op": "select", "B": 32, "W": 8, "V": 50257, "K": 8, "dtype": "bf16", "masked": True,
         "done": True},
        # states of two retention layers, eight requests of four beams
        {"name": "states 8x4", "op": "states", "B": 8, "W": 4, "layers": 2, "H": 16, "dk": 128, "dv": 128},
        # pages of four softmax layers, sixteen requests of eight beams
        {"name": "pages 16x8", "op": "pages", "B": 16, "W": 8, "layers": 4, "max_len": 2000, "lens": 2, "Hk": 4, "d": 128,
         "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most=16):
    H = rng.choice([h for h in (1, 2, 3, 4, 6, 8, 12, 16, 32) if h <= most])
    return H, rng.choice([h for h in range(1, H + 1) if H % h == 0])


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "select", "select", "states", "pages"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 20, 64, 128, 256])
    if op == "append":
        H, Hk = _heads(rng)
        d, axes, n = rng.choice([64, 96, 128, 256]), rng.choice([0, 0, 1, 3]), _log(rng, 1, 128)
        total = n if rng.random() < 0.4 else _log(rng, n, 8192)
        return {"op": op, "n": n, "total": total, "lens": rng.randrange(1 << 20), "past": _log(rng, 1, 1500), "H": H,
                "Hk": Hk, "d": d, "rot": rng.choice([d, d // 2]), "axes": axes, "page": page,
                "interleaved": rng.random() < 0.5, "dtype": dtype}
    if op == "attn":
        H, Hk = _heads(rng, 32)
        n, d = _log(rng, 1, 128), rng.choice([64, 128, 256])
        room = 64 * 16384 * 8 * 128 // (n * Hk * d) // (4 if dtype == "bf16" else 8)
        longest = _log(rng, 1, min(100000, room))
        return {"op": op, "n": n, "max_len": longest, "lens": rng.randrange(1, 1 << 20), "H": H, "Hk": Hk, "d": d,
                "page": page, "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "dtype": dtype}
    if op == "select":
        W = rng.choice([1, 2, 3, 4, 5, 8, 16])
        B, V = _log(rng, 1, 32), _log(rng, 1000, 160000)
        B = max(1, min(B, 32 * 8 * 50257 // (W * V)))
        return {"op": op, "B": B, "W": W, "V": V, "K": rng.choice([W, W, min(2 * W, 32)]), "dtype": dtype,
                "masked": rng.random() < 0.5, "done": rng.random() < 0.5}
    B, W, layers = _log(rng, 1, 16), rng.choice([2, 3, 4, 8, 16]), rng.choice([1, 2, 3])
    if op == "states":
        H = rng.choice([1, 2, 4, 8])
        return {"op": op, "B": B, "W": W, "layers": layers, "H": H, "dk": rng.choice([64, 128]),
                "dv": rng.choice([64, 128])}
    return {"op": op, "B": B, "W": W, "layers": layers, "max_len": _log(rng, 1, 2000), "lens": rng.randrange(1, 1 << 20),
            "Hk": rng.choice([1, 2, 4]), "d": rng.choice([64, 128]), "page": page, "dtype": dtype}


# ------------------------------------------------------- inputs of every case

def _cuts(case):
    """New tokens of every sequence of an append: the total cut in n parts."""
    n, total = case["n"], case["total"]
    if total == n or not case["lens"]:
        return [total // n] * n
    rng = random.Random(case["lens"])
    at = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + at, at + [total])]


def _lengths(case, n):
    """Lengths between one and the longest, spread over their logarithm; now and then an empty row."""
    if not case["lens"]:
        return [case["max_len"]] * n
    rng = random.Random(case["lens"])
    lens = [0 if rng.random() < 0.02 else _log(rng, 1, case["max_len"]) for _ in range(n)]
    lens[rng.randrange(n)] = case["max_len"]
    return lens


def _tables(lens, page, gen, spare=2):
    """Page table of the lengths, pages in no order, -1 where there is none; and how many pages the pool has."""
    need = [-(-x // page) for x in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    return table, pages


def _sections(case):
    """How many of the rot/2 pairs turn with each axis."""
    pairs, axes = case["rot"] // 2, max(case["axes"], 1)
    rest = [pairs // axes] * (axes - 1)
    return [pairs - sum(rest)] + rest


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(shape, scale=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    op, st = case["op"], {"case": case}
    if op == "append":
        n, N, H, Hk, d, dt = case["n"], case["total"], case["H"], case["Hk"], case["d"], DT[case["dtype"]]
        fused = normal((N, (H + 2 * Hk) * d), 1.0, dt)  # the layer's one projection: queries, keys and values side by side
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, d)) for x in fused.split([H * d, Hk * d, Hk * d], 1))
        new, rng = _cuts(case), random.Random(case["lens"] + 1)
        lens = [m + (rng.randint(0, case["past"]) if case["past"] else 0) for m in new]
        st["new"], st["after"], st["lens"] = new, lens, ints(lens)
        st["cu"] = None if all(m == 1 for m in new) else ints([sum(new[:i]) for i in range(n + 1)])
        st["table"], pages = _tables(lens, case["page"], gen)
        st["k_cache"], st["v_cache"] = (normal((pages, case["page"], Hk, d), 1.0, dt) for _ in range(2))
        st["sections"] = _sections(case)
        st["freq"] = torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / max(s, 1))
                                for s in st["sections"]]).to(DEV)
        # positions of their own where they are not the place in the cache
        st["pos"] = None if not case["axes"] else torch.randint(0, 4000, (N, case["axes"]), generator=gen,
                                                                device=DEV).to(torch.int32)
        return st
    if op == "attn":
        n, H, Hk, d, dt = case["n"], case["H"], case["Hk"], case["d"], DT[case["dtype"]]
        lens = _lengths(case, n)
        st["after"], st["lens"] = lens, ints(lens)
        st["q"] = normal((n, H, d), 1.0, dt)
        st["table"], pages = _tables(lens, case["page"], gen)
        st["k_cache"], st["v_cache"] = (normal((pages, case["page"], Hk, d), 1.0, dt) for _ in range(2))
        return st
    B, W = case["B"], case["W"]
    if op == "select":
        V = case["V"]
        x = normal((B, W, V), 3.0)
        if case["masked"]:
            x.masked_fill_(torch.rand((B, W, V), generator=gen, device=DEV) < 0.3, -INF)
        st["logits"] = x.to(DT[case["dtype"]])
        st["scores"] = normal((B, W), 2.0) - 20.0
        st["done"] = torch.rand((B, W), generator=gen, device=DEV) < 0.2 if case["done"] else None
        st["eos"] = V // 2
        return st
    # some beams go on as they are, some take another's place
    draws = torch.randint(0, W, (B, W), generator=gen, device=DEV)
    stay = torch.rand((B, W), generator=gen, device=DEV) < 0.25
    st["parent"] = torch.where(stay, torch.arange(W, device=DEV), draws).to(torch.int32)
    if op == "states":
        rows = B * W + 3
        st["slots"] = torch.randperm(rows, generator=gen, device=DEV)[:B * W].to(torch.int32)
        st["S"] = normal((case["layers"], rows, case["H"], case["dk"], case["dv"]), 0.1)
        return st
    lens = [x for x in _lengths(case, B) for _ in range(W)]
    st["lens"] = ints(lens)
    # every beam has pages of its own up to the one its next token goes to
    st["table"], pages = _tables([x + 1 for x in lens], case["page"], gen)
    shape = (case["layers"], pages, case["page"], case["Hk"], case["d"])
    st["k_cache"], st["v_cache"] = (normal(shape, 1.0, DT[case["dtype"]]) for _ in range(2))
    return st


# ------------------------------------------------------------ the plain forms

def _plain_append(st):
    c = st["case"]
    N, page, half, rot, cu = c["total"], c["page"], c["rot"] // 2, c["rot"], st["cu"]
    token = torch.arange(N, device=DEV)
    if cu is None:
        seq, p = token, st["lens"].long() - 1
    else:
        seq = torch.searchsorted(cu[1:].long(), token, right=True)
        p = st["lens"].long()[seq] - cu.long()[seq + 1] + token
    rows = st["table"][seq, p // page].long() * page + p % page
    pos = p[:, None] if st["pos"] is None else st["pos"]
    axis = torch.repeat_interleave(torch.arange(len(st["sections"]), device=DEV),
                                   torch.tensor(st["sections"], device=DEV))
    angle = pos.double()[:, axis] * st["freq"]  # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        f = x.float()
        if c["interleaved"]:
            a, b = f[..., 0:rot:2], f[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = f[..., :half], f[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, f[..., rot:]], -1).to(x.dtype)

    st["k_cache"].flatten(0, 1)[rows] = turn(st["k"])
    st["v_cache"].flatten(0, 1)[rows] = st["v"]
    return {"q": turn(st["q"]), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attn(st):
    c = st["case"]
    n, H, Hk, d, page, L = c["n"], c["H"], c["Hk"], c["d"], c["page"], c["max_len"]
    L = min(L, c["window"] or L)
    p = st["lens"].long()[:, None] - L + torch.arange(L, device=DEV)  # the last L places of every row
    there = (p >= 0)[:, None, None]
    p = p.clamp(min=0)
    rows = torch.gather(st["table"].long(), 1, p // page).clamp(min=0) * page + p % page
    K, V = (x.flatten(0, 1)[rows].float() for x in (st["k_cache"], st["v_cache"]))
    q = st["q"].float().reshape(n, Hk, H // Hk, d)
    s = (q @ K.permute(0, 2, 3, 1)) * d ** -0.5
    s = torch.where(there, s, -INF)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -INF, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = (e @ V.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    return {"o": o.reshape(n, H, d).to(st["q"].dtype)}


def _plain_select(st):
    c = st["case"]
    V, K, scores = c["V"], c["K"], st["scores"].double()
    x = st["logits"].double()  # candidates of two beams may be next to each other: 64 bits
    m = x.amax(-1, keepdim=True)
    cand = scores[..., None] + (x - (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))))
    if st["done"] is not None:
        ended = torch.where(torch.arange(V, device=DEV) == st["eos"], scores[..., None], -INF)
        cand = torch.where(st["done"][..., None], ended, cand)
    best, at = torch.sort(cand.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    return {"scores": best.float(), "parent": (at // V).int(), "token": (at % V).int()}


def _plain_states(st):
    c, S = st["case"], st["S"]
    slots = st["slots"].long().reshape(c["B"], c["W"])
    S[:, slots] = S[:, torch.gather(slots, 1, st["parent"].long())]
    return {"S": S}


def _plain_pages(st):
    c = st["case"]
    B, W, page, table = c["B"], c["W"], c["page"], st["table"]
    parent = st["parent"].long()
    flat = (torch.arange(B, device=DEV)[:, None] * W + parent).flatten()
    lens = st["lens"].long()
    full, fill = lens // page, lens % page
    last = torch.gather(table, 1, full[:, None])[:, 0].long()  # each beam's open page
    copied = (torch.arange(page, device=DEV) < fill[:, None])[None, ..., None, None]
    for x in (st["k_cache"], st["v_cache"]):
        x[:, last] = torch.where(copied, x[:, last[flat]], x[:, last])
    table.copy_(torch.where(torch.arange(table.shape[1], device=DEV) < full[:, None], table[flat], table))
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "table": table}


PLAIN = {"append": _plain_append, "attn": _plain_attn, "select": _plain_select, "states": _plain_states,
         "pages": _plain_pages}


def _own(st):
    import gated_delta_rule_linear_gb300 as la
    c = st["case"]
    op = c["op"]
    if op == "append":
        q = la.cache_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                            freq=st["freq"], pos=st["pos"], sections=st["sections"], interleaved=c["interleaved"],
                            cu_seqlens=st["cu"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if op == "attn":
        o, _ = la.paged_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], window=c["window"],
                             max_len=c["max_len"])
        return {"o": o}
    if op == "select":
        scores, parent, token = la.beam_select(st["logits"], st["scores"], c["K"], done=st["done"], eos=st["eos"])
        return {"scores": scores, "parent": parent, "token": token}
    if op == "states":
        la.beam_states(st["S"], st["parent"], slots=st["slots"], layered=True)
        return {"S": st["S"]}
    la.beam_cache(st["k_cache"], st["v_cache"], st["table"], st["lens"], st["parent"], layered=True)
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "table": st["table"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------ what a pass cannot avoid

def work(case):
    op = case["op"]
    if op == "append":
        e, N, d = (2 if case["dtype"] == "bf16" else 4), case["total"], case["d"]
        rows = N * (case["H"] + 2 * case["Hk"])
        return {"bytes": 2 * e * rows * d + 4 * N * case["axes"] + 8 * case["n"],
                "flops": 3 * N * (case["H"] + case["Hk"]) * case["rot"]}
    if op == "attn":
        e, H, Hk, d = (2 if case["dtype"] == "bf16" else 4), case["H"], case["Hk"], case["d"]
        seen = sum(min(x, case["window"] or x) for x in _lengths(case, case["n"]))
        return {"bytes": 2 * e * d * (seen * Hk + case["n"] * H), "flops": 4 * seen * H * d}
    B, W = case["B"], case["W"]
    if op == "select":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": B * W * (case["V"] * e + 4) + 12 * B * case["K"], "flops": 4 * B * W * case["V"]}
    # of W beams, three quarters with a parent drawn at random: these have another one in (W-1)/W, and are written;
    # a row is read once if it is anyone else's parent
    moved = 0.75 * (W - 1) / W
    read = 1.0 - (1.0 - 0.75 / W) ** (W - 1)
    if op == "states":
        row = case["H"] * case["dk"] * case["dv"] * 4
        return {"bytes": int(B * W * case["layers"] * row * (moved + read)), "flops": 0}
    e, page = (2 if case["dtype"] == "bf16" else 4), case["page"]
    lens = _lengths(case, B)
    fill = sum(x % page for x in lens) * W
    row = case["layers"] * 2 * case["Hk"] * case["d"] * e
    return {"bytes": int((fill * row + 4 * sum(x // page for x in lens) * W) * (moved + read)) + 8 * B * W, "flops": 0}


# ------------------------------------------------- the definitions in 64 bits

def _exact_append(st):
    c = st["case"]
    page, rot = c["page"], c["rot"]
    where, place = [], []
    table = st["table"].tolist()
    for s, m in enumerate(st["new"]):
        for p in range(st["after"][s] - m, st["after"][s]):
            place.append(p)
            where.append(table[s][p // page] * page + p % page)
    where = torch.tensor(where, device=DEV)
    pos = torch.tensor(place, device=DEV)[:, None] if st["pos"] is None else st["pos"]
    parts, at = [], 0
    for a, s in enumerate(st["sections"]):  # one turn e^{i pos f} for each pair of an axis
        parts.append(pos[:, a:a + 1].double() * st["freq"][at:at + s])
        at += s
    angle = torch.cat(parts, 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def one(x):
        y = x.double().clone()
        r = y[..., :rot]
        pairs = r.unflatten(-1, (-1, 2)) if c["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y[..., :rot] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return y

    K, V = st["k_cache"].double(), st["v_cache"].double()
    K.flatten(0, 1).index_copy_(0, where, one(st["k"]))
    V.flatten(0, 1).index_copy_(0, where, st["v"].double())
    return {"q": one(st["q"]), "k_cache": K, "v_cache": V}


def _exact_attn(st):
    c = st["case"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    share = c["H"] // c["Hk"]
    for s, L in enumerate(st["after"]):
        if L == 0:
            continue
        pages = st["table"][s, :-(-L // c["page"])].long()
        first = max(0, L - c["window"]) if c["window"] else 0
        for h in range(c["Hk"]):
            K, V = (x[pages, :, h].flatten(0, 1)[first:L].double() for x in (st["k_cache"], st["v_cache"]))
            q = st["q"][s, h * share:(h + 1) * share].double()
            o[s, h * share:(h + 1) * share] = torch.softmax(q @ K.T / math.sqrt(c["d"]), -1) @ V
    return {"o": o}


def _exact_select(st):
    c = st["case"]
    K, V, out = c["K"], c["V"], {"scores": [], "parent": [], "token": []}
    for b in range(c["B"]):
        found = []
        for w in range(c["W"]):
            base = float(st["scores"][b, w])
            if st["done"] is not None and bool(st["done"][b, w]):
                found.append((-base, w, st["eos"]))
                continue
            logp = torch.log_softmax(st["logits"][b, w].double(), -1)
            best, at = torch.sort(-logp, stable=True)
            found += [(x - base, w, v) for x, v in zip(best[:K].tolist(), at[:K].tolist())]
        found = sorted(found)[:K]
        out["scores"].append([-x for x, _, _ in found])
        out["parent"].append([w for _, w, _ in found])
        out["token"].append([v for _, _, v in found])
    return {"scores": torch.tensor(out["scores"], dtype=torch.float64, device=DEV),
            "parent": torch.tensor(out["parent"], dtype=torch.int32, device=DEV),
            "token": torch.tensor(out["token"], dtype=torch.int32, device=DEV)}


def _exact_states(st):
    c, old = st["case"], st["S"].double()
    S, slots, parent = old.clone(), st["slots"].tolist(), st["parent"].tolist()
    for b in range(c["B"]):
        for w in range(c["W"]):
            S[:, slots[b * c["W"] + w]] = old[:, slots[b * c["W"] + parent[b][w]]]
    return {"S": S}


def _exact_pages(st):
    c = st["case"]
    page, W = c["page"], c["W"]
    K, V = st["k_cache"].double(), st["v_cache"].double()
    before, parent, lens = st["table"].tolist(), st["parent"].tolist(), st["lens"].tolist()
    table = [list(row) for row in before]
    for i, row in enumerate(table):
        j = i // W * W + parent[i // W][i % W]
        full, fill = divmod(lens[i], page)
        row[:full] = before[j][:full]
        K[:, row[full], :fill] = st["k_cache"][:, before[j][full], :fill].double()
        V[:, row[full], :fill] = st["v_cache"][:, before[j][full], :fill].double()
    return {"k_cache": K, "v_cache": V, "table": torch.tensor(table, dtype=torch.int32, device=DEV)}


EXACT = {"append": _exact_append, "attn": _exact_attn, "select": _exact_select, "states": _exact_states,
         "pages": _exact_pages}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
