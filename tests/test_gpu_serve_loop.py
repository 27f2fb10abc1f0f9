"""A small hybrid stack (a retention layer, then a softmax layer over a paged
cache) decoded by beam search with all the serving operators together, against
a search in float64 that computes every hypothesis from its tokens alone."""
import math

import pytest
import torch

import gated_delta_rule_linear_gb300 as la
import servelib as ref
from layerlib import gammas, retention, starts

H, HK, D, WIDTH, V, EOS = 4, 2, 64, 96, 60, 7
B, W, PAGE, STEPS = 3, 4, 4, 9
PROMPTS = [5, 12, 8]

# Float32 against float64: a logit of up to about 8 behind six products of up to 256 terms, each good to 256 * 2^-24 of
# its size, is off by less than 8 * 6 * 256 * 2^-24 < 1e-3, and a score of STEPS tokens by STEPS times that; the search
# takes the same way if no two neighbours are closer than twice this.
OFF = 1e-3 * STEPS
SEED = 22


def model(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda a, b: torch.randn(a, b, generator=gen) * a ** -0.5  # noqa: E731
    return {"emb": torch.randn(V, WIDTH, generator=gen), "qkv1": r(WIDTH, (2 * HK + H) * D), "out1": r(H * D, WIDTH) * 4,
            "qkv2": r(WIDTH, (H + 2 * HK) * D), "out2": r(H * D, WIDTH) * 4, "head": 2.5 * r(WIDTH, V),
            "prompts": [torch.randint(8, V, (n,), generator=gen).tolist() for n in PROMPTS]}


FREQ = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))


def heads(x, *n):
    return [t.unflatten(-1, (-1, D)) for t in x.split([h * D for h in n], -1)]


def logits_of(m, tokens):
    """Next-token logits of a hypothesis, from its tokens."""
    m = {k: v.double() if torch.is_tensor(v) else v for k, v in m.items()}
    n = len(tokens)
    x = m["emb"][tokens]
    q, k, v = heads(x @ m["qkv1"], HK, HK, H)
    x = x + retention(q * D ** -0.5, k, v, gammas(H), [n])[0].flatten(1) @ m["out1"]
    q, k, v = heads(x @ m["qkv2"], H, HK, HK)
    pos = torch.arange(n)[:, None]
    q, k = (ref.turned(t, pos, FREQ, [D // 2], False)[0] for t in (q, k))
    s = torch.einsum("hd,thd->ht", q[-1], k.repeat_interleave(H // HK, 1)) * D ** -0.5
    o = torch.einsum("ht,thd->hd", torch.softmax(s, -1), v.repeat_interleave(H // HK, 1))
    return (x[-1] + o.flatten() @ m["out2"]) @ m["head"]


def search(m):
    """Tokens and scores of the beams, and the smallest distance of two that were compared."""
    gap, out = math.inf, []
    for prompt in m["prompts"]:
        beams = [([], 0.0, False)] + [([], -math.inf, False)] * (W - 1)
        for _ in range(STEPS):
            logits = torch.stack([logits_of(m, prompt + t) for t, _, _ in beams])[None]
            scores = torch.tensor([[s for _, s, _ in beams]], dtype=torch.float64)
            c = ref.candidates(logits, scores, torch.tensor([[d for _, _, d in beams]]), EOS)
            order = torch.sort(c.flatten(), descending=True).values[:W + 1]
            gap = min(gap, float((order[:-1] - order[1:]).min()))
            best, parent, token = (t[0].tolist() for t in ref.selection(c, W))
            beams = [(beams[p][0] + [v], s, beams[p][2] or v == EOS) for s, p, v in zip(best, parent, token)]
        out.append(beams)
    return out, gap


def test_the_search_is_well_apart():
    assert search(model(SEED))[1] > 2 * OFF


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_hybrid_beam_search(captured):
    m = model(SEED)
    want, gap = search(m)
    assert gap > 2 * OFF
    g = {k: v.cuda() if torch.is_tensor(v) else v for k, v in m.items()}
    dev, i32 = "cuda", torch.int32
    rows = B * W
    need = -(-(max(PROMPTS) + STEPS + 1) // PAGE)
    table = torch.randperm(rows * need, device=dev).to(i32).reshape(rows, need)
    kc, vc = (torch.full((rows * need, PAGE, HK, D), math.nan, device=dev) for _ in range(2))
    states = torch.full((rows + 2, H, D, D), math.nan, device=dev)
    slots = torch.randperm(rows + 2, device=dev)[:rows].to(i32)
    decay, freq = gammas(H).to(dev), FREQ.to(dev)

    def attend(x, table, lens, cu=None):
        """Softmax layer on new tokens; the output of each sequence's last one."""
        q, k, v = heads(x @ g["qkv2"], H, HK, HK)
        q = la.cache_append(q, k, v, kc, vc, table, lens, freq=freq, cu_seqlens=cu)
        if cu is not None:
            q, x = q[cu[1:].long() - 1], x[cu[1:].long() - 1]
        o, _ = la.paged_attn(q, kc, vc, table, lens)
        return (x + o.flatten(1) @ g["out2"]) @ g["head"]

    # prompts: their states and pages are the first beam's, then every beam's
    cu = torch.tensor(starts(PROMPTS), dtype=i32, device=dev)
    x = g["emb"][torch.tensor(sum(m["prompts"], []), device=dev)]
    q, k, v = heads(x @ g["qkv1"], HK, HK, H)
    first = slots[::W].contiguous()
    o, _ = la.packed_fwd(q * D ** -0.5, k, v, cu, "retnet", g=decay, S_final=states, slots=first)
    x = x + o.flatten(1) @ g["out1"]
    lens = torch.tensor(PROMPTS, dtype=i32, device=dev)
    logits = attend(x, table[::W], lens, cu).unsqueeze(1).repeat(1, W, 1)
    lens = lens.repeat_interleave(W)
    fork = torch.zeros((B, W), dtype=i32, device=dev)
    la.beam_states(states, fork, slots=slots)
    la.beam_cache(kc, vc, table, lens, fork)

    scores = torch.full((B, W), -math.inf, device=dev)
    scores[:, 0] = 0.0
    done = torch.zeros((B, W), dtype=torch.bool, device=dev)
    tokens = torch.zeros((B, W, STEPS), dtype=torch.int64, device=dev)
    step = torch.zeros((), dtype=torch.int64, device=dev)
    grid = torch.arange(STEPS, device=dev)

    def one_step():
        best, parent, token = la.beam_select(logits, scores, done=done, eos=EOS)
        la.beam_states(states, parent, slots=slots)
        la.beam_cache(kc, vc, table, lens, parent)
        p = parent.long()
        scores.copy_(best)
        done.copy_(torch.gather(done, 1, p) | (token == EOS))
        old = torch.gather(tokens, 1, p[..., None].expand(-1, -1, STEPS))
        tokens.copy_(torch.where(grid == step, token.long()[..., None], old))
        lens.add_(1)
        step.add_(1)
        x = g["emb"][token.flatten().long()]
        q, k, v = heads(x @ g["qkv1"], HK, HK, H)
        o = la.packed_step(q * D ** -0.5, k, v, states, "retnet", g=decay, slots=slots)
        logits.copy_(attend(x + o.flatten(1) @ g["out1"], table, lens).reshape(B, W, V))

    if captured:
        kept = [t.clone() for t in (logits, scores, done, tokens, step, lens, table, kc, vc, states)]
        one_step()  # what a first call sets up
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one_step()
        for t, old in zip((logits, scores, done, tokens, step, lens, table, kc, vc, states), kept):
            t.copy_(old)
        for _ in range(STEPS):
            graph.replay()
    else:
        for _ in range(STEPS):
            one_step()
    torch.cuda.synchronize()
    for b, beams in enumerate(want):
        for w, (hyp, score, ended) in enumerate(beams):
            assert tokens[b, w].tolist() == hyp
            assert bool(done[b, w]) == ended
            assert abs(float(scores[b, w]) - score) < OFF
