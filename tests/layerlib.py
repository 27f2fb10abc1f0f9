"""Float64 references of the layer operators and the bounds the tests hold the
kernels to.

Bounds are worst cases counted per element, not fitted: a rounding to a type of
spacing eps is off by at most eps/2 of the value (bf16 2^-8, fp32 2^-24), and
every reference comes with the same sum over absolute values, against which the
roundings inside the sum are counted.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gammas(H, decay=True):
    """log gamma_h = log(1 - 2^(-5-h)), h modulo 11."""
    return torch.tensor([math.log1p(-(2.0 ** (-5 - h % 11))) for h in range(H)]) if decay else None


def wide(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def retention(q, k, v, g, lens, S0=None, positive=False):
    """o and S_final, token by token; with ``positive``, of the absolute values."""
    H = v.shape[1]
    q, k, v = wide(q, H), wide(k, H), v.double()
    if positive:
        q, k, v = q.abs(), k.abs(), v.abs()
    gamma = torch.ones(H, dtype=torch.float64) if g is None else torch.exp(g.double())
    o = torch.zeros_like(v)
    out = []
    for s, (a, n) in enumerate(zip(starts(lens), lens)):
        S = torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64) if S0 is None else S0[s].double().clone()
        S = S.abs() if positive else S
        for t in range(a, a + n):
            S = S * gamma[:, None, None] + k[t][..., None] * v[t][:, None]
            o[t] = torch.einsum("hk,hkv->hv", q[t], S)
        out.append(S)
    return o, torch.stack(out)


def retention_bwd(q, k, v, dO, g, lens, S0=None, dS=None, positive=False):
    """dq, dk, dv, dS0 by the recurrences of the definition."""
    H, Hk = v.shape[1], q.shape[1]
    q, k, v, dO = wide(q, H), wide(k, H), v.double(), dO.double()
    if positive:
        q, k, v, dO = q.abs(), k.abs(), v.abs(), dO.abs()
    gamma = (torch.ones(H, dtype=torch.float64) if g is None else torch.exp(g.double()))[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dS0 = []
    for s, (a, n) in enumerate(zip(starts(lens), lens)):
        zero = torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64)
        S = zero if S0 is None else S0[s].double()
        W = zero if dS is None else dS[s].double()
        if positive:
            S, W = S.abs(), W.abs()
        for t in range(a, a + n):
            S = S * gamma + k[t][..., None] * v[t][:, None]
            dq[t] = torch.einsum("hkv,hv->hk", S, dO[t])
        for t in reversed(range(a, a + n)):
            G = W + q[t][..., None] * dO[t][:, None]
            dk[t] = torch.einsum("hkv,hv->hk", G, v[t])
            dv[t] = torch.einsum("hkv,hk->hv", G, k[t])
            W = gamma * G
        dS0.append(W)
    fold = lambda x: x.reshape(len(x), Hk, H // Hk, x.shape[2]).sum(2)  # noqa: E731
    return fold(dq), fold(dk), dv, torch.stack(dS0)


def hold(got, want, bound, what):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() - bound)
    worst = int(over.argmax()) if over.numel() else 0
    assert not over.numel() or over.max() <= 0, (
        f"{what}: off by {(got - want).abs().flatten()[worst]:.3e}, allowed {bound.flatten()[worst]:.3e}, "
        f"value {want.flatten()[worst]:.3e}, {int((over > 0).sum())} of {over.numel()}")


def packed_bound(want, size, T, dtype, out_dtype=None):
    """Of an output of packed retention over sequences of up to T tokens, from
    the sum over absolute values ``size``. bf16: the scores and the state's
    copy are rounded once (2^-8 of their part of the sum), the output once.
    Sums of float32 products: T + 256 roundings of up to 2^-23 (the tensor
    cores may cut instead of rounding)."""
    inner = (HALF[dtype] if dtype == torch.bfloat16 else 0.0) + (T + 256) * 2.0 ** -23
    return HALF[out_dtype or dtype] * want.abs() + inner * size + 1e-30


def state_bound(size, T, dtype):
    """Of a float32 state: decay-scaled keys are held as a bf16 high and low part
    (2^-16 of the product), float32 sums as above."""
    return ((2.0 ** -16 if dtype == torch.bfloat16 else 0.0) + (T + 256) * 2.0 ** -23) * size + 1e-30
