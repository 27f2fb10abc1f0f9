"""ctypes binding of the layer operators of libla.so: include/la_layer.h under
the same names, and wrappers that take torch CUDA tensors.

As in ``_binding``: argument marshalling only, every step of the computation
runs in the library's CUDA kernels, and a non-zero status raises ``LAError``.
The wrappers run on the device of their tensors and allocate their outputs on
the stream that they launch on.
"""
from __future__ import annotations

import ctypes
import os

from ._binding import CONSTANTS, HEADER, MODE_IDS, LAError, _ptr, _read_constants, la_last_error
from . import _binding

LAYER_HEADER = os.path.join(os.path.dirname(HEADER), "la_layer.h")
LAYER_CONSTANTS = _read_constants(LAYER_HEADER)
globals().update(LAYER_CONSTANTS)

ACT_IDS = {"silu": LAYER_CONSTANTS["LA_ACT_SILU"], "sigmoid": LAYER_CONSTANTS["LA_ACT_SIGMOID"]}

_P, _I, _L, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
LAYER_SIGNATURES = {
    "la_packed_fwd": ([_P] * 9 + [_I] * 8 + [_L] * 3 + [_I, _P], _I),
    "la_packed_bwd": ([_P] * 12 + [_I] * 7 + [_L] * 3 + [_I, _P], _I),
    "la_packed_step": ([_P] * 7 + [_I] * 6 + [_L] * 3 + [_I, _P], _I),
    "la_rotary": ([_P] * 6 + [_I] * 10 + [_L] * 2 + [_F] * 2 + [_I, _P], _I),
    "la_epilogue": ([_P] * 3 + [_I] + [_P] * 5 + [_F] + [_I] * 5 + [_P], _I),
    "la_epilogue_bwd": ([_P] * 3 + [_I] + [_P] * 11 + [_F] + [_I] * 5 + [_P], _I),
}

_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(_binding.load_library(), name)
        f.argtypes, f.restype = LAYER_SIGNATURES[name]
        _fns[name] = f
    return f


# ---- raw C entry points (same names and argument order as la_layer.h) --------

def la_packed_fwd(q, k, v, g, o, S0, S_final, cu_seqlens, slots, n_seq, total, max_len, n_slots, H, Hk, dk, dv,
                  ldq, ldk, ldv, mode, stream):
    return _fn("la_packed_fwd")(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o), _ptr(S0), _ptr(S_final),
                                _ptr(cu_seqlens), _ptr(slots), n_seq, total, max_len, n_slots, H, Hk, dk, dv,
                                ldq, ldk, ldv, mode, stream)


def la_packed_bwd(q, k, v, g, dO, S0, dS_final, dq, dk_out, dv_out, dS0, cu_seqlens, n_seq, total, max_len, H, Hk,
                  dk, dv, ldq, ldk, ldv, mode, stream):
    return _fn("la_packed_bwd")(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(dO), _ptr(S0), _ptr(dS_final), _ptr(dq),
                                _ptr(dk_out), _ptr(dv_out), _ptr(dS0), _ptr(cu_seqlens), n_seq, total, max_len, H,
                                Hk, dk, dv, ldq, ldk, ldv, mode, stream)


def la_packed_step(q, k, v, g, o, S, slots, n, n_slots, H, Hk, dk, dv, ldq, ldk, ldv, mode, stream):
    return _fn("la_packed_step")(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o), _ptr(S), _ptr(slots), n, n_slots, H,
                                 Hk, dk, dv, ldq, ldk, ldv, mode, stream)


def la_rotary(q, k, q_out, k_out, pos, freq, n_axes, s0, s1, s2, N, H, Hk, d, T_in, T_out, ldq, ldk, scale_q,
              scale_k, flags, stream):
    return _fn("la_rotary")(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(pos), _ptr(freq), n_axes, s0, s1, s2,
                            N, H, Hk, d, T_in, T_out, ldq, ldk, scale_q, scale_k, flags, stream)


def la_epilogue(x, w, gate, act, res, scale, w_next, out, next, eps, N, G, d, T, flags, stream):
    return _fn("la_epilogue")(_ptr(x), _ptr(w), _ptr(gate), act, _ptr(res), _ptr(scale), _ptr(w_next), _ptr(out),
                              _ptr(next), eps, N, G, d, T, flags, stream)


def la_epilogue_bwd(x, w, gate, act, res, scale, w_next, d_out, d_next, dx, dgate, dres, dw, dscale, dw_next, eps,
                    N, G, d, T, flags, stream):
    return _fn("la_epilogue_bwd")(_ptr(x), _ptr(w), _ptr(gate), act, _ptr(res), _ptr(scale), _ptr(w_next),
                                  _ptr(d_out), _ptr(d_next), _ptr(dx), _ptr(dgate), _ptr(dres), _ptr(dw),
                                  _ptr(dscale), _ptr(dw_next), eps, N, G, d, T, flags, stream)


# ---- torch-tensor wrappers -----------------------------------------------------

class _On:
    """The tensors' device and the stream of a call: current inside, left as it was behind it."""

    def __init__(self, device, stream):
        import torch
        self.cuda, self.device, self.stream, self.back = torch.cuda, device, stream, []

    def __enter__(self):
        if self.device.index != self.cuda.current_device():
            self.back.append(self.cuda.device(self.device))
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError(f"stream on {self.stream.device}, tensors on {self.device}")
            self.back.append(self.cuda.stream(self.stream))
        for c in self.back:
            c.__enter__()
        return self.cuda.current_stream().cuda_stream

    def __exit__(self, *e):
        for c in reversed(self.back):
            c.__exit__(*e)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != device):
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _dense(dtype, **tensors):
    for name, t in tensors.items():
        if t is not None and (t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous {dtype}, got {t.dtype}")


def _shape(t, name, *shape):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _rows(t, name):
    """Token stride of a token-major [N, heads, d] tensor: heads and channels dense, tokens at any stride."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, d], got {tuple(t.shape)}")
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name}: the heads of a token must be dense")
    return sn if n > 1 else max(sn, h * d) if n else h * d


def _flag(dtype):
    import torch
    if dtype == torch.float32:
        return CONSTANTS["LA_F32"]
    if dtype != torch.bfloat16:
        raise TypeError(f"tensors must be bfloat16 or float32, got {dtype}")
    return 0


def _qkv(q, k, v):
    """(N, H, Hk, dk, dv, token strides) of a packed call's inputs."""
    ld = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    (N, Hk, dk), (_, H, dv) = q.shape, v.shape
    _shape(k, "k", N, Hk, dk)
    _shape(v, "v", N, H, dv)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must have one dtype")
    return N, H, Hk, dk, dv, ld


def _run(rc):
    if rc != 0:
        raise LAError(rc, la_last_error())


def _mode(mode, dtype):
    return (MODE_IDS[mode] if isinstance(mode, str) else int(mode)) | _flag(dtype)


def packed_fwd(q, k, v, cu_seqlens, mode, g=None, S0=None, slots=None, S_final=None, with_state=True, max_len=0,
               o=None, stream=None):
    """Causal retention over packed sequences (la_packed_fwd), mode "retnet" or
    "linear". q, k [total,Hk,dk], v [total,H,dv] (bf16 or fp32; token stride
    free); cu_seqlens int32 [n+1]; g [H] fp32; S0, S_final [n,H,dk,dv] fp32, or
    a pool [rows,H,dk,dv] with slots int32 [n] (S_final may be S0: updated in
    place; with slots and no S_final, one is needed to get states back).
    Returns (o, S_final or None)."""
    import torch
    N, H, Hk, dk, dv, ld = _qkv(q, k, v)
    dev, f32, i32 = q.device, torch.float32, torch.int32
    _same_device(dev, q=q, k=k, v=v, cu_seqlens=cu_seqlens, g=g, S0=S0, slots=slots, S_final=S_final, o=o)
    _dense(i32, cu_seqlens=cu_seqlens, slots=slots)
    _dense(f32, g=g, S0=S0, S_final=S_final)
    _dense(q.dtype, o=o)
    _shape(g, "g", H)
    _shape(o, "o", N, H, dv)
    n = cu_seqlens.numel() - 1
    _shape(slots, "slots", n)
    rows = n
    for name, t in (("S0", S0), ("S_final", S_final)):
        if t is not None:
            _shape(t, name, t.shape[0] if slots is not None else n, H, dk, dv)
            rows = t.shape[0]
    if S0 is not None and S_final is not None and S0.shape != S_final.shape:
        raise ValueError("S0 and S_final must have one shape")
    with _On(dev, stream) as handle:
        if o is None:
            o = torch.empty((N, H, dv), dtype=q.dtype, device=dev)
        if not with_state:
            S_final = None
        elif S_final is None and slots is None:
            S_final = torch.empty((n, H, dk, dv), dtype=f32, device=dev)
        _run(la_packed_fwd(q, k, v, g, o, S0, S_final, cu_seqlens, slots, n, N, max_len, rows, H, Hk, dk, dv, *ld,
                           _mode(mode, q.dtype), handle))
    return o, S_final


def packed_bwd(q, k, v, dO, cu_seqlens, mode, g=None, S0=None, dS_final=None, with_dS0=True, max_len=0, stream=None):
    """Backward pass of packed_fwd (la_packed_bwd): dq, dk, dv (dtype of q) and
    dS0 (fp32, or None). dO [total,H,dv]; S0, dS_final [n,H,dk,dv] fp32 or None."""
    import torch
    N, H, Hk, dk, dv, ld = _qkv(q, k, v)
    dev, f32 = q.device, torch.float32
    _same_device(dev, q=q, k=k, v=v, dO=dO, cu_seqlens=cu_seqlens, g=g, S0=S0, dS_final=dS_final)
    _dense(torch.int32, cu_seqlens=cu_seqlens)
    _dense(f32, g=g, S0=S0, dS_final=dS_final)
    _dense(q.dtype, dO=dO)
    n = cu_seqlens.numel() - 1
    _shape(g, "g", H)
    _shape(dO, "dO", N, H, dv)
    _shape(S0, "S0", n, H, dk, dv)
    _shape(dS_final, "dS_final", n, H, dk, dv)
    with _On(dev, stream) as handle:
        dq = torch.empty((N, Hk, dk), dtype=q.dtype, device=dev)
        dk_, dv_ = torch.empty_like(dq), torch.empty((N, H, dv), dtype=q.dtype, device=dev)
        dS0 = torch.empty((n, H, dk, dv), dtype=f32, device=dev) if with_dS0 else None
        _run(la_packed_bwd(q, k, v, g, dO, S0, dS_final, dq, dk_, dv_, dS0, cu_seqlens, n, N, max_len, H, Hk, dk, dv,
                           *ld, _mode(mode, q.dtype), handle))
    return dq, dk_, dv_, dS0


def packed_step(q, k, v, S, mode, g=None, slots=None, o=None, stream=None):
    """One token for each row (la_packed_step): q, k [n,Hk,dk], v [n,H,dv]; S
    [rows,H,dk,dv] fp32, updated in place at slots int32 [n] (None: row i).
    Returns o [n,H,dv]."""
    import torch
    N, H, Hk, dk, dv, ld = _qkv(q, k, v)
    dev = q.device
    _same_device(dev, q=q, k=k, v=v, S=S, g=g, slots=slots, o=o)
    _dense(torch.float32, S=S, g=g)
    _dense(torch.int32, slots=slots)
    _dense(q.dtype, o=o)
    _shape(g, "g", H)
    _shape(S, "S", S.shape[0], H, dk, dv)
    _shape(slots, "slots", N)
    _shape(o, "o", N, H, dv)
    with _On(dev, stream) as handle:
        if o is None:
            o = torch.empty((N, H, dv), dtype=q.dtype, device=dev)
        _run(la_packed_step(q, k, v, g, o, S, slots, N, S.shape[0], H, Hk, dk, dv, *ld, _mode(mode, q.dtype), handle))
    return o


def _tokens_of(t, name):
    """(N, heads, d, T, token stride) of a token-major [N,heads,d] or dense head-major [B,heads,T,d] tensor."""
    if t.dim() == 4:
        if not t.is_contiguous():
            raise ValueError(f"{name}: a head-major tensor must be contiguous")
        B, H, T, d = t.shape
        return B * T, H, d, T, H * d
    ld = _rows(t, name)
    N, H, d = t.shape
    return N, H, d, 0, ld


def rotary(q, k, pos, freq, sections=None, interleaved=False, inverse=False, scale_q=1.0, scale_k=1.0, T_out=0,
           q_out=None, k_out=None, stream=None):
    """Rotary positions (la_rotary) on q [N,H,d] and k [N,Hk,d] (or None), or
    head-major [B,H,T,d]; pos int32 [N,axes]; freq float64 [pairs];
    sections: pairs of each axis (None: one axis). T_out > 0 returns head-major
    [N/T_out,H,T_out,d]. inverse turns back: the backward pass. Returns (q, k)."""
    import torch
    N, H, d, T, ldq = _tokens_of(q, "q")
    Hk, ldk = 0, 0
    if k is not None:
        Nk, Hk, dk, Tk, ldk = _tokens_of(k, "k")
        if (Nk, dk, Tk) != (N, d, T) or k.dtype != q.dtype:
            raise ValueError("q and k must agree in tokens, channels, layout and dtype")
    dev = q.device
    _same_device(dev, q=q, k=k, pos=pos, freq=freq, q_out=q_out, k_out=k_out)
    _dense(torch.int32, pos=pos)
    _dense(torch.float64, freq=freq)
    _dense(q.dtype, q_out=q_out, k_out=k_out)
    sections = [freq.numel()] if sections is None else list(sections)
    if sum(sections) != freq.numel() or not 1 <= len(sections) <= 3:
        raise ValueError("sections: the pairs of one to three axes, as many as freq has")
    _shape(pos, "pos", N, len(sections))
    s = sections + [0] * (3 - len(sections))
    if T_out and N % T_out:
        raise ValueError("T_out must divide the tokens")
    flags = _flag(q.dtype) | (LAYER_CONSTANTS["LA_ROT_INTERLEAVED"] if interleaved else 0) \
        | (LAYER_CONSTANTS["LA_ROT_INVERSE"] if inverse else 0)
    with _On(dev, stream) as handle:
        outs = []
        for name, heads, t in (("q_out", H, q_out), ("k_out", Hk, k_out)):
            shape = (N // T_out, heads, T_out, d) if T_out else (N, heads, d)
            if heads == 0:
                t = None
            elif t is None:
                t = torch.empty(shape, dtype=q.dtype, device=dev)
            _shape(t, name, *shape)
            outs.append(t)
        _run(la_rotary(q, k, outs[0], outs[1], pos, freq, len(sections), *s, N, H, Hk, d, T, T_out, ldq, ldk,
                       scale_q, scale_k, flags, handle))
    return outs[0], outs[1]


def _block(x, w, gate, act, res, scale, w_next, **more):
    """(N, G, d, T, act id) of an epilogue call."""
    import torch
    N, G, d, T, _ = _tokens_of(x, "x")
    _same_device(x.device, x=x, w=w, gate=gate, res=res, scale=scale, w_next=w_next, **more)
    _dense(x.dtype, x=x, gate=gate, res=res, **more)
    _dense(torch.float32, w=w, scale=scale, w_next=w_next)
    for name, t in dict(gate=gate, res=res, **more).items():
        _shape(t, name, N, G, d)
    for name, t in (("w", w), ("scale", scale), ("w_next", w_next)):
        _shape(t, name, d)
    return N, G, d, T, ACT_IDS[act] if gate is not None else 0


def epilogue(x, w=None, gate=None, act="silu", res=None, scale=None, w_next=None, with_next=None, eps=1e-5, out=None,
             next=None, stream=None):
    """End of a block (la_epilogue): out = res + scale * rmsnorm(x) w act(gate),
    next = rmsnorm(out) w_next. x [N,G,d] or head-major [B,G,T,d]; gate, res
    [N,G,d]; w, scale, w_next [d] fp32. next is computed with w_next, next or
    with_next. Returns (out, next or None)."""
    import torch
    N, G, d, T, a = _block(x, w, gate, act, res, scale, w_next, out=out, next=next)
    if with_next is None:
        with_next = w_next is not None or next is not None
    with _On(x.device, stream) as handle:
        if out is None:
            out = torch.empty((N, G, d), dtype=x.dtype, device=x.device)
        if with_next and next is None:
            next = torch.empty((N, G, d), dtype=x.dtype, device=x.device)
        _run(la_epilogue(x, w, gate, a, res, scale, w_next, out, next if with_next else None, eps, N, G, d, T,
                         _flag(x.dtype), handle))
    return out, (next if with_next else None)


def epilogue_bwd(x, d_out, w=None, gate=None, act="silu", res=None, scale=None, w_next=None, d_next=None, eps=1e-5,
                 stream=None):
    """Backward pass of epilogue (la_epilogue_bwd) from its inputs. d_out,
    d_next [N,G,d], one of them may be None. Returns a dict with dx (x's
    layout), dgate, dres, dw, dscale, dw_next (None where the forward had no
    such input)."""
    import torch
    N, G, d, T, a = _block(x, w, gate, act, res, scale, w_next, d_out=d_out, d_next=d_next)
    with _On(x.device, stream) as handle:
        wide = lambda t: None if t is None else torch.empty((N, G, d), dtype=x.dtype, device=x.device)  # noqa: E731
        thin = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        r = {"dx": torch.empty_like(x), "dgate": wide(gate), "dres": wide(res), "dw": thin(w), "dscale": thin(scale),
             "dw_next": thin(w_next)}
        _run(la_epilogue_bwd(x, w, gate, a, res, scale, w_next, d_out, d_next, r["dx"], r["dgate"], r["dres"],
                             r["dw"], r["dscale"], r["dw_next"], eps, N, G, d, T, _flag(x.dtype), handle))
    return r
