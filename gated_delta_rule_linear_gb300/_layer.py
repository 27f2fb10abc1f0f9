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

def _refuse(t, name, dtype, shape, idx):
    if not t.is_cuda or t.get_device() != idx:
        raise ValueError(f"{name} must be on CUDA device {idx}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(t, name, dtype, shape, idx):
    """A dense tensor of this type and shape on device idx (None passes). One pass over the attributes: calls
    of a few tokens are bound by their host side."""
    if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != idx or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, idx)


def _index(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    return t.get_device()


class _On:
    """The tensors' device and the call's stream: current inside, left as they were behind it."""

    def __init__(self, idx, stream):
        import torch
        self.cuda, self.idx, self.stream, self.back = torch.cuda, idx, stream, []

    def __enter__(self):
        if self.idx != self.cuda.current_device():
            self.back.append(self.cuda.device(self.idx))
        if self.stream is not None:
            if self.stream.device_index != self.idx:
                raise ValueError(f"stream on device {self.stream.device_index}, tensors on {self.idx}")
            self.back.append(self.cuda.stream(self.stream))
        for c in self.back:
            c.__enter__()
        return self.cuda.current_stream().cuda_stream

    def __exit__(self, *e):
        for c in reversed(self.back):
            c.__exit__(*e)


def _launch(idx, stream, body):
    """body(stream handle) on the tensors' device: at once where that and the stream are current already."""
    import torch
    if stream is None and idx == torch._C._cuda_getDevice():
        return body(torch._C._cuda_getCurrentRawStream(idx))
    with _On(idx, stream) as handle:
        return body(handle)


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(t, name):
    """Token stride of a token-major [N, heads, d] tensor: heads and channels dense, tokens at any stride."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, d], got {tuple(t.shape)}")
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name}: the heads of a token must be dense")
    return sn if n > 1 and sn > h * d else h * d if n <= 1 or sn == h * d else sn


def _flag(dtype):
    import torch
    if dtype is torch.float32:
        return CONSTANTS["LA_F32"]
    if dtype is not torch.bfloat16:
        raise TypeError(f"tensors must be bfloat16 or float32, got {dtype}")
    return 0


def _qkv(q, k, v):
    """(N, H, Hk, dk, dv, token strides, device) of a packed call's inputs."""
    lq, lk, lv = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    idx, dt = _index(q, "q"), q.dtype
    N, Hk, dk = q.shape
    n, H, dv = v.shape
    if k.shape != q.shape or n != N:
        raise ValueError(f"k must have q's shape and v as many tokens: {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    if k.dtype is not dt or v.dtype is not dt:
        raise TypeError("q, k and v must have one dtype")
    if k.get_device() != idx or v.get_device() != idx:
        raise ValueError("q, k and v must be on one device")
    return N, H, Hk, dk, dv, lq, lk, lv, idx


def _run(name, *args):
    rc = (_fns.get(name) or _fn(name))(*args)
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
    place; with slots and no S_final, final states are not kept).
    Returns (o, S_final or None)."""
    import torch
    N, H, Hk, dk, dv, lq, lk, lv, idx = _qkv(q, k, v)
    mid, f32, i32 = _mode(mode, q.dtype), torch.float32, torch.int32
    n = cu_seqlens.numel() - 1
    _check(cu_seqlens, "cu_seqlens", i32, (n + 1,), idx)
    _check(slots, "slots", i32, (n,), idx)
    _check(g, "g", f32, (H,), idx)
    rows = n
    if slots is not None:
        pool = S0 if S0 is not None else S_final
        rows = 0 if pool is None else pool.shape[0]
    _check(S0, "S0", f32, (rows, H, dk, dv), idx)
    if not with_state:
        S_final = None
    _check(S_final, "S_final", f32, (rows, H, dk, dv), idx)
    _check(o, "o", q.dtype, (N, H, dv), idx)

    def body(handle):
        out = q.new_empty((N, H, dv)) if o is None else o
        state = S_final
        if with_state and state is None and slots is None:
            state = q.new_empty((n, H, dk, dv), dtype=f32)
        _run("la_packed_fwd", q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(g), out.data_ptr(), _at(S0), _at(state),
             cu_seqlens.data_ptr(), _at(slots), n, N, max_len, rows, H, Hk, dk, dv, lq, lk, lv, mid, handle)
        return out, state

    return _launch(idx, stream, body)


def packed_bwd(q, k, v, dO, cu_seqlens, mode, g=None, S0=None, dS_final=None, with_dS0=True, max_len=0, stream=None):
    """Backward pass of packed_fwd (la_packed_bwd): dq, dk, dv (dtype of q) and
    dS0 (fp32, or None). dO [total,H,dv]; S0, dS_final [n,H,dk,dv] fp32 or None."""
    import torch
    N, H, Hk, dk, dv, lq, lk, lv, idx = _qkv(q, k, v)
    mid, f32 = _mode(mode, q.dtype), torch.float32
    n = cu_seqlens.numel() - 1
    _check(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), idx)
    _check(g, "g", f32, (H,), idx)
    _check(dO, "dO", q.dtype, (N, H, dv), idx)
    _check(S0, "S0", f32, (n, H, dk, dv), idx)
    _check(dS_final, "dS_final", f32, (n, H, dk, dv), idx)

    def body(handle):
        dq, dk_, dv_ = q.new_empty((N, Hk, dk)), q.new_empty((N, Hk, dk)), q.new_empty((N, H, dv))
        dS0 = q.new_empty((n, H, dk, dv), dtype=f32) if with_dS0 else None
        _run("la_packed_bwd", q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(g), dO.data_ptr(), _at(S0), _at(dS_final),
             dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(), _at(dS0), cu_seqlens.data_ptr(), n, N, max_len, H, Hk, dk,
             dv, lq, lk, lv, mid, handle)
        return dq, dk_, dv_, dS0

    return _launch(idx, stream, body)


def packed_step(q, k, v, S, mode, g=None, slots=None, o=None, stream=None):
    """One token for each row (la_packed_step): q, k [n,Hk,dk], v [n,H,dv]; S
    [rows,H,dk,dv] fp32, updated in place at slots int32 [n] (None: row i).
    Returns o [n,H,dv]."""
    import torch
    N, H, Hk, dk, dv, lq, lk, lv, idx = _qkv(q, k, v)
    mid, rows = _mode(mode, q.dtype), S.shape[0]
    _check(S, "S", torch.float32, (rows, H, dk, dv), idx)
    _check(g, "g", torch.float32, (H,), idx)
    _check(slots, "slots", torch.int32, (N,), idx)
    _check(o, "o", q.dtype, (N, H, dv), idx)

    def body(handle):
        out = q.new_empty((N, H, dv)) if o is None else o
        _run("la_packed_step", q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(g), out.data_ptr(), S.data_ptr(), _at(slots),
             N, rows, H, Hk, dk, dv, lq, lk, lv, mid, handle)
        return out

    return _launch(idx, stream, body)


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
    idx, dt, Hk, ldk = _index(q, "q"), q.dtype, 0, 0
    if k is not None:
        Nk, Hk, dk, Tk, ldk = _tokens_of(k, "k")
        if Nk != N or dk != d or Tk != T or k.dtype is not dt or k.get_device() != idx:
            raise ValueError("q and k must agree in tokens, channels, layout, dtype and device")
    pairs = freq.numel()
    s = (pairs,) if sections is None else tuple(sections)
    axes = len(s)
    if sum(s) != pairs or not 1 <= axes <= 3:
        raise ValueError("sections: the pairs of one to three axes, as many as freq has")
    _check(pos, "pos", torch.int32, (N, axes), idx)
    _check(freq, "freq", torch.float64, (pairs,), idx)
    if T_out and N % T_out:
        raise ValueError("T_out must divide the tokens")
    shape = (N // T_out, H, T_out, d) if T_out else (N, H, d)
    kshape = (N // T_out, Hk, T_out, d) if T_out else (N, Hk, d)
    _check(q_out, "q_out", dt, shape, idx)
    _check(k_out, "k_out", dt, kshape, idx)
    flags = _flag(dt) | (LAYER_CONSTANTS["LA_ROT_INTERLEAVED"] if interleaved else 0) \
        | (LAYER_CONSTANTS["LA_ROT_INVERSE"] if inverse else 0)

    def body(handle):
        a = q.new_empty(shape) if q_out is None else q_out
        b = None if k is None else q.new_empty(kshape) if k_out is None else k_out
        _run("la_rotary", q.data_ptr(), _at(k), a.data_ptr(), _at(b), pos.data_ptr(), freq.data_ptr(), axes,
             *(s + (0, 0))[:3], N, H, Hk, d, T, T_out, ldq, ldk, scale_q, scale_k, flags, handle)
        return a, b

    return _launch(idx, stream, body)


def _block(x, w, gate, act, res, scale, w_next):
    """(N, G, d, T, act id, device) of an epilogue call."""
    import torch
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    N, G, d, T, _ = _tokens_of(x, "x")
    idx, dt, f32 = _index(x, "x"), x.dtype, torch.float32
    _check(gate, "gate", dt, (N, G, d), idx)
    _check(res, "res", dt, (N, G, d), idx)
    _check(w, "w", f32, (d,), idx)
    _check(scale, "scale", f32, (d,), idx)
    _check(w_next, "w_next", f32, (d,), idx)
    return N, G, d, T, ACT_IDS[act] if gate is not None else 0, idx


def epilogue(x, w=None, gate=None, act="silu", res=None, scale=None, w_next=None, with_next=None, eps=1e-5, out=None,
             next=None, stream=None):
    """End of a block (la_epilogue): out = res + scale * rmsnorm(x) w act(gate),
    next = rmsnorm(out) w_next. x [N,G,d] or head-major [B,G,T,d]; gate, res
    [N,G,d]; w, scale, w_next [d] fp32. next is computed with w_next, next or
    with_next. Returns (out, next or None)."""
    N, G, d, T, a, idx = _block(x, w, gate, act, res, scale, w_next)
    if with_next is None:
        with_next = w_next is not None or next is not None
    flags = _flag(x.dtype)
    _check(out, "out", x.dtype, (N, G, d), idx)
    _check(next, "next", x.dtype, (N, G, d), idx)

    def body(handle):
        o = x.new_empty((N, G, d)) if out is None else out
        n = None if not with_next else x.new_empty((N, G, d)) if next is None else next
        _run("la_epilogue", x.data_ptr(), _at(w), _at(gate), a, _at(res), _at(scale), _at(w_next), o.data_ptr(), _at(n),
             eps, N, G, d, T, flags, handle)
        return o, n

    return _launch(idx, stream, body)


def epilogue_bwd(x, d_out, w=None, gate=None, act="silu", res=None, scale=None, w_next=None, d_next=None, eps=1e-5,
                 stream=None):
    """Backward pass of epilogue (la_epilogue_bwd) from its inputs. d_out,
    d_next [N,G,d], one of them may be None. Returns a dict with dx (x's
    layout), dgate, dres, dw, dscale, dw_next (None where the forward had no
    such input)."""
    import torch
    N, G, d, T, a, idx = _block(x, w, gate, act, res, scale, w_next)
    flags = _flag(x.dtype)
    _check(d_out, "d_out", x.dtype, (N, G, d), idx)
    _check(d_next, "d_next", x.dtype, (N, G, d), idx)

    def body(handle):
        wide = (N, G, d)
        dx, dgate = torch.empty_like(x), None if gate is None else x.new_empty(wide)
        dres = None if res is None else x.new_empty(wide)
        dw, dscale, dw_next = (None if t is None else torch.empty_like(t) for t in (w, scale, w_next))
        _run("la_epilogue_bwd", x.data_ptr(), _at(w), _at(gate), a, _at(res), _at(scale), _at(w_next), _at(d_out),
             _at(d_next), dx.data_ptr(), _at(dgate), _at(dres), _at(dw), _at(dscale), _at(dw_next), eps, N, G, d, T, flags,
             handle)
        return {"dx": dx, "dgate": dgate, "dres": dres, "dw": dw, "dscale": dscale, "dw_next": dw_next}

    return _launch(idx, stream, body)
