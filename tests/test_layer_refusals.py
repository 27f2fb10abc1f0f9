"""Host-side refusals of include/la_layer.h, one argument wrong at a time (no GPU needed): every call here
differs in one argument from one that passes the checks, and is refused for that argument."""
import os

import pytest
import torch

import gated_delta_rule_linear_gb300 as la
from gated_delta_rule_linear_gb300 import build as labuild

A = 0x10000  # fake, aligned device addresses: never dereferenced by a refused call
INF, NAN = float("inf"), float("nan")
INVALID, UNSUPPORTED = "LA_ERR_INVALID_ARG", "LA_ERR_UNSUPPORTED"


@pytest.fixture(scope="module", autouse=True)
def lib():
    labuild.build()
    return la.load_library()


SHAPE = dict(H=4, Hk=2, dk=128, dv=128, ldq=256, ldk=256, ldv=512, mode=0, stream=None)
GOOD = {  # no two tensors the same
    "la_packed_fwd": dict(q=A, k=2 * A, v=3 * A, g=None, o=4 * A, S0=5 * A, S_final=6 * A, cu_seqlens=7 * A, slots=8 * A,
                          n_seq=3, total=64, max_len=0, n_slots=5, **SHAPE),
    "la_packed_bwd": dict(q=A, k=2 * A, v=3 * A, g=None, dO=4 * A, S0=5 * A, dS_final=6 * A, dq=7 * A, dk_out=8 * A,
                          dv_out=9 * A, dS0=10 * A, cu_seqlens=11 * A, n_seq=3, total=64, max_len=0, **SHAPE),
    "la_packed_step": dict(q=A, k=2 * A, v=3 * A, g=None, o=4 * A, S=5 * A, slots=6 * A, n=4, n_slots=5, **SHAPE),
    "la_rotary": dict(q=A, k=2 * A, q_out=3 * A, k_out=4 * A, pos=5 * A, freq=6 * A, n_axes=1, s0=32, s1=0, s2=0, N=8,
                      H=2, Hk=1, d=64, T_in=0, T_out=0, ldq=128, ldk=64, scale_q=1.0, scale_k=1.0, flags=0, stream=None),
    "la_epilogue": dict(x=A, w=2 * A, gate=3 * A, act=0, res=4 * A, scale=5 * A, w_next=6 * A, out=7 * A, next=8 * A,
                        eps=1e-5, N=8, G=2, d=64, T=0, flags=0, stream=None),
    "la_epilogue_bwd": dict(x=A, w=2 * A, gate=3 * A, act=0, res=4 * A, scale=5 * A, w_next=6 * A, d_out=7 * A,
                            d_next=8 * A, dx=9 * A, dgate=10 * A, dres=11 * A, dw=12 * A, dscale=13 * A, dw_next=14 * A,
                            eps=1e-5, N=8, G=2, d=64, T=0, flags=0, stream=None),
}

HEADS = "H must be a multiple of Hk"
STRIDES = "token strides must cover"
ALIGNED = "16-byte aligned"
PACKED = [
    (dict(mode=9), INVALID, "unknown mode"),
    (dict(mode=0x200), INVALID, "unknown mode"),          # no non-causal form
    (dict(mode=1), UNSUPPORTED, "takes LA_LINEAR"),
    (dict(mode=4, g=32 * A), UNSUPPORTED, "takes LA_LINEAR"),  # a decay for each head only
    (dict(mode=5), UNSUPPORTED, "takes LA_LINEAR"),
    (dict(mode=2), INVALID, "g goes with LA_RETNET"),
    (dict(g=32 * A), INVALID, "g goes with LA_RETNET"),
    (dict(mode=2, g=32 * A + 2), INVALID, "g must be 4-byte aligned"),
    (dict(H=0), INVALID, HEADS),
    (dict(H=-4), INVALID, HEADS),
    (dict(H=3, Hk=2), INVALID, HEADS),
    (dict(Hk=0), INVALID, HEADS),
    (dict(H=65536, Hk=1, ldv=65536 * 128), INVALID, HEADS),
    (dict(dk=96), UNSUPPORTED, "dk and dv must be"),
    (dict(dv=256), UNSUPPORTED, "dk and dv must be"),
    (dict(ldq=248), INVALID, STRIDES),                     # narrower than the heads
    (dict(ldk=248), INVALID, STRIDES),
    (dict(ldv=504), INVALID, STRIDES),
    (dict(ldq=260), INVALID, STRIDES),                     # not a multiple of 16 bytes
    (dict(ldk=260), INVALID, STRIDES),
    (dict(ldv=516), INVALID, STRIDES),
    (dict(ldq=-256), INVALID, STRIDES),
    (dict(ldv=1 << 31), INVALID, STRIDES),
    (dict(q=None), INVALID, "are required"),
    (dict(k=None), INVALID, "are required"),
    (dict(v=None), INVALID, "are required"),
    (dict(q=A + 8), INVALID, ALIGNED),
    (dict(k=2 * A + 8), INVALID, ALIGNED),
    (dict(v=3 * A + 8), INVALID, ALIGNED),
]
SEQ = [
    (dict(cu_seqlens=None), INVALID, "cu_seqlens is required"),
    (dict(cu_seqlens=7 * A + 2), INVALID, "cu_seqlens and slots must be 4-byte aligned"),
    (dict(n_seq=0), INVALID, "n_seq must be >= 1"),
    (dict(total=-1), INVALID, "n_seq must be >= 1"),
    (dict(max_len=-1), INVALID, "n_seq must be >= 1"),
    (dict(S0=5 * A + 4), INVALID, ALIGNED),
]
NORM = [
    (dict(flags=1), INVALID, "unknown flag"),
    (dict(x=None), INVALID, "are required"),
    (dict(x=A + 1), INVALID, "aligned to their elements"),
    (dict(gate=3 * A + 1), INVALID, "aligned to their elements"),
    (dict(res=4 * A + 1), INVALID, "aligned to their elements"),
    (dict(x=A + 2, flags=la.LA_F32), INVALID, "aligned to their elements"),
    (dict(w=2 * A + 2), INVALID, "aligned to their elements"),
    (dict(scale=5 * A + 2), INVALID, "aligned to their elements"),
    (dict(w_next=6 * A + 2), INVALID, "aligned to their elements"),
    (dict(act=2), INVALID, "unknown act"),
    (dict(act=-1), INVALID, "unknown act"),
    (dict(eps=0.0), INVALID, "eps must be"),
    (dict(eps=-1e-5), INVALID, "eps must be"),
    (dict(eps=NAN), INVALID, "eps must be"),
    (dict(eps=INF), INVALID, "eps must be"),
    (dict(N=-1), INVALID, "N must be >= 0"),
    (dict(G=0), INVALID, "N must be >= 0"),
    (dict(N=1 << 30, G=4), INVALID, "N must be >= 0"),
    (dict(d=0), UNSUPPORTED, "d must be 1..16384"),
    (dict(d=16385), UNSUPPORTED, "d must be 1..16384"),
    (dict(T=3), INVALID, "N must be a multiple of T"),
    (dict(T=-2), INVALID, "N must be a multiple of T"),
]
CASES = {
    "la_packed_fwd": PACKED + SEQ + [
        (dict(o=None), INVALID, "are required"),
        (dict(o=4 * A + 8), INVALID, ALIGNED),
        (dict(S_final=6 * A + 8), INVALID, ALIGNED),
        (dict(slots=None, n_slots=2), INVALID, "n_slots must be"),   # fewer rows than sequences
        (dict(n_slots=-1), INVALID, "n_slots must be"),
        (dict(slots=8 * A + 1), INVALID, "cu_seqlens and slots must be 4-byte aligned"),
        (dict(o=A), INVALID, "o must not be an input"),
        (dict(o=2 * A), INVALID, "o must not be an input"),
        (dict(o=3 * A), INVALID, "o must not be an input"),
    ],
    "la_packed_bwd": PACKED + SEQ + [
        (dict(dO=None), INVALID, "are required"),
        (dict(dq=None), INVALID, "are required"),
        (dict(dk_out=None), INVALID, "are required"),
        (dict(dv_out=None), INVALID, "are required"),
        (dict(dO=4 * A + 8), INVALID, ALIGNED),
        (dict(dS_final=6 * A + 4), INVALID, ALIGNED),
        (dict(dq=7 * A + 2), INVALID, ALIGNED),
        (dict(dk_out=8 * A + 2), INVALID, ALIGNED),
        (dict(dv_out=9 * A + 2), INVALID, ALIGNED),
        (dict(dS0=10 * A + 4), INVALID, ALIGNED),
        (dict(dq=A), INVALID, "outputs must not be inputs"),
        (dict(dk_out=7 * A), INVALID, "outputs must not be inputs"),
        (dict(dv_out=4 * A), INVALID, "outputs must not be inputs"),
        (dict(dS0=5 * A), INVALID, "outputs must not be inputs"),
        (dict(dS0=6 * A), INVALID, "outputs must not be inputs"),
    ],
    "la_packed_step": PACKED + [
        (dict(n=-1), INVALID, "n must be >= 0"),
        (dict(n_slots=-1), INVALID, "n must be >= 0"),
        (dict(slots=None, n=6), INVALID, "n must be >= 0"),          # more rows than states
        (dict(o=None), INVALID, "are required"),
        (dict(S=None), INVALID, "are required"),
        (dict(S=5 * A + 4), INVALID, ALIGNED),
        (dict(o=4 * A + 8), INVALID, ALIGNED),
        (dict(slots=6 * A + 2), INVALID, "slots 4-byte aligned"),
        (dict(n=1 << 30), INVALID, "n*H too large"),
        (dict(o=3 * A), INVALID, "o must not be an input"),
    ],
    "la_rotary": [
        (dict(flags=0x200), INVALID, "unknown flag"),
        (dict(k=None), INVALID, "k and k_out go together"),
        (dict(k_out=None), INVALID, "k and k_out go together"),
        (dict(q=None), INVALID, "are required"),
        (dict(q_out=None), INVALID, "are required"),
        (dict(pos=None), INVALID, "are required"),
        (dict(freq=None), INVALID, "are required"),
        (dict(q=A + 1), INVALID, "aligned to their elements"),
        (dict(k_out=4 * A + 1), INVALID, "aligned to their elements"),
        (dict(pos=5 * A + 2), INVALID, "aligned to their elements"),
        (dict(freq=6 * A + 4), INVALID, "aligned to their elements"),
        (dict(n_axes=0), INVALID, "n_axes must be 1..3"),
        (dict(n_axes=4), INVALID, "n_axes must be 1..3"),
        (dict(s1=-1), INVALID, "n_axes must be 1..3"),
        (dict(s0=16, s1=4), INVALID, "n_axes must be 1..3"),         # a section of an axis that is not there
        (dict(n_axes=2, s0=16, s2=4), INVALID, "n_axes must be 1..3"),
        (dict(s0=33), INVALID, "pairs must be at least one and fit d"),
        (dict(s0=0), INVALID, "pairs must be at least one and fit d"),
        (dict(d=1), UNSUPPORTED, "d must be 2..512"),
        (dict(d=1024, ldq=2048, ldk=1024), UNSUPPORTED, "d must be 2..512"),
        (dict(N=-1), INVALID, "N must be >= 0"),
        (dict(H=0), INVALID, "N must be >= 0"),
        (dict(Hk=0), INVALID, "N must be >= 0"),
        (dict(H=65536, ldq=65536 * 64), INVALID, "N must be >= 0"),
        (dict(T_in=5), INVALID, "N must be a multiple of T_in"),
        (dict(T_out=7), INVALID, "N must be a multiple of T_in"),
        (dict(T_out=-1), INVALID, "N must be a multiple of T_in"),
        (dict(ldq=127), INVALID, "token strides must cover"),
        (dict(ldk=63), INVALID, "token strides must cover"),
        (dict(scale_q=INF), INVALID, "scales must be finite"),
        (dict(scale_k=NAN), INVALID, "scales must be finite"),
        (dict(q_out=A, T_out=4), INVALID, "only with the same layout"),   # in place into another layout
        (dict(q_out=A, ldq=256), INVALID, "only with the same layout"),   # ... or out of strided rows
        (dict(k_out=2 * A, ldk=128), INVALID, "only with the same layout"),
        (dict(q_out=4 * A), INVALID, "are two tensors"),
        (dict(q_out=2 * A), INVALID, "are two tensors"),
        (dict(k_out=A), INVALID, "are two tensors"),
    ],
    "la_epilogue": NORM + [
        (dict(out=None), INVALID, "are required"),
        (dict(out=7 * A + 1), INVALID, "aligned to their elements"),
        (dict(next=8 * A + 1), INVALID, "aligned to their elements"),
        (dict(next=None), INVALID, "w_next goes with next"),
        (dict(next=7 * A), INVALID, "out and next are two tensors"),
        (dict(T=4, out=A), INVALID, "not a head-major x"),
        (dict(T=4, next=A), INVALID, "not a head-major x"),
    ],
    "la_epilogue_bwd": NORM + [
        (dict(d_out=None, d_next=None, dw_next=None, w_next=None), INVALID, "one of d_out and d_next"),
        (dict(gate=None), INVALID, "dgate needs gate"),
        (dict(d_next=None), INVALID, "need d_next"),
        (dict(d_next=None, w_next=None), INVALID, "need d_next"),
        (dict(d_next=None, dw_next=None), INVALID, "need d_next"),
        (dict(dx=9 * A + 1), INVALID, "aligned to their elements"),
        (dict(dw=12 * A + 2), INVALID, "aligned to their elements"),
        (dict(dscale=13 * A + 2), INVALID, "aligned to their elements"),
        (dict(dw_next=14 * A + 2), INVALID, "aligned to their elements"),
        (dict(dx=A), INVALID, "outputs must not be inputs"),
        (dict(dx=7 * A), INVALID, "outputs must not be inputs"),
        (dict(dgate=7 * A), INVALID, "outputs must not be inputs"),
        (dict(dres=8 * A), INVALID, "outputs must not be inputs"),
        (dict(dw=2 * A), INVALID, "outputs must not be inputs"),
        (dict(dscale=12 * A), INVALID, "outputs must not be inputs"),
    ],
}


@pytest.mark.parametrize("fn,kw,code,message", [(fn, *c) for fn, cases in CASES.items() for c in cases],
                         ids=lambda x: x if isinstance(x, str) else None)
def test_refusal(fn, kw, code, message):
    rc = getattr(la, fn)(**{**GOOD[fn], **kw})
    said = la.la_last_error()
    assert rc == la.CONSTANTS[code] and said.startswith(fn + ":") and message in said, (rc, said)


@pytest.mark.parametrize("fn,kw", [
    # the arguments that the cases start from, with what the host itself answers: nothing to do, or no device
    ("la_packed_step", dict(n=0)), ("la_rotary", dict(N=0)), ("la_epilogue", dict(N=0)),
    ("la_epilogue_bwd", dict(N=0, dw=None, dscale=None, dw_next=None)),
])
def test_nothing_to_do(fn, kw):
    assert getattr(la, fn)(**{**GOOD[fn], **kw}) == 0, la.la_last_error()


@pytest.mark.parametrize("fn", ["la_packed_fwd", "la_packed_bwd", "la_packed_step", "la_rotary", "la_epilogue",
                                "la_epilogue_bwd"])
def test_the_arguments_before_the_change_pass(fn):
    # Without a device a call that passes every check ends at the launch. With one it would run on the fake addresses:
    # there the cases themselves show it, as each names its own check.
    if torch.cuda.is_available() or os.path.exists("/dev/nvidiactl") or os.path.exists("/dev/nvidia0"):
        pytest.skip("a device is there")
    rc = getattr(la, fn)(**GOOD[fn])
    said = la.la_last_error()
    assert rc == la.LA_ERR_CUDA, (rc, said)
