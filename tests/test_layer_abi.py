"""Host-side checks of include/la_layer.h (no GPU needed): the library exports
what the header declares and rejects bad arguments before touching a device."""
import os
import re
import subprocess

import pytest

import gated_delta_rule_linear_gb300 as la
from gated_delta_rule_linear_gb300 import build as labuild

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "la_layer.h")
A = 0x10000  # fake, aligned device address: never dereferenced by a refused call


@pytest.fixture(scope="module", autouse=True)
def lib():
    labuild.build()
    return la.load_library()


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(la_[a-z_]+)\s*\(", text))
    assert names == set(la.LAYER_SIGNATURES) == {"la_packed_fwd", "la_packed_bwd", "la_packed_step", "la_rotary",
                                                 "la_epilogue", "la_epilogue_bwd"}
    out = subprocess.run(["nm", "-D", "--defined-only", la.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (la_[a-z_]+)\b", out))
    for name in names:  # as many arguments in the binding as in the header
        decl = re.search(rf"\b{name}\s*\(([^)]*)\)", text).group(1)
        assert len(decl.split(",")) == len(la.LAYER_SIGNATURES[name][0]), name


def refused(fn, args, kw, code):
    rc = getattr(la, fn)(**{**args, **kw})
    msg = la.la_last_error()
    assert rc == la.CONSTANTS[code], (rc, msg)
    assert msg.startswith(fn + ":"), msg


PACKED = [
    (dict(mode=9), "LA_ERR_INVALID_ARG"),
    (dict(mode=0x200), "LA_ERR_INVALID_ARG"),            # no non-causal form
    (dict(mode=4, g=A), "LA_ERR_UNSUPPORTED"),           # a decay for each head only
    (dict(mode=5), "LA_ERR_UNSUPPORTED"),
    (dict(mode=2), "LA_ERR_INVALID_ARG"),                # retnet needs g
    (dict(g=A), "LA_ERR_INVALID_ARG"),                   # linear takes none
    (dict(mode=2, g=A + 2), "LA_ERR_INVALID_ARG"),
    (dict(H=0), "LA_ERR_INVALID_ARG"),
    (dict(H=3, Hk=2), "LA_ERR_INVALID_ARG"),             # shared heads divide
    (dict(Hk=0), "LA_ERR_INVALID_ARG"),
    (dict(dk=96), "LA_ERR_UNSUPPORTED"),
    (dict(dv=256), "LA_ERR_UNSUPPORTED"),
    (dict(ldq=64), "LA_ERR_INVALID_ARG"),                # narrower than the heads
    (dict(ldk=260), "LA_ERR_INVALID_ARG"),               # not a multiple of 16 bytes
    (dict(ldv=(1 << 31)), "LA_ERR_INVALID_ARG"),
    (dict(q=None), "LA_ERR_INVALID_ARG"),
    (dict(v=A + 8), "LA_ERR_INVALID_ARG"),
]
SEQ = [
    (dict(cu_seqlens=None), "LA_ERR_INVALID_ARG"),
    (dict(cu_seqlens=A + 2), "LA_ERR_INVALID_ARG"),
    (dict(n_seq=0), "LA_ERR_INVALID_ARG"),
    (dict(total=-1), "LA_ERR_INVALID_ARG"),
    (dict(max_len=-1), "LA_ERR_INVALID_ARG"),
    (dict(S0=A + 4), "LA_ERR_INVALID_ARG"),
]


@pytest.mark.parametrize("kw,code", PACKED + SEQ + [
    (dict(o=None), "LA_ERR_INVALID_ARG"),
    (dict(S_final=A + 8), "LA_ERR_INVALID_ARG"),
    (dict(S0=A, n_slots=2), "LA_ERR_INVALID_ARG"),       # fewer rows than sequences, no slots
    (dict(S0=A, slots=A, n_slots=-1), "LA_ERR_INVALID_ARG"),
    (dict(slots=A + 1), "LA_ERR_INVALID_ARG"),
])
def test_packed_fwd_refusals(kw, code):
    refused("la_packed_fwd", dict(q=A, k=A, v=A, g=None, o=A, S0=None, S_final=None, cu_seqlens=A, slots=None, n_seq=3,
                                  total=64, max_len=0, n_slots=3, H=4, Hk=2, dk=128, dv=128, ldq=256, ldk=256, ldv=512,
                                  mode=0, stream=None), kw, code)


@pytest.mark.parametrize("kw,code", PACKED + SEQ + [
    (dict(dO=None), "LA_ERR_INVALID_ARG"),
    (dict(dq=None), "LA_ERR_INVALID_ARG"),
    (dict(dk_out=A + 2), "LA_ERR_INVALID_ARG"),
    (dict(dS0=A + 4), "LA_ERR_INVALID_ARG"),
    (dict(dS_final=A + 4), "LA_ERR_INVALID_ARG"),
])
def test_packed_bwd_refusals(kw, code):
    refused("la_packed_bwd", dict(q=A, k=A, v=A, g=None, dO=A, S0=None, dS_final=None, dq=A, dk_out=A, dv_out=A, dS0=None,
                                  cu_seqlens=A, n_seq=3, total=64, max_len=0, H=4, Hk=2, dk=128, dv=128, ldq=256, ldk=256,
                                  ldv=512, mode=0, stream=None), kw, code)


@pytest.mark.parametrize("kw,code", PACKED + [
    (dict(n=-1), "LA_ERR_INVALID_ARG"),
    (dict(n=5), "LA_ERR_INVALID_ARG"),                   # more rows than states, no slots
    (dict(S=None), "LA_ERR_INVALID_ARG"),
    (dict(S=A + 4), "LA_ERR_INVALID_ARG"),
    (dict(n=1 << 30, slots=A), "LA_ERR_INVALID_ARG"),
])
def test_packed_step_refusals(kw, code):
    refused("la_packed_step", dict(q=A, k=A, v=A, g=None, o=A, S=A, slots=None, n=4, n_slots=4, H=4, Hk=2, dk=128, dv=128,
                                   ldq=256, ldk=256, ldv=512, mode=0, stream=None), kw, code)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=0x200), "LA_ERR_INVALID_ARG"),
    (dict(k=None), "LA_ERR_INVALID_ARG"),                # k_out without k
    (dict(q=None), "LA_ERR_INVALID_ARG"),
    (dict(freq=A + 4), "LA_ERR_INVALID_ARG"),
    (dict(pos=None), "LA_ERR_INVALID_ARG"),
    (dict(n_axes=0), "LA_ERR_INVALID_ARG"),
    (dict(n_axes=4), "LA_ERR_INVALID_ARG"),
    (dict(s1=4), "LA_ERR_INVALID_ARG"),                  # a section of an axis that is not there
    (dict(s0=33), "LA_ERR_INVALID_ARG"),                 # more pairs than channels
    (dict(s0=0), "LA_ERR_INVALID_ARG"),
    (dict(d=1024), "LA_ERR_UNSUPPORTED"),
    (dict(N=-1), "LA_ERR_INVALID_ARG"),
    (dict(H=0), "LA_ERR_INVALID_ARG"),
    (dict(Hk=0), "LA_ERR_INVALID_ARG"),
    (dict(T_in=5), "LA_ERR_INVALID_ARG"),
    (dict(T_out=7), "LA_ERR_INVALID_ARG"),
    (dict(ldq=64), "LA_ERR_INVALID_ARG"),
    (dict(scale_q=float("inf")), "LA_ERR_INVALID_ARG"),
    (dict(q_out=A, T_out=4), "LA_ERR_INVALID_ARG"),      # in place into another layout
    (dict(q_out=A, ldq=256), "LA_ERR_INVALID_ARG"),      # ... or out of strided rows
])
def test_rotary_refusals(kw, code):
    refused("la_rotary", dict(q=A, k=A, q_out=2 * A, k_out=2 * A, pos=A, freq=A, n_axes=1, s0=32, s1=0, s2=0, N=8, H=2, Hk=1,
                              d=64, T_in=0, T_out=0, ldq=128, ldk=64, scale_q=1.0, scale_k=1.0, flags=0, stream=None), kw,
            code)


BLOCK = [
    (dict(flags=1), "LA_ERR_INVALID_ARG"),
    (dict(x=None), "LA_ERR_INVALID_ARG"),
    (dict(x=A + 1), "LA_ERR_INVALID_ARG"),
    (dict(w=A + 2), "LA_ERR_INVALID_ARG"),
    (dict(act=2), "LA_ERR_INVALID_ARG"),
    (dict(eps=0.0), "LA_ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "LA_ERR_INVALID_ARG"),
    (dict(eps=float("inf")), "LA_ERR_INVALID_ARG"),
    (dict(N=-1), "LA_ERR_INVALID_ARG"),
    (dict(G=0), "LA_ERR_INVALID_ARG"),
    (dict(d=0), "LA_ERR_UNSUPPORTED"),
    (dict(d=16385), "LA_ERR_UNSUPPORTED"),
    (dict(T=3), "LA_ERR_INVALID_ARG"),
]


@pytest.mark.parametrize("kw,code", BLOCK + [
    (dict(out=None), "LA_ERR_INVALID_ARG"),
    (dict(next=None), "LA_ERR_INVALID_ARG"),             # w_next without next
    (dict(next=2 * A), "LA_ERR_INVALID_ARG"),            # out and next are one tensor
    (dict(T=4, out=A), "LA_ERR_INVALID_ARG"),            # over a head-major x
])
def test_epilogue_refusals(kw, code):
    refused("la_epilogue", dict(x=A, w=A, gate=A, act=0, res=A, scale=A, w_next=A, out=2 * A, next=3 * A, eps=1e-5, N=8, G=2,
                                d=64, T=0, flags=0, stream=None), kw, code)


@pytest.mark.parametrize("kw,code", BLOCK + [
    (dict(d_out=None, d_next=None, dw_next=None, w_next=None), "LA_ERR_INVALID_ARG"),
    (dict(gate=None), "LA_ERR_INVALID_ARG"),             # dgate without gate
    (dict(d_next=None), "LA_ERR_INVALID_ARG"),           # w_next without d_next
    (dict(dw=A + 2), "LA_ERR_INVALID_ARG"),
])
def test_epilogue_bwd_refusals(kw, code):
    refused("la_epilogue_bwd", dict(x=A, w=A, gate=A, act=0, res=A, scale=A, w_next=A, d_out=A, d_next=A, dx=2 * A,
                                    dgate=3 * A, dres=4 * A, dw=A, dscale=A, dw_next=A, eps=1e-5, N=8, G=2, d=64, T=0,
                                    flags=0, stream=None), kw, code)


SHAPE = dict(H=4, Hk=2, dk=128, dv=128, ldq=256, ldk=256, ldv=512, mode=0, stream=None)
APART = {
    "la_packed_fwd": dict(q=A, k=2 * A, v=3 * A, g=None, o=4 * A, S0=5 * A, S_final=5 * A, cu_seqlens=6 * A, slots=None,
                          n_seq=3, total=64, max_len=0, n_slots=3, **SHAPE),
    "la_packed_bwd": dict(q=A, k=2 * A, v=3 * A, g=None, dO=4 * A, S0=5 * A, dS_final=6 * A, dq=7 * A, dk_out=8 * A,
                          dv_out=9 * A, dS0=10 * A, cu_seqlens=11 * A, n_seq=3, total=64, max_len=0, **SHAPE),
    "la_packed_step": dict(q=A, k=2 * A, v=3 * A, g=None, o=4 * A, S=5 * A, slots=None, n=4, n_slots=4, **SHAPE),
    "la_rotary": dict(q=A, k=2 * A, q_out=3 * A, k_out=4 * A, pos=5 * A, freq=6 * A, n_axes=1, s0=32, s1=0, s2=0, N=8,
                      H=1, Hk=1, d=64, T_in=0, T_out=0, ldq=64, ldk=64, scale_q=1.0, scale_k=1.0, flags=0, stream=None),
    "la_epilogue_bwd": dict(x=A, w=2 * A, gate=3 * A, act=0, res=4 * A, scale=5 * A, w_next=6 * A, d_out=7 * A,
                            d_next=8 * A, dx=9 * A, dgate=10 * A, dres=11 * A, dw=12 * A, dscale=13 * A, dw_next=14 * A,
                            eps=1e-5, N=8, G=2, d=64, T=0, flags=0, stream=None),
}


@pytest.mark.parametrize("fn,out,other", [
    ("la_packed_fwd", "o", "q"), ("la_packed_fwd", "o", "k"), ("la_packed_fwd", "o", "v"),
    ("la_packed_bwd", "dq", "q"), ("la_packed_bwd", "dk_out", "v"), ("la_packed_bwd", "dv_out", "dO"),
    ("la_packed_bwd", "dq", "dk_out"), ("la_packed_bwd", "dS0", "dS_final"), ("la_packed_bwd", "dS0", "S0"),
    ("la_packed_step", "o", "q"), ("la_packed_step", "o", "v"),
    ("la_rotary", "q_out", "k"), ("la_rotary", "k_out", "q"), ("la_rotary", "q_out", "k_out"),
    ("la_epilogue_bwd", "dx", "x"), ("la_epilogue_bwd", "dx", "d_out"), ("la_epilogue_bwd", "dgate", "gate"),
    ("la_epilogue_bwd", "dres", "d_next"), ("la_epilogue_bwd", "dres", "dx"), ("la_epilogue_bwd", "dw", "w"),
    ("la_epilogue_bwd", "dscale", "dw_next"),
])
def test_an_output_is_no_input(fn, out, other):
    refused(fn, APART[fn], {out: APART[fn][other]}, "LA_ERR_INVALID_ARG")


def test_wrappers_refuse_cpu_tensors():
    import torch
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        la.packed_fwd(x, x, x, torch.zeros(2, dtype=torch.int32), "linear")
    with pytest.raises(ValueError):
        la.packed_step(x, x, x, torch.zeros(4, 2, 64, 64), "linear")
    with pytest.raises(ValueError):
        la.rotary(x, None, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        la.epilogue(x)
    with pytest.raises(ValueError):
        la.epilogue_bwd(x, x)
