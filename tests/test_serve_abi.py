"""Host-side checks of include/la_serve.h (no GPU needed): the library exports what the header declares, and refuses
calls that differ in one argument from one that passes the checks, for that argument."""
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_linear_gb300 as la
from gated_delta_rule_linear_gb300 import build as labuild

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "la_serve.h")
A = 0x10000  # fake, aligned device addresses: never dereferenced by a refused call
INF, NAN = float("inf"), float("nan")
INVALID, UNSUPPORTED = "LA_ERR_INVALID_ARG", "LA_ERR_UNSUPPORTED"


@pytest.fixture(scope="module", autouse=True)
def lib():
    labuild.build()
    return la.load_library()


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(la_[a-z_]+)\s*\(", text))
    assert names == set(la.SERVE_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", la.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (la_[a-z_]+)\b", out))
    kinds = {"*": "c_void_p", "int": "c_int", "long long": "c_long", "float": "c_float"}
    for name in names:  # the binding's arguments are the header's, in kind and number
        decl = re.search(rf"\b{name}\s*\(([^)]*)\)", text, re.S).group(1)
        args = [" ".join(a.split()) for a in decl.split(",")]
        want = [kinds["*"] if "*" in a or a.startswith("la_stream_t") else kinds["long long"] if a.startswith("long long")
                else kinds[a.split()[0]] for a in args]
        assert [t.__name__.replace("c_longlong", "c_long") for t in la.SERVE_SIGNATURES[name][0]] == want, name


CACHE = dict(page_size=16, n_pages=9, max_pages=5, ld_table=5)
GOOD = {
    "la_cache_append": dict(q=A, k=2 * A, v=3 * A, q_out=4 * A, k_cache=5 * A, v_cache=6 * A, table=7 * A, lens=8 * A,
                            cu_seqlens=9 * A, pos=10 * A, freq=11 * A, n_axes=2, s0=20, s1=12, s2=0, n_seq=3, total=9,
                            H=4, Hk=2, d=64, ldq=256, ldk=128, ldv=128, ld_page=2048, flags=0, stream=None, **CACHE),
    "la_paged_attn": dict(q=A, k_cache=2 * A, v_cache=3 * A, o=4 * A, lse=5 * A, table=6 * A, lens=7 * A, n=3, H=4, Hk=2,
                          d=64, max_len=0, window=0, scale=0.125, ldq=256, ld_page=2048, flags=0, stream=None, **CACHE),
    "la_beam_select": dict(logits=A, scores=2 * A, done=3 * A, scores_out=4 * A, parent=5 * A, token=6 * A, B=2, W=4,
                           V=100, K=4, ld=104, eos=5, flags=0, stream=None),
    "la_beam_states": dict(pool=A, slots=2 * A, parent=3 * A, B=2, W=4, n_slots=9, layers=2, row_bytes=64, ld_row=64,
                           ld_layer=640, stream=None),
    "la_beam_cache": dict(k_cache=A, v_cache=2 * A, table=3 * A, lens=4 * A, parent=5 * A, B=2, W=4, layers=2,
                          token_bytes=256, ld_page=4096, ld_layer=40960, stream=None, **CACHE),
}

PAGES = [
    (dict(page_size=0), INVALID, "page_size must be"),
    (dict(n_pages=-1), INVALID, "page_size must be"),
    (dict(max_pages=-1), INVALID, "page_size must be"),
    (dict(ld_table=4), INVALID, "ld_table must be"),
    (dict(ld_page=2047), INVALID, "ld_page must cover"),
    (dict(page_size=2000000000), INVALID, "ld_page must cover"),
    (dict(table=7 * A + 2), INVALID, "table and lens must be 4-byte aligned"),
    (dict(lens=8 * A + 1), INVALID, "table and lens must be 4-byte aligned"),
]
BAD = {
    "la_cache_append": PAGES + [
        (dict(flags=2), INVALID, "unknown flag"),
        (dict(q=None), INVALID, "q and q_out go together"),
        (dict(q_out=None), INVALID, "q and q_out go together"),
        (dict(n_seq=-1), INVALID, "n_seq and total"),
        (dict(total=-1), INVALID, "n_seq and total"),
        (dict(cu_seqlens=None), INVALID, "n_seq and total"),  # nine tokens of three sequences
        (dict(H=0), INVALID, "H and Hk"),
        (dict(H=65536, ldq=65536 * 64), INVALID, "H and Hk"),
        (dict(Hk=0), INVALID, "H and Hk"),
        (dict(d=0), UNSUPPORTED, "d must be 1..512"),
        (dict(d=513), UNSUPPORTED, "d must be 1..512"),
        (dict(n_axes=4), INVALID, "n_axes must be"),
        (dict(n_axes=1), INVALID, "n_axes must be"),
        (dict(s2=1), INVALID, "n_axes must be"),
        (dict(s0=-1), INVALID, "n_axes must be"),
        (dict(s0=21), INVALID, "pairs must be"),
        (dict(s0=0, s1=0), INVALID, "pairs must be"),
        (dict(s0=2 ** 31 - 1, s1=2 ** 31 - 1), INVALID, "pairs must be"),
        (dict(freq=None), INVALID, "freq goes with"),
        (dict(n_axes=0, s0=0, s1=0, pos=None), INVALID, "freq goes with"),
        (dict(n_axes=0, s0=0, s1=0, freq=None), INVALID, "pos goes with"),
        (dict(pos=None), INVALID, "pos goes with"),
        (dict(ldq=255), INVALID, "token strides"),
        (dict(ldk=127), INVALID, "token strides"),
        (dict(ldv=127), INVALID, "token strides"),
        (dict(k=None), INVALID, "are required"),
        (dict(v=None), INVALID, "are required"),
        (dict(lens=None), INVALID, "are required"),
        (dict(table=None), INVALID, "are required"),
        (dict(k_cache=None), INVALID, "are required"),
        (dict(v_cache=None), INVALID, "are required"),
        (dict(q=A + 1), INVALID, "aligned to their elements"),
        (dict(k_cache=5 * A + 2, flags=la.LA_F32), INVALID, "aligned to their elements"),
        (dict(cu_seqlens=9 * A + 2), INVALID, "aligned to their elements"),
        (dict(pos=10 * A + 2), INVALID, "aligned to their elements"),
        (dict(freq=11 * A + 4), INVALID, "aligned to their elements"),
        (dict(k_cache=2 * A), INVALID, "must not be inputs"),
        (dict(v_cache=3 * A), INVALID, "must not be inputs"),
        (dict(v_cache=5 * A), INVALID, "must not be inputs"),
        (dict(q_out=2 * A), INVALID, "must not be inputs"),
        (dict(q_out=6 * A), INVALID, "must not be inputs"),
        (dict(k_cache=A), INVALID, "must not be inputs"),
        (dict(q_out=A, ldq=264), INVALID, "only if that is dense"),
    ],
    "la_paged_attn": PAGES + [
        (dict(flags=1), INVALID, "unknown flag"),
        (dict(n=-1), INVALID, "must be >= 0"),
        (dict(max_len=-1), INVALID, "must be >= 0"),
        (dict(window=-1), INVALID, "must be >= 0"),
        (dict(H=0), INVALID, "H must be a multiple"),
        (dict(H=3), INVALID, "H must be a multiple"),
        (dict(Hk=0), INVALID, "H must be a multiple"),
        (dict(H=65536, ldq=65536 * 64), INVALID, "H must be a multiple"),
        (dict(d=96), UNSUPPORTED, "d must be 64, 128 or 256"),
        (dict(d=32), UNSUPPORTED, "d must be 64, 128 or 256"),
        (dict(scale=INF), INVALID, "scale must be finite"),
        (dict(scale=NAN), INVALID, "scale must be finite"),
        (dict(ldq=248), INVALID, "ldq must cover"),
        (dict(ldq=260), INVALID, "ldq must cover"),
        (dict(ld_page=2052), INVALID, "ldq must cover"),
        (dict(n=2 ** 29), INVALID, "n*H too large"),
        (dict(q=None), INVALID, "are required"),
        (dict(o=None), INVALID, "are required"),
        (dict(lens=None), INVALID, "are required"),
        (dict(table=None), INVALID, "are required"),
        (dict(k_cache=None), INVALID, "are required"),
        (dict(v_cache=None), INVALID, "are required"),
        (dict(q=A + 8), INVALID, "16-byte aligned"),
        (dict(o=4 * A + 8), INVALID, "16-byte aligned"),
        (dict(k_cache=2 * A + 8), INVALID, "16-byte aligned"),
        (dict(v_cache=3 * A + 8), INVALID, "16-byte aligned"),
        (dict(lse=5 * A + 2), INVALID, "16-byte aligned"),
        (dict(o=A), INVALID, "must not be inputs"),
        (dict(o=3 * A), INVALID, "must not be inputs"),
        (dict(lse=4 * A), INVALID, "must not be inputs"),
    ],
    "la_beam_select": [
        (dict(flags=2), INVALID, "unknown flag"),
        (dict(B=-1), INVALID, "B must be >= 0"),
        (dict(V=0), INVALID, "B must be >= 0"),
        (dict(W=0), UNSUPPORTED, "W must be 1..32"),
        (dict(W=33), UNSUPPORTED, "W must be 1..32"),
        (dict(K=0), UNSUPPORTED, "K must be 1..32"),
        (dict(K=33), UNSUPPORTED, "K must be 1..32"),
        (dict(W=1, V=3, ld=3, eos=1), INVALID, "K must be <= W*V"),
        (dict(V=2 ** 30, ld=2 ** 30), INVALID, "W*V below 2^31"),
        (dict(W=1, V=2 ** 31 - 1, ld=2 ** 31), INVALID, "W*V below 2^31"),
        (dict(B=2 ** 28), INVALID, "too large"),
        (dict(ld=99), INVALID, "ld must be >= V"),
        (dict(eos=100), INVALID, "eos must be"),
        (dict(eos=-1), INVALID, "eos must be"),
        (dict(logits=None), INVALID, "are required"),
        (dict(scores=None), INVALID, "are required"),
        (dict(scores_out=None), INVALID, "are required"),
        (dict(parent=None), INVALID, "are required"),
        (dict(token=None), INVALID, "are required"),
        (dict(logits=A + 1), INVALID, "aligned to their elements"),
        (dict(logits=A + 2, flags=la.LA_F32), INVALID, "aligned to their elements"),
        (dict(parent=5 * A + 2), INVALID, "aligned to their elements"),
        (dict(scores_out=2 * A), INVALID, "must not be inputs"),
        (dict(token=5 * A), INVALID, "must not be inputs"),
        (dict(parent=3 * A), INVALID, "must not be inputs"),
    ],
    "la_beam_states": [
        (dict(B=-1), INVALID, "must be >= 0"),
        (dict(layers=-1), INVALID, "must be >= 0"),
        (dict(n_slots=-1), INVALID, "must be >= 0"),
        (dict(row_bytes=-4), INVALID, "must be >= 0"),
        (dict(W=0), UNSUPPORTED, "W must be 1..32"),
        (dict(W=33), UNSUPPORTED, "W must be 1..32"),
        (dict(slots=None, n_slots=7), INVALID, "n_slots must be >= B*W"),
        (dict(B=2 ** 27), INVALID, "too large"),
        (dict(row_bytes=62), INVALID, "multiples of 4"),
        (dict(ld_row=66), INVALID, "multiples of 4"),
        (dict(ld_layer=642), INVALID, "multiples of 4"),
        (dict(ld_row=60), INVALID, "ld_row must cover"),
        (dict(ld_layer=-640), INVALID, "ld_row must cover"),
        (dict(row_bytes=2 ** 34, ld_row=2 ** 34), INVALID, "below 2^34"),
        (dict(pool=None), INVALID, "are required"),
        (dict(parent=None), INVALID, "are required"),
        (dict(pool=A + 2), INVALID, "4-byte aligned"),
        (dict(slots=2 * A + 2), INVALID, "4-byte aligned"),
        (dict(parent=3 * A + 2), INVALID, "4-byte aligned"),
        (dict(pool=3 * A), INVALID, "must not be another"),
    ],
    "la_beam_cache": PAGES[:4] + [
        (dict(ld_page=4092), INVALID, "ld_page must cover"),
        (dict(table=3 * A + 2), INVALID, "table and lens"),
        (dict(lens=4 * A + 2), INVALID, "table and lens"),
        (dict(B=-1), INVALID, "must be >= 0"),
        (dict(layers=-1), INVALID, "must be >= 0"),
        (dict(token_bytes=-4), INVALID, "must be >= 0"),
        (dict(W=0), UNSUPPORTED, "W must be 1..32"),
        (dict(W=33), UNSUPPORTED, "W must be 1..32"),
        (dict(layers=2 ** 26), INVALID, "too large"),
        (dict(token_bytes=254), INVALID, "multiples of 4"),
        (dict(ld_page=4098), INVALID, "multiples of 4"),
        (dict(ld_layer=40962), INVALID, "multiples of 4"),
        (dict(ld_layer=-4), INVALID, "ld_layer must be"),
        (dict(token_bytes=2 ** 32, ld_page=2 ** 40), INVALID, "below 2^34"),
        (dict(table=None), INVALID, "are required"),
        (dict(lens=None), INVALID, "are required"),
        (dict(parent=None), INVALID, "are required"),
        (dict(k_cache=None), INVALID, "are required"),
        (dict(v_cache=None), INVALID, "are required"),
        (dict(k_cache=A + 2), INVALID, "4-byte aligned"),
        (dict(parent=5 * A + 2), INVALID, "4-byte aligned"),
        (dict(v_cache=A), INVALID, "must not be another"),
        (dict(table=4 * A), INVALID, "must not be another"),
    ],
}


@pytest.mark.parametrize("fn,kw,code,text", [(f, *case) for f, cases in BAD.items() for case in cases])
def test_refusal(fn, kw, code, text):
    rc = getattr(la, fn)(**{**GOOD[fn], **kw})
    msg = la.la_last_error()
    assert rc == la.CONSTANTS[code], (rc, msg)
    assert msg.startswith(fn + ": ") and text in msg, msg


@pytest.mark.parametrize("fn,kw", [
    ("la_cache_append", dict(total=0)), ("la_cache_append", dict(n_seq=0)), ("la_paged_attn", dict(n=0)),
    ("la_beam_select", dict(B=0)), ("la_beam_states", dict(B=0)), ("la_beam_states", dict(layers=0)),
    ("la_beam_states", dict(row_bytes=0)), ("la_beam_cache", dict(B=0)), ("la_beam_cache", dict(max_pages=0, ld_table=0)),
])
def test_nothing_to_do(fn, kw):
    """The call that the refusals start from passes the checks: with nothing to do it returns before any launch."""
    assert getattr(la, fn)(**{**GOOD[fn], **kw}) == la.CONSTANTS["LA_OK"], la.la_last_error()


def test_wrappers_refuse():
    f = torch.zeros
    x, i = f(4, 2, 64), torch.int32
    cache, table, lens = f(3, 16, 2, 64), f(4, 5, dtype=i), f(4, dtype=i)
    for call in (lambda: la.cache_append(x, x, x, cache, cache, table, lens), lambda: la.paged_attn(x, cache, cache, table, lens),
                 lambda: la.beam_select(f(2, 3, 9), f(2, 3)), lambda: la.beam_states(cache, f(1, 3, dtype=i)),
                 lambda: la.beam_cache(cache, cache, table, lens, f(2, 2, dtype=i))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        la.beam_select(f(2, 9), f(2))
    with pytest.raises(ValueError):
        la.paged_attn(f(4, 128), cache, cache, table, lens)
