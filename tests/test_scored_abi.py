"""What the scored entry points, key weights and cache eviction refuse, and the fitted tanh (no GPU needed)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import exact_tiled_attention_46_b200 as fa
from exact_tiled_attention_46_b200 import build as fabuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNS, OK = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_OK
P = 1 << 20            # a fake, aligned "device" address: never dereferenced on these paths
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


def score(softcap=0.0, slopes=None, q_docs=None, k_docs=None, prefix=None):
    return ctypes.byref(fa._Score(softcap, slopes, q_docs, k_docs, prefix))


FWD = dict(q=P, k=P, v=P, o=P, o_lo=None, lse=None, B=1, Hq=2, Hkv=1, Lq=8, Lk=8, D=64, scale=0.1, causal=1, score=score(),
           o_dtype=0, ws=None, nbytes=0, stream=None)
FWD_BAD = [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(o=None), BAD), (dict(q=P + 2), BAD), (dict(lse=P + 2), BAD),
    (dict(Hq=3, Hkv=2), BAD), (dict(B=0), BAD), (dict(Lq=-1), BAD), (dict(D=96), UNS), (dict(scale=0.0), BAD),
    (dict(scale=INF), BAD), (dict(o_dtype=5), BAD), (dict(score=None), BAD), (dict(score=score(softcap=-1.0)), BAD),
    (dict(score=score(softcap=NAN)), BAD), (dict(score=score(softcap=INF)), BAD),
    (dict(scale=1e30, score=score(softcap=1e-30)), BAD),                 # scale / softcap overflows
    (dict(score=score(slopes=P + 1)), BAD), (dict(score=score(q_docs=P)), BAD), (dict(score=score(k_docs=P)), BAD),
    (dict(score=score(q_docs=P, k_docs=P)), BAD),                        # documents need the workspace
    (dict(score=score(q_docs=P, k_docs=P), ws=P, nbytes=31), BAD),
    (dict(score=score(q_docs=P, k_docs=P), ws=P + 4, nbytes=1 << 20), BAD),
    (dict(score=score(prefix=P), causal=0), BAD), (dict(score=score(prefix=P + 2)), BAD),
    (dict(score=score(slopes=P), Lk=1 << 24), UNS), (dict(B=70000), UNS), (dict(B=1 << 16, Hq=1 << 16), UNS), (dict(o_lo=P + 8), BAD), (dict(o_lo=P, o_dtype=1), BAD),
]


@pytest.mark.parametrize("change,expect", FWD_BAD, ids=range(len(FWD_BAD)))
def test_fwd_refuses(L, change, expect):
    assert L.fa_fwd_scored(*dict(FWD, **change).values()) == expect


def test_slopes_refuse_a_scale_that_they_cannot_be_divided_by(L):
    for fn, base in ((L.fa_fwd_scored, FWD), (L.fa_bwd_scored, BWD)):
        assert fn(*dict(base, scale=2.0 ** -65, score=score(slopes=P)).values()) == UNS


def test_empty_calls_do_nothing(L):
    assert L.fa_fwd_scored(*dict(FWD, Lq=0).values()) == OK
    assert L.fa_key_weights(P, P, P, P, 0, 0, 1, 2, 1, 8, 0, 64, 0.1, 1, score(), P, 0, None) == OK


BWD = dict(q=P, k=P, v=P, o=P, o_lo=None, dO=P, lse=P, dq=P, dk=P, dv=P, B=1, Hq=2, Hkv=1, Lq=8, Lk=8, D=64, scale=0.1, causal=1,
           score=score(), grad_dtype=0, ws=P, nbytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(score=None), BAD), (dict(dO=None), BAD), (dict(lse=None), BAD), (dict(dk=P + 4), BAD), (dict(D=32), UNS),
    (dict(nbytes=100), BAD), (dict(ws=P + 16), BAD), (dict(grad_dtype=2), BAD), (dict(score=score(softcap=-2.0)), BAD),
    (dict(score=score(prefix=P), causal=0), BAD), (dict(score=score(k_docs=P)), BAD), (dict(B=70000), UNS),
    (dict(score=score(slopes=P), Lq=1 << 24), UNS), (dict(o_lo=P + 2), BAD)], ids=range(14))
def test_bwd_refuses(L, change, expect):
    assert L.fa_bwd_scored(*dict(BWD, **change).values()) == expect


def test_bwd_workspace_is_checked_to_the_byte(L):
    need = fa.bwd_scored_workspace_size(1, 2, 8, 8, 64)
    assert need >= fa.bwd_workspace_size(1, 2, 8, 64) + fa.scored_workspace_size(1, 8, 8)
    assert L.fa_bwd_scored(*dict(BWD, nbytes=need - 1).values()) == BAD


def test_bwd_workspace_holds_the_keys_that_no_query_sees():
    """128 bits per key tile beside the tile facts, which other calls do without."""
    for B, Lk in ((1, 8), (3, 129), (2, 5000)):
        extra = fa.bwd_scored_workspace_size(B, 2, 64, Lk, 64) - fa.bwd_workspace_size(B, 2, 64, 64) - fa.scored_workspace_size(B, 64, Lk)
        assert extra >= B * -(-Lk // 128) * 16 and extra % 256 == 0


DEC = dict(q=P, k_new=None, v_new=None, k=P, v=P, table=None, lens=P, starts=None, o=P, lse=None, weights=None, ld=0, B=2,
           Hq=4, Hkv=2, num=2, page=100, pps=1, D=64, scale=0.1, softcap=0.0, slopes=None, o_dtype=0, ws=P, nbytes=0,
           stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), BAD), (dict(lens=None), BAD), (dict(lens=P + 1), BAD), (dict(k_new=P), BAD), (dict(v_new=P), BAD),
    (dict(Hq=5), BAD), (dict(num=3), BAD), (dict(pps=2), BAD), (dict(page=0), BAD), (dict(softcap=-1.0), BAD),
    (dict(softcap=NAN), BAD), (dict(scale=-1.0), BAD), (dict(D=80), UNS), (dict(o_dtype=3), BAD),
    (dict(table=P, page=24, num=9, pps=4), UNS), (dict(weights=P, ld=99, nbytes=1 << 30), BAD),
    (dict(weights=P + 2, ld=100, nbytes=1 << 30), BAD), (dict(starts=P + 2), BAD), (dict(slopes=P + 3), BAD),
    (dict(slopes=P, page=1 << 24, nbytes=1 << 62), UNS), (dict(nbytes=1), BAD), (dict(ws=None), BAD), (dict(ws=P + 128), BAD),
    (dict(B=70000, num=70000), UNS), (dict(table=P, page=1 << 20, num=9, pps=1 << 12), UNS)], ids=range(25))
def test_decode_refuses(L, change, expect):
    a = dict(DEC, **change)
    if "nbytes" not in change:
        a["nbytes"] = 1 << 60
    assert L.fa_decode_scored_splitkv(*a.values()) == expect


def test_decode_workspace(L):
    base = fa.decode_scored_workspace_size(2, 4, 2, 100, 64)
    assert fa.decode_scored_workspace_size(2, 4, 2, 100, 64, True) >= base + 2 * 4 * 100 * 4
    assert L.fa_decode_scored_splitkv(*dict(DEC, nbytes=base - 1).values()) == BAD
    assert L.fa_decode_scored_splitkv(*dict(DEC, weights=P, ld=100, nbytes=base).values()) == BAD
    assert fa.decode_scored_workspace_size(0, 4, 2, 100, 64) == 0 == fa.decode_scored_workspace_size(1, 5, 2, 100, 64)


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(lse=None), BAD), (dict(w=None), BAD), (dict(ld=7), BAD),
    (dict(k=P + 8), BAD), (dict(D=72), UNS), (dict(score=None), BAD), (dict(score=score(q_docs=P)), BAD),
    (dict(ws=None), BAD), (dict(nbytes=0), BAD), (dict(ws=P + 16), BAD), (dict(Hkv=3), BAD), (dict(scale=0.0), BAD),
    (dict(score=score(prefix=P), causal=0), BAD), (dict(B=70000), UNS)], ids=range(16))
def test_key_weights_refuses(L, change, expect):
    a = dict(dict(q=P, k=P, lse=P, w=P, ld=8, acc=0, B=1, Hq=4, Hkv=2, Lq=8, Lk=8, D=64, scale=0.1, causal=1,
                  score=score(), ws=P, nbytes=1 << 30, stream=None), **change)
    assert L.fa_key_weights(*a.values()) == expect


FAR = P + (1 << 24)
ROWS = dict(k=P, v=P + (1 << 16), page_table=None, page_size=64, pages_per_seq=1, num_pages=2)   # 2 * 64 * 2 * 64 * 2 bytes
OUT = dict(ROWS, k=FAR, v=FAR + (1 << 16))
EV = dict(src=ROWS, dst=OUT, w=P + (1 << 20), w_ld=64, w2=FAR + (1 << 20), w2_ld=64, n=P + (1 << 21), n2=FAR + (1 << 21),
          kept=FAR + (1 << 22), B=2, Hkv=2, D=64, keep=32, recent=8, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(src=None), BAD), (dict(dst=None), BAD), (dict(w=None), BAD), (dict(kept=None), BAD), (dict(n2=None), BAD),
    (dict(keep=0), BAD), (dict(recent=-1), BAD), (dict(recent=33), BAD), (dict(keep=65), BAD), (dict(w_ld=63), BAD),
    (dict(w2_ld=31), BAD), (dict(D=60), UNS), (dict(D=8192), UNS), (dict(src=dict(ROWS, k=None)), BAD),
    (dict(src=dict(ROWS, v=P)), BAD), (dict(src=dict(ROWS, k=P + 8)), BAD), (dict(dst=dict(OUT, page_size=0)), BAD),
    (dict(dst=dict(OUT, page_table=P, num_pages=0)), BAD), (dict(src=dict(ROWS, page_table=P + 2)), BAD),
    (dict(dst=dict(OUT, k=P)), BAD),                              # k in place, v not
    (dict(dst=dict(OUT, k=P + 4096)), BAD),                       # overlaps the source's k
    (dict(dst=dict(OUT, v=P + 4096)), BAD),
    (dict(dst=dict(ROWS, page_table=P, num_pages=4, pages_per_seq=2)), BAD),   # in place through another table
    (dict(w2=P + (1 << 20), w2_ld=40), BAD), (dict(w2=P + (1 << 20) + 128), BAD), (dict(B=70000), UNS)], ids=range(26))
def test_evict_refuses(L, change, expect):
    a = dict(EV, **change)
    for side in ("src", "dst"):
        if a[side] is not None:
            a[side] = ctypes.byref(fa._KvRows(*a[side].values()))
    assert L.fa_cache_evict(*a.values()) == expect


def test_evict_refuses_lengths_that_overlap_in_part(L):
    """One block would write a length that another one has yet to read."""
    a = dict(EV, n2=EV["n"] + 4, src=ctypes.byref(fa._KvRows(*ROWS.values())), dst=ctypes.byref(fa._KvRows(*OUT.values())))
    assert L.fa_cache_evict(*a.values()) == BAD
    assert L.fa_cache_evict(*dict(a, n2=EV["n"] - 4).values()) == BAD


def test_bindings_refuse_before_the_library():
    """CPU tensors, types, shapes and half-given pairs raise TypeError or ValueError."""
    t = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    w, n = torch.zeros(1, 2, 8), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fa.fwd_scored(t, t, t), lambda: fa.bwd_scored(t, t, t, t, t, w),
                 lambda: fa.decode_scored(t[:, 0], t, t, n), lambda: fa.key_weights(t, t, w),
                 lambda: fa.cache_evict(t, t, w, n, 4), lambda: fa.fwd_scored(None, t, t)):
        with pytest.raises(TypeError):
            call()


def test_fitted_tanh_meets_its_bound():
    txt = open(os.path.join(ROOT, "exact_tiled_attention_46_b200", "csrc", "tanh_poly.cuh")).read()
    deg = int(re.search(r"FA_TANH_POLY_DEGREE (\d+)", txt).group(1))
    c = np.array([float(re.search(rf"FA_TANH_C{i} ([-0-9.e]+)f", txt).group(1)) for i in range(deg + 1)], dtype=np.float32)
    bound = float(re.search(r"#define FA_TANH_MAX_REL_ERR ([-0-9.e]+)", txt).group(1))
    limit = float(re.search(r"#define FA_TANH_LIMIT ([-0-9.e]+)f", txt).group(1))
    y = np.linspace(1e-4, limit, 200001)
    p = np.zeros_like(y)
    for a in c[::-1].astype(np.float64):
        p = p * y * y + a
    assert np.max(np.abs(y * p / np.tanh(y) - 1)) <= bound * 1.001
    assert bound < 2.0 ** -23                                      # below fp32's own rounding of the score
    assert math.isclose(float(c[0]), 1.0, rel_tol=2.0 ** -23)
