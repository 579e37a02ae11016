"""The scored operators with more work items than the GPU has SMs, every value against the fp64 oracle.

Small problems give each CTA one item at most, of one query tile. Here items hold two query tiles of different key
ranges, CTAs take several items one after the other (shared-memory rings, TMEM buffers and barrier phases carry over),
and some items have nothing to do.
"""
import numpy as np
import pytest
import torch

import exact_tiled_attention_46_b200 as fa

import scored as S
from parity import need_gpu
from scored import BF, FP16, f64
from test_scored_gpu import check_decode, cuda, decode_problem, forward

pytestmark = pytest.mark.gpu
SMS = 148


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert fa.device_status(reset=True) == (0, 0)


def tiles(n, rows=128):
    return -(-n // rows)


# (query range of 256, batch row, head): two rounds of the SMs at least
FORWARD = {
    "cap": dict(shape=(4, 36, 12, 520, 520, 128), cap=30.0, boost=4.0),
    "docs_bias": dict(shape=(5, 30, 10, 530, 610, 64), docs=(70, 300), bias=True),
    "docs_cap_prefix": dict(shape=(4, 40, 20, 515, 515, 64), docs=(200, 150), cap=20.0, prefix=[500, 0, 77, 300]),
    "bias_both_sides": dict(shape=(5, 32, 4, 500, 700, 128), causal=False, bias=True, cap=9.0),
    "more_queries": dict(shape=(4, 38, 19, 600, 170, 64), cap=15.0),
    "plain_prefix": dict(shape=(5, 31, 31, 510, 510, 128), prefix=[0, 400, 510, 1, 256]),
}


@pytest.mark.parametrize("name", FORWARD)
def test_forward_many_items(name):
    c = dict(FORWARD[name])
    p = S.Problem(*c.pop("shape"), seed=51, **c)
    B, Hq, Hkv, Lq, Lk, D = p.shape
    assert tiles(Lq, 256) * B * Hq > 2 * SMS
    o, lse = forward(p, o_dtype=torch.float32)
    S.check_fwd(p, o, lse, bf16_output=False)
    lo = torch.empty_like(p.q).cuda()
    o2, lse2 = forward(p, o_lo=lo)
    assert torch.equal(o2, o.to(torch.bfloat16)) and torch.equal(lse2, lse)
    assert torch.equal(lo, (o - o2.float()).to(torch.bfloat16))


# (key tile, batch row, kv head)
BACKWARD = {
    "cap": dict(shape=(4, 24, 24, 400, 400, 64), cap=30.0, boost=4.0),
    "cap_128": dict(shape=(5, 36, 18, 390, 390, 128), cap=30.0),
    "docs_bias": dict(shape=(5, 32, 16, 300, 660, 64), docs=(50, 140), bias=True),
    "docs_cap_bias_prefix": dict(shape=(6, 20, 20, 333, 333, 128), docs=(120, 200), cap=12.0, bias=True, prefix=[300, 0, 1, 130, 333, 50]),
    "not_causal": dict(shape=(5, 30, 15, 260, 640, 64), causal=False, bias=True),
    "more_queries": dict(shape=(8, 20, 20, 500, 250, 128)),
}


def check_gradients(p, dq, dk, dv, fine):
    """scored.check_bwd's bounds (fp32 outputs) and one step that so many draws come to meet: dO enters as fp16, its
    largest magnitude scaled into [2^-2, 2^0), where fp16's smallest half step is 2^-25. So an element is off by at
    most 2^-25 / 2^-2 of that magnitude, which counts where dO itself is tiny: once in dV, once in dP.
    """
    B, Hq, Hkv, Lq, Lk, D = p.shape
    rk, rv, bk, bv = (np.zeros((B, Lk, Hkv, D)) for _ in range(4))
    dq, dk, dv = f64(dq), f64(dk), f64(dv)
    off = 2.0 ** -23 * float(p.do.abs().max())
    for b, h, g, P, l, d, ok, Q, K, V, dO, err in p.heads():
        O, o_err = S.o_bound(P, V, err, fine)
        dP = dO @ V.T
        Delta = np.sum(dO * O, axis=1, keepdims=True)
        dZ = P * (dP - Delta) * d
        e = 4.0 * err[:, None]
        delta = np.sum(np.abs(dO) * ((BF * BF if fine else BF) * np.abs(O) + (1 + BF) * o_err), axis=1, keepdims=True)
        dp_err = 2.0 ** -21 * np.abs(dO) @ np.abs(V).T + off * np.abs(V).sum(axis=1)
        tiny = 2.0 ** -24 * 2.0 * np.abs(dO).max(initial=0.0) * np.abs(V).max(initial=0.0) * D * ok
        z_err = (FP16 + e) * np.abs(dZ) + P * d * (delta + dp_err) + tiny + 2.0 ** -20 * P * np.abs(dP - Delta)
        p_err = (FP16 + e) * P + 2.0 ** -25 * ok
        rv[b, :, g] += P.T @ dO
        bv[b, :, g] += p_err.T @ np.abs(dO) + 2.0 ** -20 * (P.T @ np.abs(dO)) + off * P.sum(axis=0)[:, None]
        rk[b, :, g] += p.scale * (dZ.T @ Q)
        bk[b, :, g] += p.scale * (z_err.T @ np.abs(Q)) + 2.0 ** -20 * p.scale * (np.abs(dZ).T @ np.abs(Q))
        S.check(dq[b, :, h], p.scale * (dZ @ K),
                p.scale * (z_err @ np.abs(K)) + 2.0 ** -20 * p.scale * (np.abs(dZ) @ np.abs(K)), f"dQ[{b},:,{h}]", 2.0 ** -23)
    S.check(dv, rv, bv, "dV", 2.0 ** -23)
    S.check(dk, rk, bk, "dK", 2.0 ** -23)


@pytest.mark.parametrize("name", BACKWARD)
def test_backward_many_items(name):
    c = dict(BACKWARD[name])
    p = S.Problem(*c.pop("shape"), seed=52, **c)
    B, Hq, Hkv, Lq, Lk, D = p.shape
    assert tiles(Lk) * B * Hkv > 2 * SMS
    o, lse = forward(p)
    grads = fa.bwd_scored(*cuda(p, "q", "k", "v"), o, p.do.cuda(), lse, grad_dtype=torch.float32, **p.how("cuda"))
    check_gradients(p, *grads, fine="docs" in c or c.get("cap") or c.get("bias"))


# parts of a key tile's (query tile, head) pairs: one where they are eight at most
WEIGHTS = {
    "one_part": dict(shape=(6, 20, 20, 380, 510, 64), cap=20.0),
    "one_part_docs": dict(shape=(5, 30, 30, 300, 300, 128), docs=(60, 170), bias=True),
    "parts": dict(shape=(3, 64, 8, 500, 900, 128), cap=20.0, bias=True),
    "parts_docs": dict(shape=(4, 60, 6, 600, 900, 64), docs=(100, 400), cap=9.0),
    "parts_prefix": dict(shape=(4, 48, 6, 400, 800, 128), prefix=[700, 0, 300, 129], bias=True),
}


@pytest.mark.parametrize("name", WEIGHTS)
def test_key_weights_many_items(name):
    c = dict(WEIGHTS[name])
    p = S.Problem(*c.pop("shape"), seed=53, **c)
    B, Hq, Hkv, Lq, Lk, D = p.shape
    one = tiles(Lq) * (Hq // Hkv) <= 8
    assert one == name.startswith("one") and tiles(Lk) * B * Hkv * (1 if one else 2) > 2 * SMS
    _, lse = forward(p)
    q, k = cuda(p, "q", "k")
    w = fa.key_weights(q, k, lse, **p.how("cuda"))
    ref, tol = np.zeros((B, Hkv, Lk)), np.zeros((B, Hkv, Lk))
    for b, h, g, P, l, d, ok, Q, K, V, dO, err in p.heads():
        ref[b, g] += P.sum(axis=0)
        tol[b, g] += ((4.0 * err + 2.0 ** -20)[:, None] * P).sum(axis=0)
    # score and log-sum are off by err each, the fp32 sum by its rounding steps
    assert (np.abs(f64(w) - ref) <= tol + 2.0 ** -18 * ref + 1e-30).all()
    wide = torch.full((B, Hkv, Lk + 3), 1.0, device="cuda")
    fa.key_weights(q, k, lse, weights=wide, **p.how("cuda"))
    assert torch.equal(wide[:, :, :Lk], 1.0 + w) and (wide[:, :, Lk:] == 1.0).all()


LENGTHS = [0, 1, 700, 255, 256, 257, 512, 699]
DECODE = {
    "weights": dict(B=40, Hq=24, Hkv=8, D=128, rows=700, cap=8.0),
    "append_bias": dict(B=40, Hq=24, Hkv=8, D=64, rows=701, append=True, cap=8.0, bias=True),
    "paged_append": dict(B=48, Hq=8, Hkv=8, D=128, rows=704, page=32, append=True),
    "starts_groups": dict(B=24, Hq=48, Hkv=4, D=64, rows=700, starts=[0, 1, 300, 255, 100, 256, 511, 5] * 3, bias=True),
}


@pytest.mark.parametrize("name", DECODE)
def test_decode_many_items(name):
    """More chunks than the three CTAs of every SM take at once: the items come from the counter."""
    c = dict(DECODE[name])
    G = c["Hq"] // c["Hkv"]
    heads = 1 if G == 1 else 4 if G <= 4 else 8
    groups = c["B"] * c["Hkv"] * tiles(G, heads)
    chunk = next((n for n in (1024, 512, 256) if groups * tiles(c["rows"] + bool(c.get("append")), n) >= 6 * SMS), 128)
    assert groups * tiles(c["rows"], chunk) > 2 * 3 * SMS
    q, k, v, args, reference, n_of = decode_problem(lens=(LENGTHS * 6)[:c["B"]], seed=54, **c)
    w0 = args["weights"].clone()
    kv0 = k.clone(), v.clone()
    o, lse = fa.decode_scored(q, k, v, o_dtype=torch.float32, **args)
    check_decode(o, lse, args["weights"], reference(), bf16_output=False)
    got = args["weights"].clone()
    args["weights"].copy_(w0)
    k.copy_(kv0[0]); v.copy_(kv0[1])
    o2, lse2 = fa.decode_scored(q, k, v, o_dtype=torch.float32, **args)
    assert torch.equal(o2, o) and torch.equal(lse2, lse) and torch.equal(args["weights"], got)      # whatever the order
