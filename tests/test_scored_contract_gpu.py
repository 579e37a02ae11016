"""What the scored operators promise beside their formulas: precision without asking for it, and nothing from masked memory."""
import math

import numpy as np
import pytest
import torch

import exact_tiled_attention_46_b200 as fa
import oracle.scored as osc

import scored as S
from parity import need_gpu
from scored import BF, f64
from test_scored_gpu import CASES, cuda, decode_problem, forward, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert fa.device_status(reset=True) == (0, 0)


# -------------------------------------------------------------- precision --
# Without changes the call is the plain forward, bit for bit, whose P is bf16.
CHANGED = [n for n in CASES if n != "plain"]


@pytest.mark.parametrize("name", CHANGED)
def test_forward_keeps_sixteen_bits_of_p(name):
    """O in fp32 against the bound of P in two bf16 parts (half steps of half steps), 2^8 below that of one part."""
    p = problem(name, seed=6)
    o, lse = forward(p, o_dtype=torch.float32)
    for b, h, g, P, l, d, ok, Q, K, V, dO, err in p.heads():
        O, lim = S.o_bound(P, V, err, fine=True)
        S.check(f64(o)[b, :, h], O, lim, f"O[{b},:,{h}]", 2.0 ** -23)
    assert torch.equal(forward(p)[0], o.to(torch.bfloat16))


@pytest.mark.parametrize("name", CHANGED)
def test_backward_undoes_the_rounding_of_o(name):
    """The gradient without o_lo is that of O to 16 bits: the bits of the call with o_lo, inside the bound of two parts."""
    p = problem(name, seed=7)
    lo = torch.empty_like(p.q).cuda()
    o, lse = forward(p, o_lo=lo)
    args = (*cuda(p, "q", "k", "v"), o, p.do.cuda(), lse)
    grads = fa.bwd_scored(*args, grad_dtype=torch.float32, **p.how("cuda"))
    S.check_bwd(p, *grads, bf16_output=False, fine=True)
    given = fa.bwd_scored(*args, o_lo=lo, grad_dtype=torch.float32, **p.how("cuda"))
    assert torch.equal(grads[1], given[1]) and torch.equal(grads[2], given[2])       # dQ is summed in any order


def test_backward_of_a_part_of_the_context_takes_o_as_it_is():
    """O and log-sums of all keys beside a part of them: where o is no rounding of the part's own O, Delta is o's."""
    p = S.Problem(1, 4, 2, 200, 400, 64, causal=False, cap=8.0, seed=12)
    q, k, v, do = cuda(p, "q", "k", "v", "do")
    o, lse = forward(p)
    for part in (slice(0, 256), slice(256, 400)):
        ks, vs = k[:, part].contiguous(), v[:, part].contiguous()
        got = fa.bwd_scored(q, ks, vs, o, do, lse, grad_dtype=torch.float32, **p.how("cuda"))
        ref = fa.bwd_scored(q, ks, vs, o, do, lse, o_lo=torch.zeros_like(o), grad_dtype=torch.float32, **p.how("cuda"))
        assert torch.equal(got[2], ref[2])
        # an element that happens to round to o all the same moves Delta by half a step of its own at most
        for b, h, g, P, l, d, ok, Q, K, V, dO, err in p.heads():
            delta = BF * np.sum(np.abs(dO * (P @ V)), axis=1, keepdims=True) * (1 + 2.0 ** -6)
            Pp, dp, Kp = P[:, part], d[:, part], np.abs(K[part])
            # fp16's half step of dS twice, and fp32 sums
            dS = np.abs(Pp * (dO @ V[part].T - np.sum(dO * (P @ V), axis=1, keepdims=True)) * dp)
            lim = p.scale * (delta * (Pp * dp) + 2 * S.FP16 * (dS + delta * Pp) + 2.0 ** -20) @ Kp
            assert (np.abs(f64(got[0] - ref[0])[b, :, h]) <= lim).all()


# ----------------------------------------------------------------- decode --
@pytest.mark.parametrize("rows,bad,cap,append", [(90, 40, 0.0, False), (90, 0, 5.0, True), (900, 500, 5.0, True),
                                                 (900, 899, 0.0, False), (5000, 3, 0.0, True), (5000, 4999, 9.0, False)])
@pytest.mark.parametrize("value", (math.nan, math.inf))
def test_decode_shows_a_nan_score(rows, bad, cap, append, value):
    """A key whose score is no number makes its heads' results NaN and touches no other head or sequence."""
    q, k, v, args, _, _ = decode_problem(2, 6, 3, 64, [rows, rows], rows + 1, cap=cap, append=append, seed=rows)
    w0 = args["weights"].clone()
    o, lse = fa.decode_scored(q, k, v, **args)
    w = args["weights"].clone()
    args["weights"].copy_(w0)
    # an infinite score without a cap is one as well (inf - inf); with a cap it is the cap
    k[1, bad, 2] = 0.0
    k[1, bad, 2, 5] = value
    q[1, 4:, 5] = 1.0
    o2, lse2 = fa.decode_scored(q, k, v, **args)
    w2 = args["weights"]
    n = rows + (1 if append else 0)
    assert torch.equal(o2[0], o[0]) and torch.equal(o2[1, :4], o[1, :4]) and torch.equal(lse2[1, :4], lse[1, :4])
    assert torch.equal(w2[0], w[0]) and torch.equal(w2[1, :2], w[1, :2]) and torch.equal(w2[1, 2, n:], w0[1, 2, n:])
    if cap and value == math.inf:
        assert torch.isfinite(o2).all() and torch.isfinite(lse2).all() and torch.isfinite(w2).all()
    else:
        assert torch.isnan(o2[1, 4:]).all() and torch.isnan(lse2[1, 4:]).all() and torch.isnan(w2[1, 2, :n]).all()


def test_decode_shows_a_nan_query():
    q, k, v, args, _, _ = decode_problem(2, 4, 2, 128, [300, 0], 300, seed=2)
    q[:, 1, 7] = math.nan
    w0 = args["weights"].clone()
    o, lse = fa.decode_scored(q, k, v, **args)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, 1]) and torch.isfinite(o[0, [0, 2, 3]]).all()
    assert torch.isnan(args["weights"][0, 0, :300]).all() and torch.isfinite(args["weights"][0, 1]).all()
    assert torch.isneginf(lse[1]).all() and not o[1].any() and torch.equal(args["weights"][1], w0[1])


# ------------------------------------------------- what masked memory holds --
NEIGHBOURS = {
    "docs": dict(shape=(2, 4, 2, 330, 330, 64), docs=(60, 11)),
    "docs_cap": dict(shape=(2, 4, 2, 330, 330, 128), docs=(60, 11), cap=6.0),
    "docs_cap_bias": dict(shape=(2, 4, 1, 330, 330, 64), docs=(60, 11), cap=6.0, bias=True),
    "docs_not_causal": dict(shape=(2, 2, 2, 200, 200, 64), docs=(60, 0), causal=False, bias=True),
    "causal": dict(shape=(2, 4, 2, 260, 260, 128)),
    "causal_cap": dict(shape=(2, 4, 2, 260, 300, 64), cap=6.0),
    "prefix": dict(shape=(2, 2, 2, 260, 260, 64), prefix=[100, 31], bias=True),
}


def gradients(p, **kw):
    lo = torch.empty_like(p.q).cuda()
    o, lse = forward(p, o_lo=lo)
    return o, lse, fa.bwd_scored(*cuda(p, "q", "k", "v"), o, p.do.cuda(), lse, grad_dtype=torch.float32, **p.how("cuda"), **kw)


def same_sums(a, b, mag):
    """dQ sums its key tiles in any order: a rounding step of fp32 per addition, of sums of at most `mag`."""
    return float((a - b).abs().max() if a.numel() else 0.0) <= 2.0 ** -19 * mag


@pytest.mark.parametrize("pad", (math.nan, math.inf, -3e38, 40.0))
@pytest.mark.parametrize("c", (dict(B=3, Hq=4, Hkv=2, D=128, lens=[0, 37, 300], rows=320),
                               dict(B=3, Hq=20, Hkv=1, D=64, lens=[1, 38, 299], rows=320),
                               dict(B=2, Hq=24, Hkv=2, D=128, lens=[65, 301], rows=320, page=16),
                               dict(B=2, Hq=8, Hkv=1, D=64, lens=[65, 301], rows=320, starts=[3, 290])), ids=range(4))
def test_capped_decode_does_not_depend_on_rows_beside_its_own(c, pad):
    """The same bits whatever stands in the row to append, behind it, and before the first row; called again, the row is there."""
    q, k, v, args, _, _ = decode_problem(**c, append=True, cap=20.0, seed=31, pad=0.0)
    w0 = args["weights"].clone()
    want = [t.clone() for t in fa.decode_scored(q, k, v, **args)] + [args["weights"].clone()]
    args["weights"].copy_(w0)
    again = list(fa.decode_scored(q, k, v, **args)) + [args["weights"]]
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    q, k, v, args, _, _ = decode_problem(**c, append=True, cap=20.0, seed=31, pad=pad)
    for _ in range(2):
        args["weights"].copy_(w0)
        got = list(fa.decode_scored(q, k, v, **args)) + [args["weights"]]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("value", (math.nan, math.inf, 3e38, 200.0))
@pytest.mark.parametrize("name", ("docs", "docs_cap", "docs_cap_bias", "docs_not_causal"))
def test_documents_do_not_change_bits_of_each_other(name, value):
    """A document's keys, of any size, change no bit of o, lse and key weights of the others."""
    c = dict(NEIGHBOURS[name])
    p = S.Problem(*c.pop("shape"), seed=24, **c)
    o, lse = forward(p)
    w = fa.key_weights(*cuda(p, "q", "k"), lse, **p.how("cuda"))
    hit = p.docs[1][0] == p.docs[1][0, 150]
    p.k[0, hit] = value
    o2, lse2 = forward(p)
    w2 = fa.key_weights(*cuda(p, "q", "k"), lse2, **p.how("cuda"))
    keep = ~hit.cuda()
    assert torch.equal(o2[1], o[1]) and torch.equal(o2[0, keep], o[0, keep])
    assert torch.equal(lse2[0][:, keep], lse[0][:, keep])
    assert torch.equal(w2[1], w[1]) and torch.equal(w2[0][:, keep], w[0][:, keep])

@pytest.mark.parametrize("which", ("q", "k", "v", "do"))
@pytest.mark.parametrize("value", (math.nan, -math.inf))
@pytest.mark.parametrize("name", NEIGHBOURS)
def test_gradient_of_an_inf_or_nan_stays_with_its_pairs(name, value, which):
    """One element of one row of batch 0: NaN gradients for that row and for what is paired with it, nothing elsewhere."""
    c = dict(NEIGHBOURS[name])
    p = S.Problem(*c.pop("shape"), seed=21, **c)
    B, Hq, Hkv, Lq, Lk, D = p.shape
    _, _, ref = gradients(p)
    x, at = getattr(p, which), 150
    head = (x.shape[2] - 1)
    top = x.abs().max()
    x[0, at, head, 9] = 0.0
    assert x.abs().max() == top                                  # the scale of the others stays
    x[0, at, head, 9] = value
    o, lse, got = gradients(p)
    G = Hq // Hkv
    heads = list(range(head * G, head * G + G)) if which in "kv" else [head]
    ok = osc.scored_mask(0, Lq, Lk, p.causal, *(p.oracle_how()[n] for n in ("q_docs", "k_docs", "prefix")))
    nan_q, nan_k = np.zeros((B, Hq, Lq), bool), np.zeros((B, Hkv, Lk), bool)
    for h in heads:
        rows = ~np.isfinite(f64(o)[0, :, h]).all(axis=1) | np.isnan(f64(lse)[0, h])
        if which in ("q", "do"):
            rows[at] |= ok[at].any()
        nan_k[0, h // G] |= ok[rows].any(axis=0)
        nan_q[0, h] = rows
        if which in "kv":
            nan_q[0, h] |= ok[:, at]
            nan_k[0, h // G, at] |= ok[:, at].any()
    assert nan_q.any() and nan_k.any() and not nan_q[0, heads[0]].all()
    # keys whose queries all give what they gave (an infinite key may leave its queries a finite, other softmax)
    other = nan_k.copy()
    if which in "kv":
        other[0, head] |= ok[ok[:, at]].any(axis=0)
    for g, r, bad, new in zip(got, ref, (nan_q, nan_k, nan_k), (nan_q, other, other)):
        bad, new = (torch.from_numpy(m).permute(0, 2, 1).cuda() for m in (bad, new))
        assert torch.isnan(g[bad]).all() and torch.isfinite(g[~bad]).all()
        assert same_sums(g[~new], r[~new], 64.0) if g is got[0] else torch.equal(g[~new], r[~new])


@pytest.mark.parametrize("D,cap,bias", [(64, 0.0, False), (128, 7.0, False), (64, 7.0, False), (64, 0.0, True), (128, 7.0, True)])
@pytest.mark.parametrize("causal", (True, False))
def test_keys_that_no_query_sees_leave_the_gradient_alone(D, cap, bias, causal):
    """Documents before the window's own, in its tiles and in tiles of their own: NaN, inf and huge numbers there."""
    Lq, Lk = 200, 700
    kd = np.repeat(np.arange(7), 100)[None, :].astype(np.int32) + np.array([[0], [3]], np.int32)
    p = S.Problem(2, 4, 2, Lq, Lk, D, causal=causal, cap=cap, bias=bias, docs=kd, seed=22)
    p.docs[0][0, :], p.docs[0][1, :] = torch.tensor([5, 6]).repeat_interleave(100), 9      # of batch 1 only the last document
    hidden = ~np.isin(np.arange(Lk)[None, :] // 100, (5, 6)) | (np.array([[0], [1]]) & (np.arange(Lk)[None, :] // 100 == 5))
    hidden = torch.from_numpy(hidden.astype(bool))
    o, lse, ref = gradients(p)
    S.check_bwd(p, *ref, bf16_output=False, fine=True)
    for bad_k, bad_v in ((math.nan, math.inf), (3e38, -3e38), (-math.inf, 1e30)):
        p.k[hidden], p.v[hidden] = bad_k, bad_v
        o2, lse2, got = gradients(p)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
        assert not got[1][hidden.cuda()].any() and not got[2][hidden.cuda()].any()
        assert torch.isfinite(got[0]).all() and same_sums(got[0], ref[0], 64.0)


def test_keys_of_documents_in_any_order_that_no_query_has():
    """Document numbers in no order on both sides; a seen key after the causal edge counts as unseen."""
    rng = np.random.default_rng(23)
    kd = rng.integers(0, 40, (2, 500)).astype(np.int32)
    p = S.Problem(2, 2, 2, 300, 500, 64, docs=kd, seed=23)
    qd = rng.integers(20, 60, (2, 300)).astype(np.int32)
    p.docs = (torch.from_numpy(qd), p.docs[1])
    for causal, prefix in ((True, None), (False, None), (True, [130, 0])):
        p.causal, p.prefix = causal, None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
        ok = np.stack([osc.scored_mask(b, 300, 500, causal, qd, kd, prefix) for b in range(2)])
        hidden = torch.from_numpy(~ok.any(axis=1))
        k, v = p.k.clone(), p.v.clone()
        _, _, ref = gradients(p)
        S.check_bwd(p, *ref, bf16_output=False, fine=True)
        p.k[hidden], p.v[hidden] = 2e38, math.nan
        _, _, got = gradients(p)
        assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2]) and same_sums(got[0], ref[0], 64.0)
        p.k, p.v = k, v



# ------------------------------------------------------------ range of v --
@pytest.mark.parametrize("cap,bias,boost", [(0.0, False, 1.0), (0.0, True, 8.0), (20.0, False, 8.0), (30.0, True, 8.0), (50.0, False, 16.0),
                                            (50.0, True, 16.0), (50.6, False, 40.0), (55.0, False, 16.0), (70.0, True, 16.0)])
def test_values_far_from_one(cap, bias, boost):
    """V times a power of two gives O times that, to the bit upwards (p up to 2^32, 330 keys, |v| up to 2^78: below 2^127),
    and within the bounds down to 2^-40."""
    for sign in (1.0, -1.0):
        p = S.Problem(1, 2, 1, 260, 330, 64, cap=cap, bias=bias, boost=boost, docs=(150, 0), seed=41)
        p.k[:, :, :, 0], p.q[:, :, :, 0] = 4.0, sign * boost                      # scores towards one end of the cap
        o, lse = forward(p, o_dtype=torch.float32)
        S.check_fwd(p, o, lse, bf16_output=False)
        v = p.v.clone()
        p.v = v * 2.0 ** 75
        big, _ = forward(p, o_dtype=torch.float32)
        assert torch.equal(big, o * 2.0 ** 75)
        p.v = v * 2.0 ** -40
        if sign > 0 or not cap:
            small, lse = forward(p, o_dtype=torch.float32)
            S.check_fwd(p, small, lse, bf16_output=False)


# ------------------------------------------------------------------ capture --
def test_training_step_without_documents_captured():
    """No kernel of documents' facts ahead: the chain begins with a memset. Two graphs, one workspace, replayed in turn."""
    p, p2 = (S.Problem(2, 4, 2, 300, 300, 64, cap=9.0, bias=True, seed=s) for s in (61, 62))
    B, Hq, Hkv, Lq, Lk, D = p.shape
    q, k, v, do = cuda(p, "q", "k", "v", "do")
    how = p.how("cuda")
    ws = torch.empty(fa.bwd_scored_workspace_size(B, Hq, Lq, Lk, D), dtype=torch.uint8, device="cuda")

    def step():
        o, lse = fa.fwd_scored(q, k, v, **how)
        return (o, lse) + fa.bwd_scored(q, k, v, o, do, lse, workspace=ws, grad_dtype=torch.float32, **how)

    step()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for src in (p2, p):
        for a, b in zip((q, k, v, do), cuda(src, "q", "k", "v", "do")):
            a.copy_(b)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            S.check_fwd(src, *out[:2])
            S.check_bwd(src, *out[2:], bf16_output=False, fine=True)
        assert torch.equal(outs[0][3], outs[1][3]) and torch.equal(outs[0][4], outs[1][4])


# -------------------------------------------------------------- huge numbers --
@pytest.mark.parametrize("which", ("q", "k", "v", "do"))
@pytest.mark.parametrize("name", ("docs", "docs_cap", "docs_not_causal"))
def test_gradient_beside_a_document_of_huge_numbers(name, which):
    """Finite, and far past the range that the fp16 scales reach: the other documents' gradients keep their bits."""
    c = dict(NEIGHBOURS[name])
    p = S.Problem(*c.pop("shape"), seed=71, **c)
    x = getattr(p, which)
    hit = p.docs[1][0] == p.docs[1][0, 150]
    x[0, hit] = 0.0
    _, _, ref = gradients(p)
    x[0, hit] = 3e38
    _, _, got = gradients(p)
    keep = ~hit.cuda()
    for g, r in zip(got[1:], ref[1:]):
        assert torch.equal(g[1], r[1]) and torch.equal(g[0, keep], r[0, keep])
    assert same_sums(got[0][1], ref[0][1], 64.0) and same_sums(got[0][0, keep], ref[0][0, keep], 64.0)
