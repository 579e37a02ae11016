"""Cases of attention with capped, distance-biased and document-masked scores, and of a cache thinned by attention weight.

Five kinds of case, each with its plain form and the calls that a user makes:

* ``fwd``     prefill forward: scores capped by a tanh, a bias that grows with
              the distance, documents packed into one row, a prefix that every
              query sees
* ``train``   the same forward and its gradient, as one training step makes them
* ``decode``  one new token over a (paged) cache, with its row appended or not
              and the attention weight of every cached row added up or not
* ``weights`` the attention weight that a prompt's queries give each key
* ``evict``   the rows with the largest weight, and the most recent ones, moved
              to the front of a smaller cache

What decides how much work a case is (documents, lengths) follows from the case
alone; the values follow from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

NEG_INF = float("-inf")
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def _attn(kind, name, B, Hq, Hkv, Lq, Lk, D, causal=True, cap=0.0, bias=False, doc=0, pad=0, prefix=0, boost=1):
    """doc: mean document length (0: no documents); pad: unused tokens at the end of the last row."""
    return {"name": name, "kind": kind, "B": B, "Hq": Hq, "Hkv": Hkv, "Lq": Lq, "Lk": Lk, "D": D, "causal": causal,
            "cap": cap, "bias": bias, "doc": doc, "pad": pad, "prefix": prefix, "boost": boost}


def _decode(name, B, Hq, Hkv, D, lo, hi, page=0, append=False, weights=False, cap=0.0, bias=False, start=False):
    return {"name": name, "kind": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "page": page,
            "append": append, "weights": weights, "cap": cap, "bias": bias, "start": start}


def _evict(name, B, Hkv, D, lo, hi, keep, recent):
    return {"name": name, "kind": "evict", "B": B, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "keep": keep,
            "recent": recent}


def listed():
    return [
        # short documents of a fine-tuning set packed into one row, with unused tokens at its end
        _attn("fwd", "fwd_docs_short", 1, 8, 8, 1000, 1000, 64, doc=90, pad=37),
        # a batch of prompts of a model whose scores are capped
        _attn("fwd", "fwd_capped", 4, 16, 16, 2048, 2048, 128, cap=50.0, boost=4),
        # a long prompt of a model with a distance bias, its first part seen by every query
        _attn("fwd", "fwd_bias_prefix_long", 1, 32, 8, 8191, 8191, 128, bias=True, prefix=1501),
        # a small fine-tuning step with everything at once
        _attn("train", "train_small_mixed", 2, 4, 2, 257, 257, 64, cap=30.0, bias=True, doc=60, pad=5),
        # a training step of a model with capped scores and shared key heads
        _attn("train", "train_capped", 2, 16, 4, 2048, 2048, 128, cap=50.0, boost=4),
        # pre-training on packed documents with a distance bias
        _attn("train", "train_docs_long", 8, 16, 16, 4096, 4096, 64, bias=True, doc=900),
        # one chat's next token: few rows, latency counts; the cache's first rows belong to another document
        _decode("decode_one_chat", 1, 8, 2, 128, 3000, 5000, page=16, append=True, cap=50.0, start=True),
        # a full batch of long contexts whose rows' weights are added up for a later eviction
        _decode("decode_batch_weights", 64, 32, 8, 128, 1024, 32768, weights=True, cap=50.0),
        # the last queries of a long prompt vote on which of its keys to keep
        _attn("weights", "weights_window", 4, 32, 8, 64, 8192, 128, cap=50.0),
        # every query of a prompt votes
        _attn("weights", "weights_prompt", 1, 32, 8, 4095, 4095, 128),
        # one long prompt cut down to a quarter
        _evict("evict_one_prompt", 1, 8, 128, 4001, 4001, 1024, 128),
        # a batch of long prompts cut down to a fixed budget
        _evict("evict_batch", 16, 8, 128, 8192, 32768, 4096, 512),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["fwd", "train", "decode", "weights", "evict"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    bias = rng.random() < 0.4
    if kind == "evict":
        hi = _spread(rng, 64, 32768)
        keep = _spread(rng, 1, hi)
        return _evict("", _spread(rng, 1, 16), Hkv, D, max(1, hi // 4), hi, keep, rng.randint(0, keep))
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2, 4])
    if kind == "decode":
        append = rng.random() < 0.5
        B = _spread(rng, 1, 64)
        # an appended cache is an output: it stays below a gigabyte
        hi = _spread(rng, 1, 32768 if not append else max(1, min(32768, (1 << 28) // (B * Hkv * D))))
        page = rng.choice([0, 16, 32, 48, 64, 256])
        return _decode("", B, Hq, Hkv, D, max(1, hi // 3), hi, page, append, rng.random() < 0.5, cap, bias,
                       rng.random() < 0.3)
    causal = rng.random() < 0.8
    top = {"fwd": 8192, "train": 4096, "weights": 4096}[kind]
    B = _spread(rng, 1, 8)
    Lq = _spread(rng, 1, top)
    Lk = Lq + (_spread(rng, 1, 8192) if rng.random() < (0.6 if kind == "weights" else 0.25) else 0)
    room = {"fwd": 32 * 8191 * 8191 * 128, "train": 8 * 16 * 4096 * 4096 * 64 // 4,
            "weights": 32 * 4095 * 4095 * 128}[kind]
    while B * Hq * Lq * Lk * D > room:
        if B > 1:
            B = (B + 1) // 2
        else:
            Lq, Lk = (Lq + 1) // 2, (Lk + 1) // 2
    doc = _spread(rng, 5, 2000) if rng.random() < 0.5 else 0
    pad = rng.randint(0, Lq // 8) if doc else 0
    prefix = rng.randint(1, Lk) if causal and rng.random() < 0.3 else 0
    return _attn(kind, "", B, Hq, Hkv, Lq, Lk, D, causal, cap, bias, doc, pad, prefix, rng.choice([1, 4]))


def _layout(case):
    """The generator of what a case fixes for every seed: documents, lengths, pages."""
    return random.Random(",".join(f"{k}={v}" for k, v in sorted(case.items()) if k != "name"))


def _doc_rows(case):
    """Document numbers of the keys, one list per batch row; -1 on unused tokens (the queries are the last Lq)."""
    rng = _layout(case)
    rows = []
    for b in range(case["B"]):
        n = case["Lk"] - (case["pad"] if b == case["B"] - 1 else 0)
        ids, d = [], 0
        while len(ids) < n:
            ids += [d] * min(n - len(ids), max(1, int(rng.expovariate(1.0 / case["doc"]))))
            d += 1
        rows.append(ids + [-1] * (case["Lk"] - n))
    return rows


def _prefixes(case):
    rng = _layout(case)
    return [case["prefix"]] + [rng.randint(0, case["prefix"]) for _ in range(case["B"] - 1)]


def _lengths(case):
    rng = _layout(case)
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _starts(case, lengths):
    rng = _layout(case)
    return [rng.randint(0, n // 2) for n in lengths]


def _pairs(case):
    """Allowed (query, key) pairs of one query head, over the batch."""
    Lq, Lk = case["Lq"], case["Lk"]
    docs = np.array(_doc_rows(case)) if case["doc"] else np.zeros((case["B"], Lk), dtype=np.int64)
    pre = _prefixes(case)
    total = 0
    for b in range(case["B"]):
        d = docs[b]
        for i in range(Lq):
            me = d[i + Lk - Lq]
            if me < 0:
                continue
            lo, hi = np.searchsorted(np.where(d < 0, 1 << 30, d), [me, me + 1])
            if not case["causal"]:
                total += int(hi - lo)
            else:
                upto = max(i + Lk - Lq + 1, pre[b] if case["prefix"] else 0)
                total += max(0, int(min(hi, upto) - lo))
    return total


def work(case):
    kind, D, B = case["kind"], case["D"], case["B"]
    if kind == "evict":
        n = _lengths(case)
        kept = sum(min(x, case["keep"]) for x in n) * case["Hkv"]
        return {"bytes": sum(n) * case["Hkv"] * 4 + kept * (2 * 2 * 2 * D + 4 + 4), "flops": 0}
    if kind == "decode":
        n = _lengths(case)
        s = _starts(case, n) if case["start"] else [0] * B
        rows = sum(x - y for x, y in zip(n, s))
        by = rows * case["Hkv"] * D * 4 + B * case["Hq"] * (4 * D + 4)
        if case["append"]:
            by += B * case["Hkv"] * D * 8
        if case["weights"]:
            by += rows * case["Hkv"] * 8
        return {"bytes": by, "flops": 4 * D * case["Hq"] * (rows + (B if case["append"] else 0))}
    pairs = _pairs(case) * case["Hq"]
    qo = B * case["Lq"] * case["Hq"] * D * 2
    kv = B * case["Lk"] * case["Hkv"] * D * 2
    lse = B * case["Lq"] * case["Hq"] * 4
    if kind == "weights":
        return {"bytes": qo + kv + lse + B * case["Lk"] * case["Hkv"] * 4, "flops": 2 * D * pairs}
    if kind == "fwd":
        return {"bytes": 2 * qo + 2 * kv + lse, "flops": 4 * D * pairs}
    # forward, then five products; q, k, v and dO read, o and the gradients written
    return {"bytes": 4 * qo + 4 * kv + lse, "flops": 14 * D * pairs}


# ----------------------------------------------------------------- inputs --
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32, device=DEV)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, B, Hkv, D = case["kind"], case["B"], case["Hkv"], case["D"]
    s = {"case": case}
    if kind == "evict":
        n = _lengths(case)
        L = max(n)
        s["k"], s["v"] = _normal(gen, B, L, Hkv, D), _normal(gen, B, L, Hkv, D)
        # what softmax leaves: most rows next to nothing, a few much, some exactly alike
        u = torch.rand(B, Hkv, L, generator=gen, device=DEV)
        s["w"] = torch.where(u < 0.05, torch.zeros_like(u), torch.exp(-12.0 * u) * 40.0)
        s["n"] = _ints(n)
        s["k2"] = torch.zeros(B, case["keep"], Hkv, D, dtype=torch.bfloat16, device=DEV)
        s["v2"] = torch.zeros_like(s["k2"])
        s["w2"] = torch.zeros(B, Hkv, case["keep"], device=DEV)
        s["n2"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        return s
    Hq = case["Hq"]
    s["scale"] = 1.0 / math.sqrt(D)
    s["slopes"] = _slopes(Hq) if case["bias"] else None
    if kind == "decode":
        n = _lengths(case)
        s["n"] = _ints(n)
        s["starts"] = _ints(_starts(case, n)) if case["start"] else None
        rows = max(n) + 1
        page = case["page"]
        s["q"] = _normal(gen, B, Hq, D)
        s["table"] = None
        if page:
            per = -(-rows // page)
            pool = B * per + 3
            order = list(range(pool))
            _layout(case).shuffle(order)
            s["table"] = _ints(order[:B * per]).view(B, per)
            s["k"], s["v"] = _normal(gen, pool, page, Hkv, D), _normal(gen, pool, page, Hkv, D)
            rows = per * page
        else:
            s["k"], s["v"] = _normal(gen, B, rows, Hkv, D), _normal(gen, B, rows, Hkv, D)
        s["k1"] = _normal(gen, B, Hkv, D) if case["append"] else None
        s["v1"] = _normal(gen, B, Hkv, D) if case["append"] else None
        s["w"] = torch.rand(B, Hkv, rows, generator=gen, device=DEV) if case["weights"] else None
        return s
    Lq, Lk = case["Lq"], case["Lk"]
    s["q"] = _normal(gen, B, Lq, Hq, D)
    if case["boost"] > 1:
        s["q"][:, :, :Hq // 2] *= case["boost"]
    s["k"] = _normal(gen, B, Lk, Hkv, D)
    s["docs"] = None
    if case["doc"]:
        kd = _ints(_doc_rows(case))
        s["docs"] = (kd[:, Lk - Lq:].contiguous(), kd)
    s["prefix"] = _ints(_prefixes(case)) if case["prefix"] else None
    if kind == "weights":
        # the forward has left the log-sums of the prompt's rows
        s["lse"] = torch.stack([torch.stack([_plain_probs(s, b, h)[1] for h in range(Hq)]) for b in range(B)])
        return s
    s["v"] = _normal(gen, B, Lk, Hkv, D)
    if kind == "train":
        s["do"] = _normal(gen, B, Lq, Hq, D)
    return s


# ------------------------------------------------------------ plain forms --
def _allowed(s, b):
    c = s["case"]
    i = torch.arange(c["Lq"], device=DEV)[:, None] + (c["Lk"] - c["Lq"])
    j = torch.arange(c["Lk"], device=DEV)[None, :]
    ok = (j <= i) if c["causal"] else (j >= 0).expand(c["Lq"], c["Lk"])
    if s["prefix"] is not None:
        ok = ok | (j < s["prefix"][b])
    if s["docs"] is not None:
        qd, kd = s["docs"][0][b][:, None], s["docs"][1][b][None, :]
        ok = ok & (qd == kd) & (qd >= 0)
    return ok


def _plain_probs(s, b, h, ok=None):
    """(P [Lq, Lk], log-sum [Lq], derivative of the cap or None) of one head, in 32 bits."""
    c = s["case"]
    g = c["Hq"] // c["Hkv"]
    x = (s["q"][b, :, h].float() @ s["k"][b, :, h // g].float().T) * s["scale"]
    slope = None
    if c["cap"]:
        t = torch.tanh(x / c["cap"])
        x = c["cap"] * t
        slope = 1.0 - t * t
    if s["slopes"] is not None:
        i = torch.arange(c["Lq"], device=DEV)[:, None] + (c["Lk"] - c["Lq"])
        j = torch.arange(c["Lk"], device=DEV)[None, :]
        x = x - s["slopes"][h] * (i - j).abs()
    ok = _allowed(s, b) if ok is None else ok
    x = torch.where(ok, x, NEG_INF)
    m = x.amax(dim=1, keepdim=True)
    m = torch.where(m == NEG_INF, 0.0, m)
    e = torch.exp(x - m)
    l = e.sum(dim=1, keepdim=True)
    return e / torch.where(l > 0, l, 1.0), (m + torch.log(l))[:, 0], slope


def _plain_fwd(s):
    c = s["case"]
    B, Hq, Lq, D = c["B"], c["Hq"], c["Lq"], c["D"]
    g = Hq // c["Hkv"]
    train = c["kind"] == "train"
    o = torch.empty(B, Lq, Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, Hq, Lq, device=DEV)
    if train:
        dq = torch.empty(B, Lq, Hq, D, dtype=torch.bfloat16, device=DEV)
        dk = torch.zeros(B, c["Lk"], c["Hkv"], D, device=DEV)
        dv = torch.zeros_like(dk)
    for b in range(B):
        ok = _allowed(s, b)
        for h in range(Hq):
            p, lse[b, h], slope = _plain_probs(s, b, h, ok)
            v = s["v"][b, :, h // g].float()
            of = p @ v
            o[b, :, h] = of.to(torch.bfloat16)
            if train:
                do = s["do"][b, :, h].float()
                dv[b, :, h // g] += p.T @ do
                ds = p * (do @ v.T - (do * of).sum(dim=1, keepdim=True))
                if slope is not None:
                    ds = ds * slope
                ds = ds * s["scale"]
                dq[b, :, h] = (ds @ s["k"][b, :, h // g].float()).to(torch.bfloat16)
                dk[b, :, h // g] += ds.T @ s["q"][b, :, h].float()
    if train:
        return o, lse, dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)
    return o, lse


def _cache_rows(s, b, n):
    """The first n cached rows of sequence b: k, v [n, Hkv, D]."""
    if s["table"] is None:
        return s["k"][b, :n], s["v"][b, :n]
    page = s["case"]["page"]
    r = torch.arange(n, device=DEV)
    p = s["table"][b][r // page].long()
    return s["k"][p, r % page], s["v"][p, r % page]


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    g = Hq // Hkv
    if c["append"]:
        at, every = s["n"].long(), torch.arange(B, device=DEV)
        if s["table"] is None:
            s["k"][every, at], s["v"][every, at] = s["k1"], s["v1"]
        else:
            p = s["table"][every, at // c["page"]].long()
            s["k"][p, at % c["page"]], s["v"][p, at % c["page"]] = s["k1"], s["v1"]
    o = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, Hq, device=DEV)
    w = s["w"].clone() if c["weights"] else None
    lengths = _lengths(c)
    starts = _starts(c, lengths) if c["start"] else [0] * B
    for b in range(B):
        n = lengths[b] + int(c["append"])
        k, v = _cache_rows(s, b, n)
        k, v = k[starts[b]:].float(), v[starts[b]:].float()
        x = torch.matmul(s["q"][b].float().view(Hkv, g, D), k.permute(1, 2, 0)) * s["scale"]
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        if s["slopes"] is not None:
            back = torch.arange(n - 1 - starts[b], -1, -1, device=DEV)
            x = x - s["slopes"].view(Hkv, g, 1) * back
        m = x.amax(dim=2, keepdim=True)
        e = torch.exp(x - m)
        l = e.sum(dim=2, keepdim=True)
        p = e / l
        o[b] = torch.matmul(p, v.transpose(0, 1)).view(Hq, D).to(torch.bfloat16)
        lse[b] = (m + torch.log(l)).view(Hq)
        if w is not None:
            if c["append"]:
                w[b, :, n - 1] = 0.0
            w[b, :, starts[b]:n] += p.sum(dim=1)
    return _decode_out(s, o, lse, w)


def _decode_out(s, o, lse, w):
    out = [o, lse]
    if w is not None:
        out.append(w)
    if s["case"]["append"]:
        out += [s["k"], s["v"]]
    return out


def _plain_weights(s):
    c = s["case"]
    w = torch.zeros(c["B"], c["Hkv"], c["Lk"], device=DEV)
    for b in range(c["B"]):
        ok = _allowed(s, b)
        for h in range(c["Hq"]):
            w[b, h // (c["Hq"] // c["Hkv"])] += _plain_probs(s, b, h, ok)[0].sum(dim=0)
    return w


def _plain_evict(s):
    c = s["case"]
    keep, recent = c["keep"], c["recent"]
    kept = torch.full((c["B"], c["Hkv"], keep), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(_lengths(c)):
        m = min(n, keep)
        if n <= keep:
            idx = torch.arange(n, device=DEV).expand(c["Hkv"], n)
        else:
            old = n - recent
            best = torch.sort(s["w"][b, :, :old], dim=1, descending=True, stable=True).indices[:, :keep - recent]
            last = torch.arange(old, n, device=DEV).expand(c["Hkv"], recent)
            idx = torch.cat([best, last], dim=1).sort(dim=1).values
        h = torch.arange(c["Hkv"], device=DEV)[:, None]
        s["k2"][b, :m] = s["k"][b][idx, h].transpose(0, 1)
        s["v2"][b, :m] = s["v"][b][idx, h].transpose(0, 1)
        s["w2"][b, :, :m] = s["w"][b][h, idx]
        kept[b, :, :m] = idx.int()
        s["n2"][b] = m
    return s["k2"], s["v2"], s["w2"], s["n2"], kept


# ---------------------------------------------------------------- the call --
def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"fwd": _plain_fwd, "train": _plain_fwd, "decode": _plain_decode, "weights": _plain_weights,
                "evict": _plain_evict}[kind](s)
    import exact_tiled_attention_46_b200 as fa
    c = s["case"]
    if kind == "evict":
        kept = fa.cache_evict(s["k"], s["v"], s["w"], s["n"], keep=c["keep"], recent=c["recent"],
                              out=(s["k2"], s["v2"], s["w2"], s["n2"]))
        return s["k2"], s["v2"], s["w2"], s["n2"], kept
    how = {"scale": s["scale"], "softcap": c["cap"], "slopes": s["slopes"]}
    if kind == "decode":
        w = s["w"].clone() if c["weights"] else None
        o, lse = fa.decode_scored(s["q"], s["k"], s["v"], s["n"], page_table=s["table"], k_new=s["k1"], v_new=s["v1"],
                                  starts=s["starts"], weights=w, **how)
        return _decode_out(s, o, lse, w)
    how.update(causal=c["causal"], docs=s["docs"], prefix=s["prefix"])
    if kind == "weights":
        return fa.key_weights(s["q"], s["k"], s["lse"], **how)
    o, lse = fa.fwd_scored(s["q"], s["k"], s["v"], **how)
    if kind == "fwd":
        return o, lse
    return (o, lse) + tuple(fa.bwd_scored(s["q"], s["k"], s["v"], o, s["do"], lse, **how))


# ------------------------------------------------------------------ exact --
def _exact_geometry(s, c, b):
    """(hidden pairs, distances) of one batch row, from positions on the host."""
    qpos = np.arange(c["Lk"] - c["Lq"], c["Lk"])
    kpos = np.arange(c["Lk"])
    hidden = np.zeros((c["Lq"], c["Lk"]), dtype=bool)
    if c["causal"]:
        hidden = kpos[None, :] > qpos[:, None]
        if c["prefix"]:
            hidden[:, :_prefixes(c)[b]] = False
    if c["doc"]:
        d = np.array(s["doc_rows"][b])
        hidden = hidden | (d[qpos][:, None] != d[None, :]) | (d[qpos][:, None] < 0)
    dist = np.abs(qpos[:, None] - kpos[None, :]) if c["bias"] else np.zeros((1, 1))
    return torch.from_numpy(hidden).to(DEV), torch.from_numpy(dist).to(DEV, torch.float64)


def _exact_logits(c, h, q, k, hidden, dist):
    """64-bit scores of one head as the definition states them; -inf where the pair is not allowed."""
    z = torch.einsum("id,jd->ij", q, k) * (1.0 / math.sqrt(c["D"]))
    if c["cap"] > 0:
        z = torch.tanh(z / c["cap"]) * c["cap"]
    if c["bias"]:
        z = z - float(np.float32(2.0 ** (-8.0 * (h + 1) / c["Hq"]))) * dist
    return z.masked_fill(hidden, NEG_INF)


def _exact_attn(case, s):
    c = case
    g = c["Hq"] // c["Hkv"]
    train, votes = c["kind"] == "train", c["kind"] == "weights"
    s["doc_rows"] = _doc_rows(c) if c["doc"] else None
    f64 = {"dtype": torch.float64, "device": DEV}
    o, lse = torch.zeros(c["B"], c["Lq"], c["Hq"], c["D"], **f64), torch.zeros(c["B"], c["Hq"], c["Lq"], **f64)
    dq, dk = torch.zeros_like(o), torch.zeros(c["B"], c["Lk"], c["Hkv"], c["D"], **f64)
    dv, w = torch.zeros_like(dk), torch.zeros(c["B"], c["Hkv"], c["Lk"], **f64)
    for b in range(c["B"]):
        hidden, dist = _exact_geometry(s, c, b)
        for h in range(c["Hq"]):
            q = s["q"][b, :, h].double().requires_grad_(train)
            k = s["k"][b, :, h // g].double().requires_grad_(train)
            z = _exact_logits(c, h, q, k, hidden, dist)
            some = torch.isfinite(z.detach()).any(dim=1)
            lse[b, h] = torch.where(some, torch.logsumexp(z.detach(), dim=1), NEG_INF)
            # rows that see nothing give nothing
            p = torch.softmax(torch.where(some[:, None], z, 0.0), dim=1) * some[:, None]
            if votes:
                # against the log-sums that the caller holds
                w[b, h // g] += torch.where(some[:, None], torch.exp(z - s["lse"][b, h].double()[:, None]), 0.0).sum(0)
                continue
            v = s["v"][b, :, h // g].double().requires_grad_(train)
            out = p @ v
            o[b, :, h] = out.detach()
            if train:
                gq, gk, gv = torch.autograd.grad(out, (q, k, v), s["do"][b, :, h].double())
                dq[b, :, h] = gq
                dk[b, :, h // g] += gk
                dv[b, :, h // g] += gv
    if votes:
        return w
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _exact_decode(case, s):
    c = case
    g = c["Hq"] // c["Hkv"]
    n = _lengths(c)
    starts = _starts(c, n) if c["start"] else [0] * c["B"]
    o = torch.zeros(c["B"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["B"], c["Hq"], dtype=torch.float64, device=DEV)
    w = s["w"].double() if c["weights"] else None
    for b in range(c["B"]):
        rows = list(range(starts[b], n[b]))
        if s["table"] is None:
            k, v = s["k"][b, starts[b]:n[b]], s["v"][b, starts[b]:n[b]]
        else:
            table = s["table"][b].tolist()
            flat = torch.tensor([table[r // c["page"]] * c["page"] + r % c["page"] for r in rows], dtype=torch.long,
                                device=DEV)
            k, v = s["k"].flatten(0, 1)[flat], s["v"].flatten(0, 1)[flat]
        if c["append"]:
            k, v = torch.cat([k, s["k1"][b:b + 1]]), torch.cat([v, s["v1"][b:b + 1]])
            rows.append(n[b])
            if w is not None:
                w[b, :, n[b]] = 0.0
        for h in range(c["Hq"]):
            z = (k[:, h // g].double() * s["q"][b, h].double()).sum(dim=1) / math.sqrt(c["D"])
            if c["cap"] > 0:
                z = torch.tanh(z / c["cap"]) * c["cap"]
            if c["bias"]:
                pos = torch.tensor(rows, dtype=torch.float64, device=DEV)
                z = z - float(np.float32(2.0 ** (-8.0 * (h + 1) / c["Hq"]))) * (rows[-1] - pos)
            lse[b, h] = torch.logsumexp(z, dim=0)
            p = torch.softmax(z, dim=0)
            o[b, h] = (p[:, None] * v[:, h // g].double()).sum(dim=0)
            if w is not None:
                w[b, h // g, rows[0]:rows[-1] + 1] += p
    out = [o, lse] + ([w] if w is not None else [])
    if c["append"]:
        k, v = s["k"].clone(), s["v"].clone()
        for b in range(c["B"]):
            page, row = (b, n[b]) if s["table"] is None else (int(s["table"][b, n[b] // c["page"]]), n[b] % c["page"])
            k[page, row], v[page, row] = s["k1"][b], s["v1"][b]
        out += [k, v]
    return out


def _exact_evict(case, s):
    c = case
    w = s["w"].cpu().numpy()
    k, v, w2 = torch.zeros_like(s["k2"]), torch.zeros_like(s["v2"]), torch.zeros_like(s["w2"])
    kept = np.full((c["B"], c["Hkv"], c["keep"]), -1, dtype=np.int32)
    n = _lengths(c)
    for b in range(c["B"]):
        for h in range(c["Hkv"]):
            rows = np.arange(n[b])
            if n[b] > c["keep"]:
                old = n[b] - c["recent"]
                order = np.lexsort((rows[:old], -w[b, h, :old]))
                rows = np.sort(np.concatenate([order[:c["keep"] - c["recent"]], rows[old:]]))
            kept[b, h, :len(rows)] = rows
            at = torch.from_numpy(rows).to(DEV)
            k[b, :len(rows), h], v[b, :len(rows), h] = s["k"][b, at, h], s["v"][b, at, h]
            w2[b, h, :len(rows)] = s["w"][b, h, at]
    return (k, v, w2.double(), _ints([min(x, c["keep"]) for x in n]), torch.from_numpy(kept).to(DEV))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "evict":
        return _exact_evict(case, s)
    if case["kind"] == "decode":
        return _exact_decode(case, s)
    return _exact_attn(case, s)
