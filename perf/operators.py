"""The operators around packed (THD) attention that a training step runs next to it, and what is measured of each.

* ``rope``: rotary positions with several axes (time, height, width) applied to the queries and keys of packed
  rows, forward and backward (``thd_rope``).
* ``score``: attention whose scores are capped by a tanh, get a bias that falls with the distance, and are masked by
  documents inside a sequence or opened by a prefix, forward and forward + backward (``thd_attn_score_fwd`` / ``_bwd``).
* ``dropout``: dropout from a counter-based generator plus the residual, forward and backward, with a mask that is
  computed from (seed, offset, row, column) and never stored (``thd_dropout_add``).

``run`` computes them in plain torch (fp32, rounded once), or, with ``own``, through the library.
"""

import math
import random

import numpy as np
import torch

own = False

_DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few decoded tokens of a vision-language model: pure latency
        {"name": "rope 7 tokens", "op": "rope", "T": 7, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "axes": "16/24/24",
         "weave": False, "adjacent": False, "fused": False, "inverse": False, "dtype": "bf16", "far": 4096},
        # a packed training batch, queries and keys read out of the fused projection's output
        {"name": "rope packed fused qkv", "op": "rope", "T": 14632, "Hq": 16, "Hkv": 16, "D": 128, "rot": 128,
         "axes": "24/20/20", "weave": True, "adjacent": False, "fused": True, "inverse": False, "dtype": "bf16",
         "far": 16384},
        # the gradient of a long video's queries and keys
        {"name": "rope backward 131072 tokens", "op": "rope", "T": 131072, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "axes": "16/24/24", "weave": False, "adjacent": False, "fused": False, "inverse": True, "dtype": "bf16",
         "far": 1000000},
        # an image encoder: two axes, half of the head rotated, adjacent pairs, fp32, an odd number of rows
        {"name": "rope fp32 half the head", "op": "rope", "T": 9001, "Hq": 16, "Hkv": 4, "D": 64, "rot": 32,
         "axes": "8/8", "weave": False, "adjacent": True, "fused": False, "inverse": False, "dtype": "fp32",
         "far": 512},
        # two short sequences, capped scores: pure latency
        {"name": "score tiny capped", "op": "score", "train": False, "seqs": 2, "lo": 64, "hi": 128, "more": 0,
         "pad": 0, "cp": 2, "Hq": 2, "Hkv": 2, "D": 64, "causal": 1, "cap": 50.0, "bias": False, "docs": 0,
         "prefix": 0, "mix": 1},
        # a packed batch of ordinary lengths, capped scores
        {"name": "score packed capped", "op": "score", "train": False, "seqs": 8, "lo": 256, "hi": 4096,
         "more": 0, "pad": 0, "cp": 4, "Hq": 16, "Hkv": 16, "D": 128, "causal": 1, "cap": 50.0, "bias": False,
         "docs": 0, "prefix": 0, "mix": 2},
        # padded sequences, shared key heads, bias by distance, a training step
        {"name": "score train padded bias", "op": "score", "train": True, "seqs": 12, "lo": 128,
         "hi": 1600, "more": 0, "pad": 64, "cp": 4, "Hq": 32, "Hkv": 8, "D": 128, "causal": 1, "cap": 0.0,
         "bias": True, "docs": 0, "prefix": 0, "mix": 3},
        # one long sequence, capped scores, a training step: the tensor cores' case
        {"name": "score train 32768 capped", "op": "score", "train": True, "seqs": 1, "lo": 32768,
         "hi": 32768, "more": 0, "pad": 0, "cp": 4, "Hq": 4, "Hkv": 1, "D": 128, "causal": 1, "cap": 30.0,
         "bias": False, "docs": 0, "prefix": 0, "mix": 4},
        # documents packed into one long sequence that is split over the ranks as a whole, a prefix seen by all of
        # its document, bias by distance and a cap: everything at once, a training step
        {"name": "score train documents", "op": "score", "train": True, "seqs": 1, "lo": 16384, "hi": 16384,
         "more": 0, "pad": 0, "cp": 8, "Hq": 8, "Hkv": 2, "D": 64, "causal": 1, "cap": 50.0, "bias": True,
         "docs": 2000, "prefix": 700, "mix": 5},
        # the residual of a small model's short batch: pure latency
        {"name": "dropout 192 x 128", "op": "dropout", "T": 192, "C": 128, "p": 0.1, "residual": True, "ids": False,
         "dtype": "bf16"},
        # a rank's rows of a packed batch: the mask goes by the rows' global numbers
        {"name": "dropout 41888 x 4096 rank", "op": "dropout", "T": 41888, "C": 4096, "p": 0.1,
         "residual": True, "ids": True, "dtype": "bf16"},
        # the gradient, in fp32, with an odd number of columns (rows that start off every alignment)
        {"name": "dropout backward fp32", "op": "dropout", "T": 9001, "C": 1111, "p": 0.25,
         "residual": False, "ids": False, "dtype": "fp32"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "score", "score", "dropout"])
    if op == "rope":
        D = rng.choice([64, 128])
        rot = rng.choice([D, D, D // 2])
        n = rng.choice([1, 2, 3])
        a = [rot // 2 // n] * n
        a[0] += rot // 2 - sum(a)
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4]) if Hkv < 16 else 16
        return {"op": "rope", "T": _spread(rng, 1, 65536), "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
                "axes": "/".join(str(x) for x in a), "weave": rng.random() < 0.4, "adjacent": rng.random() < 0.3,
                "fused": rng.random() < 0.3, "inverse": rng.random() < 0.4,
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "far": _spread(rng, 64, 1000000)}
    if op == "dropout":
        C = _spread(rng, 5, 8192)
        return {"op": "dropout", "T": _spread(rng, 1, 41888 * 4096 // C if C > 4096 else 41888), "C": C,
                "p": round(rng.uniform(0.01, 0.6), 3), "residual": rng.random() < 0.6, "ids": rng.random() < 0.4,
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    train = rng.random() < 0.6
    cp = rng.choice([1, 2, 4, 8])
    Hkv = rng.choice([1, 2, 4])
    Hq = Hkv * rng.choice([1, 2, 4])
    seqs = _spread(rng, 1, 12)
    most = int(math.sqrt(2.0e9 / Hq))               # rows of the batch: the plain form's square of scores
    hi = max(24, _spread(rng, 24, most // seqs))
    kind = rng.choice(["cap", "bias", "both", "docs", "prefix"])
    causal = rng.choice([1, 1, 1, 0, 2])
    docs = _spread(rng, 8, max(9, hi // 2)) if kind == "docs" or rng.random() < 0.2 else 0
    return {"op": "score", "train": train, "seqs": seqs, "lo": rng.choice([1, max(1, hi // 3), hi]), "hi": hi,
            "more": _spread(rng, 1, max(2, hi // 2)) if causal == 2 else 0, "pad": rng.choice([0, 8, 64]), "cp": cp,
            "Hq": Hq, "Hkv": Hkv, "D": rng.choice([64, 128]), "causal": causal,
            "cap": rng.choice([15.0, 30.0, 50.0]) if kind in ("cap", "both") or rng.random() < 0.2 else 0.0,
            "bias": kind in ("bias", "both"), "docs": docs,
            "prefix": _spread(rng, 1, max(2, hi // 2)) if kind == "prefix" else 0, "mix": rng.randrange(1 << 20)}


# ------------------------------------------------------------------ what a score case consists of (host, from the case alone)
def _up(x, m):
    return -(-x // m) * m


def _layout(case):
    """Valid and padded offsets of queries and keys, the document number of every row and the prefix lengths."""
    r = random.Random(case["mix"])
    unit = 2 * case["cp"]
    cu_q, cu_k, pad_q, pad_k = [0], [0], [0], [0]
    doc_q, doc_k, prefix = [], [], []
    for s in range(case["seqs"]):
        n = case["lo"] if case["lo"] == case["hi"] else r.randint(case["lo"], case["hi"])
        if not case["pad"]:
            n = _up(n, unit)
        k = n + (_up(r.randint(1, case["more"]), 1 if case["pad"] else unit) if case["more"] else 0)
        mult = _up(case["pad"], unit) if case["pad"] else 1
        pn, pk = _up(n, mult), _up(k, mult)
        d = []                                       # the keys' documents; queries sit at the end of their keys
        while case["docs"] and len(d) < k:
            d += [len(d)] * r.randint(max(1, case["docs"] // 3), case["docs"] * 5 // 3)
        d = d[:k] if case["docs"] else [0] * k
        doc_k += d + [0] * (pk - k)
        doc_q += d[k - n:] + [0] * (pn - n)
        prefix.append(min(k, r.randint(1, case["prefix"])) if case["prefix"] else 0)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + k)
        pad_q.append(pad_q[-1] + pn)
        pad_k.append(pad_k[-1] + pk)
    i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return {"cu_q": i32(cu_q), "cu_k": i32(cu_k), "pad_q": i32(pad_q), "pad_k": i32(pad_k), "doc_q": i32(doc_q),
            "doc_k": i32(doc_k), "prefix": i32(prefix)}


def _pairs(case):
    """(query, key) pairs that the masks leave, and the rows of the two buffers."""
    lay, n = _layout(case), 0
    for s in range(case["seqs"]):
        lq = int(lay["cu_q"][s + 1] - lay["cu_q"][s])
        lk = int(lay["cu_k"][s + 1] - lay["cu_k"][s])
        dq = lay["doc_q"][lay["pad_q"][s]:lay["pad_q"][s] + lq]
        dk = lay["doc_k"][lay["pad_k"][s]:lay["pad_k"][s] + lk]
        at = np.arange(lq) + (lk - lq if case["causal"] == 2 else 0)
        hi = np.full(lq, lk)
        if case["causal"]:
            hi = np.maximum(np.minimum(at + 1, lk), lay["prefix"][s])
        lo = np.zeros(lq, np.int64)
        if case["docs"]:
            lo = np.searchsorted(dk, dq, "left")
            hi = np.minimum(hi, np.searchsorted(dk, dq, "right"))
        n += int(np.maximum(hi - lo, 0).sum())
    return n, int(lay["pad_q"][-1]), int(lay["pad_k"][-1])


def work(case):
    if case["op"] == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 2 * e * rows * case["D"] + 4 * len(case["axes"].split("/")) * case["T"],
                "flops": 3 * rows * case["rot"]}
    if case["op"] == "dropout":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * case["C"]
        return {"bytes": n * e * (3 if case["residual"] else 2) + (4 * case["T"] if case["ids"] else 0), "flops": 2 * n}
    pairs, tq, tk = _pairs(case)
    q, k = tq * case["Hq"] * case["D"] * 2, tk * case["Hkv"] * case["D"] * 2
    lse = 4 * tq * case["Hq"]
    fwd = 4.0 * case["D"] * case["Hq"] * pairs
    if not case["train"]:
        return {"bytes": 2 * q + 2 * k + lse, "flops": fwd}
    # backward: q, k, v, o, lse, dO again, and the three gradients
    return {"bytes": 2 * q + 2 * k + lse + 3 * q + 2 * k + lse + q + 2 * k, "flops": 3.5 * fwd}


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Angle per position of each rotated pair, and the axis whose position it takes."""
    half = case["rot"] // 2
    inv = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    parts = [int(x) for x in case["axes"].split("/")]
    if not case["weave"]:                            # one axis after the other
        axis = np.repeat(np.arange(len(parts)), parts)
    else:                                            # taking turns while an axis has pairs left
        left, axis = list(parts), []
        while len(axis) < half:
            for a in range(len(parts)):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    return inv, np.asarray(axis, np.uint8)


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    dt = _DT[case.get("dtype", "bf16")]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=_DEV) * std).to(dt)

    if case["op"] == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        s = {"case": case}
        s["inv_freq"], s["axis"] = _frequencies(case)
        if case["fused"]:                            # [T, (Hq + 2 Hkv) D], as the projection writes it
            qkv = normal(T, (Hq + 2 * Hkv) * D)
            s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
            s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        else:
            s["q"], s["k"] = normal(T, Hq, D), normal(T, Hkv, D)
        n = len(case["axes"].split("/"))
        s["pos"] = torch.randint(0, case["far"], (n, T), generator=g, device=_DEV, dtype=torch.int32)
        return s
    if case["op"] == "dropout":
        T, C = case["T"], case["C"]
        s = {"case": case, "x": normal(T, C), "residual": normal(T, C) if case["residual"] else None}
        s["ids"] = torch.randperm(4 * T, generator=g, device=_DEV)[:T].to(torch.int32) if case["ids"] else None
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=_DEV, dtype=torch.int64)  # seed, offset
        return s
    lay = _layout(case)
    s = {"case": case, "scale": 1.0 / math.sqrt(case["D"])}
    for name, v in lay.items():
        s[name] = torch.from_numpy(v).to(_DEV)
    if not case["docs"]:
        s["doc_q"] = s["doc_k"] = None
    if not case["prefix"]:
        s["prefix"] = None
    tq, tk = int(lay["pad_q"][-1]), int(lay["pad_k"][-1])
    # scores of a trained model spread over several units, more so where they need a cap
    s["q"] = normal(tq, case["Hq"], case["D"], std=3.0 if case["cap"] else 1.5)
    s["k"] = normal(tk, case["Hkv"], case["D"])
    s["v"] = normal(tk, case["Hkv"], case["D"])
    if case["train"]:
        s["do"] = normal(tq, case["Hq"], case["D"])
    s["slopes"] = None
    if case["bias"]:                                 # a geometric row of slopes, one per query head
        h = torch.arange(1, case["Hq"] + 1, device=_DEV, dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * h / case["Hq"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if case["op"] == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    if case["op"] == "dropout":
        return _dropout_own(state) if own else _dropout_plain(state)
    return _score_own(state) if own else _score_plain(state)


def _rope_own(s):
    from packed_sequence_context_gb300 import thd_attn as T
    c = s["case"]
    q, k = T.rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["axis"], adjacent=c["adjacent"], inverse=c["inverse"])
    return {"q": q, "k": k}


def _dropout_own(s):
    from packed_sequence_context_gb300 import thd_attn as T
    return {"out": T.dropout_add(s["x"], s["rng"], s["case"]["p"], residual=s["residual"], row_ids=s["ids"])}


def _score_own(s):
    from packed_sequence_context_gb300 import thd_attn as T
    c = s["case"]
    args = (s["cu_q"], s["cu_k"], s["pad_q"], s["pad_k"])
    mods = {"cp_size": c["cp"], "causal": c["causal"], "softmax_scale": s["scale"], "softcap": c["cap"],
            "dist_slopes": s["slopes"], "doc_q": s["doc_q"], "doc_kv": s["doc_k"], "prefix_len": s["prefix"]}
    o, lse, _ = T.attn_score_fwd(s["q"], s["k"], s["v"], *args, **mods)
    if not c["train"]:
        return {"o": o, "lse": lse}
    dq, dk, dv, _ = T.attn_score_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], *args, **mods)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, rot, adjacent):
    x = x.float()
    r = x[..., :rot]
    if adjacent:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _rope_plain(s):
    c = s["case"]
    inv = torch.as_tensor(s["inv_freq"], device=_DEV)
    axis = torch.as_tensor(s["axis"], device=_DEV).long()
    angle = s["pos"].double()[axis].T * inv          # [T, rot/2], in 64 bits: far positions
    angle = -angle if c["inverse"] else angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return {n: _turn(s[n], cos, sin, c["rot"], c["adjacent"]).to(s[n].dtype) for n in ("q", "k")}


def _round(c, key, mul):
    """One round of the generator on four 32-bit words (held in int64)."""
    m = 0xffffffff
    a, b = c[0] * mul[0], c[2] * mul[1]              # 32 x 32 -> 64 bits (the product wraps to the right bits)
    return [((b >> 32) & m) ^ c[1] ^ key[0], b & m, ((a >> 32) & m) ^ c[3] ^ key[1], a & m]


def _words(rows, C, rng):
    """16 random bits for every (row, column): Philox 4x32 with ten rounds, one call for eight columns of a row;
    counter (column / 8, row, offset), key the seed; column 8 g + 2 w + h takes half h of word w."""
    m = 0xffffffff
    groups = torch.arange((C + 7) // 8, device=rows.device)[None, :]
    c = [groups + 0 * rows[:, None], (rows & m)[:, None] + 0 * groups, (rng[1] & m), ((rng[1] >> 32) & m)]
    key, mul = [rng[0] & m, (rng[0] >> 32) & m], (0xD2511F53, 0xCD9E8D57)
    key2 = lambda i: [(key[0] + i * 0x9E3779B9) & m, (key[1] + i * 0xBB67AE85) & m]  # noqa: E731
    c = _round(_round(_round(_round(_round(c, key2(0), mul), key2(1), mul), key2(2), mul), key2(3), mul), key2(4), mul)
    c = _round(_round(_round(_round(_round(c, key2(5), mul), key2(6), mul), key2(7), mul), key2(8), mul), key2(9), mul)
    w = torch.stack(c, -1)                           # [T, groups, 4]
    w = torch.stack((w & 0xffff, w >> 16), -1)       # [T, groups, 4, 2]
    return w.reshape(rows.shape[0], -1)[:, :C]


def _dropout_plain(s):
    c, x = s["case"], s["x"]
    rows = s["ids"].long() if s["ids"] is not None else torch.arange(c["T"], device=_DEV)
    drop = int(round(c["p"] * 65536))
    y = torch.where(_words(rows, c["C"], s["rng"]) >= drop, x.float() * (65536.0 / (65536 - drop)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(x.dtype)}


def _seen(s):
    """Which key each query sees [Tq, Tk], and the distance between their positions."""
    c = s["case"]

    def where(cu, pad, rows):
        r = torch.arange(rows, device=_DEV)
        b = torch.bucketize(r, pad[1:-1].long(), right=True) if c["seqs"] > 1 else torch.zeros_like(r)
        at = r - pad.long()[b]
        n = (cu[1:] - cu[:-1]).long()
        return b, at, at < n[b], n

    bq, iq, okq, nq = where(s["cu_q"], s["pad_q"], s["q"].shape[0])
    bk, ik, okk, nk = where(s["cu_k"], s["pad_k"], s["k"].shape[0])
    if c["causal"] == 2:
        iq = iq + (nk - nq)[bq]
    seen = (bq[:, None] == bk[None, :]) & okq[:, None] & okk[None, :]
    if c["causal"]:
        ahead = ik[None, :] <= iq[:, None]
        if s["prefix"] is not None:
            ahead = ahead | (ik < s["prefix"].long()[bk])[None, :]
        seen = seen & ahead
    if s["doc_q"] is not None:
        seen = seen & (s["doc_q"][:, None] == s["doc_k"][None, :])
    return seen, (iq[:, None] - ik[None, :]).abs()


def _score_plain(s):
    c = s["case"]
    G, cap, scale = c["Hq"] // c["Hkv"], c["cap"], s["scale"]
    q = s["q"].float().transpose(0, 1)
    k = s["k"].float().transpose(0, 1).repeat_interleave(G, 0)
    v = s["v"].float().transpose(0, 1).repeat_interleave(G, 0)
    seen, far = _seen(s)
    y = (q @ k.transpose(1, 2)).mul_(scale)
    t = None
    if cap:
        t = y.div_(cap).tanh_()
        y = t * cap
    if s["slopes"] is not None:
        y -= s["slopes"][:, None, None] * far
    y.masked_fill_(~seen, float("-inf"))
    m = y.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = y.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log())[..., 0]
    p /= torch.where(l == 0, torch.ones_like(l), l)
    o = p @ v
    out = {"o": o.transpose(0, 1).to(torch.bfloat16).contiguous(), "lse": lse}
    if not c["train"]:
        return out
    do = s["do"].float().transpose(0, 1)
    ds = (do @ v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if cap:
        ds *= t.square_().neg_().add_(1.0)
    grad = lambda x: x.reshape(c["Hkv"], G, -1, c["D"]).sum(1)  # noqa: E731
    for name, x in (("dq", scale * (ds @ k)), ("dk", scale * grad(ds.transpose(1, 2) @ q)),
                    ("dv", grad(p.transpose(1, 2) @ do))):
        out[name] = x.transpose(0, 1).to(torch.bfloat16).contiguous()
    return out


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(s)
    if case["op"] == "dropout":
        return _dropout_exact(s)
    return _score_exact(s)


def _rope_exact(s):
    c, out = s["case"], {}
    half = c["rot"] // 2
    first = [2 * i if c["adjacent"] else i for i in range(half)]
    second = [2 * i + 1 if c["adjacent"] else half + i for i in range(half)]
    pos = s["pos"].double()
    for n in ("q", "k"):
        y = s[n].double().clone()
        for i in range(half):                        # each pair as a complex number turned by its angle
            a = pos[int(s["axis"][i])] * float(s["inv_freq"][i]) * (-1 if c["inverse"] else 1)
            z = torch.complex(s[n][..., first[i]].double(), s[n][..., second[i]].double())
            z = z * torch.polar(torch.ones_like(a), a)[:, None]
            y[..., first[i]], y[..., second[i]] = z.real, z.imag
        out[n] = y
    return out


def _dropout_exact(s):
    """The generator on unsigned 32-bit words in numpy, its multiplications split into 16-bit parts."""
    c = s["case"]
    T, C = c["T"], c["C"]
    seed, offset = (int(v) for v in s["rng"].tolist())
    ids = s["ids"].cpu().numpy().astype(np.uint32) if s["ids"] is not None else np.arange(T, dtype=np.uint32)
    drop = int(round(c["p"] * 65536))
    groups = (C + 7) // 8
    keep = torch.empty((T, C), dtype=torch.bool, device=_DEV)
    step = max(1, (1 << 22) // groups)

    def mul(a, b):                                   # (high, low) words of the product
        al, ah, bl, bh = a & 0xffff, a >> 16, b & 0xffff, b >> 16
        low, mid1, mid2 = al * bl, ah * bl, al * bh
        mid = (low >> 16) + (mid1 & 0xffff) + (mid2 & 0xffff)
        return ah * bh + (mid1 >> 16) + (mid2 >> 16) + (mid >> 16), (low & 0xffff) | (mid << 16)

    u = np.uint32
    for r0 in range(0, T, step):
        rows = ids[r0:r0 + step]
        x0 = np.broadcast_to(np.arange(groups, dtype=u), (len(rows), groups)).copy()
        x1 = np.broadcast_to(rows[:, None], x0.shape).copy()
        x2 = np.full(x0.shape, offset & 0xffffffff, u)
        x3 = np.full(x0.shape, offset >> 32, u)
        k0, k1 = seed & 0xffffffff, seed >> 32
        for _ in range(10):
            h0, l0 = mul(x0, u(0xD2511F53))
            h1, l1 = mul(x2, u(0xCD9E8D57))
            x0, x1, x2, x3 = h1 ^ x1 ^ u(k0), l1, h0 ^ x3 ^ u(k1), l0
            k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
        w = np.stack([x0, x1, x2, x3], -1).astype("<u4").view("<u2").reshape(len(rows), -1)[:, :C]
        keep[r0:r0 + step] = torch.from_numpy(w >= drop).to(_DEV)
    y = torch.where(keep, s["x"].double() * (65536.0 / (65536 - drop)), 0.0)
    return {"out": y if s["residual"] is None else y + s["residual"].double()}


def _score_exact(s):
    """Sequence by sequence and head by head, on each sequence's own rows."""
    c = s["case"]
    tq, tk, D, G = s["q"].shape[0], s["k"].shape[0], c["D"], c["Hq"] // c["Hkv"]
    f64 = {"dtype": torch.float64, "device": _DEV}
    o, lse = torch.zeros((tq, c["Hq"], D), **f64), torch.full((c["Hq"], tq), -math.inf, **f64)
    dq = torch.zeros((tq, c["Hq"], D), **f64)
    dk, dv = torch.zeros((tk, c["Hkv"], D), **f64), torch.zeros((tk, c["Hkv"], D), **f64)
    lay = _layout(c)
    for b in range(c["seqs"]):
        lq, lk = int(lay["cu_q"][b + 1] - lay["cu_q"][b]), int(lay["cu_k"][b + 1] - lay["cu_k"][b])
        rq, rk = int(lay["pad_q"][b]), int(lay["pad_k"][b])
        if not lq or not lk:
            continue
        i = torch.arange(lq, device=_DEV)[:, None] + (lk - lq if c["causal"] == 2 else 0)
        j = torch.arange(lk, device=_DEV)[None, :]
        hide = torch.zeros((lq, lk), dtype=torch.bool, device=_DEV)
        if c["causal"]:
            hide = (j > i) & (j >= int(lay["prefix"][b]))
        if c["docs"]:
            hide = hide | (s["doc_q"][rq:rq + lq, None] != s["doc_k"][None, rk:rk + lk])
        for h in range(c["Hq"]):
            q = s["q"][rq:rq + lq, h].double()
            k, v = s["k"][rk:rk + lk, h // G].double(), s["v"][rk:rk + lk, h // G].double()
            x = q @ k.T * s["scale"]
            t = torch.tanh(x / c["cap"]) if c["cap"] else None
            x = c["cap"] * t if c["cap"] else x
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * (i - j).abs()
            x = x.masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
            y = p @ v
            o[rq:rq + lq, h], lse[h, rq:rq + lq] = y, z
            if c["train"]:
                do = s["do"][rq:rq + lq, h].double()
                dv[rk:rk + lk, h // G] += p.T @ do
                g = p * (do @ v.T - (do * y).sum(-1, keepdim=True))
                g = g * (1 - t * t) * s["scale"] if c["cap"] else g * s["scale"]
                dq[rq:rq + lq, h] = g @ k
                dk[rk:rk + lk, h // G] += g.T @ q
    out = {"o": o, "lse": lse}
    return {**out, "dq": dq, "dk": dk, "dv": dv} if c["train"] else out
