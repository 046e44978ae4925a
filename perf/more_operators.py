"""The paged key-value cache next to packed (THD) attention, and what is measured of it.

* ``append``: the rows of prompts or of single new tokens into the pages of their sequences, as bf16 or as e4m3 with a
  power-of-two scale for each row (``thd_cache_append``).
* ``decode``: attention of one new token per sequence over its pages, with the tanh cap, distance slopes and documents of
  scored attention, and the weight that each cached token gets added up (``thd_attn_decode``).
* ``evict``: the slots of least accumulated weight leave a cache; what stays moves into a given number of slots, head by
  head (``thd_cache_evict``).

``run`` computes them in plain torch (fp32, rounded once), or, with ``own``, through the library.
"""

import math
import random

import torch

own = False

_DEV = "cuda"
_TOP = 448.0                                         # the largest e4m3 number


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of five conversations: pure latency
        {"name": "append 5 tokens", "op": "append", "seqs": 5, "lo": 1, "hi": 1, "old": 900, "Hkv": 8, "D": 128,
         "page": 64, "heads_first": True, "fp8": False, "fused": True, "mix": 1},
        # a packed batch of prompts, read out of the fused projection's output
        {"name": "append packed prompts", "op": "append", "seqs": 8, "lo": 256, "hi": 4096, "old": 0, "Hkv": 16, "D": 128,
         "page": 16, "heads_first": False, "fp8": False, "fused": True, "mix": 2},
        # long prompts into an 8-bit cache
        {"name": "append 131072 tokens fp8", "op": "append", "seqs": 4, "lo": 32768, "hi": 32768, "old": 0, "Hkv": 8,
         "D": 128, "page": 64, "heads_first": True, "fp8": True, "fused": False, "mix": 3},
        # one short conversation, small heads: pure latency
        {"name": "decode one of 700", "op": "decode", "seqs": 1, "lo": 700, "hi": 700, "Hkv": 2, "group": 4, "D": 64,
         "page": 16, "heads_first": False, "fp8": False, "cap": 0.0, "bias": False, "docs": False, "weights": False,
         "mix": 4},
        # a serving batch of ordinary, ragged lengths
        {"name": "decode batch of 32", "op": "decode", "seqs": 32, "lo": 256, "hi": 4096, "Hkv": 8, "group": 4, "D": 128,
         "page": 64, "heads_first": True, "fp8": False, "cap": 0.0, "bias": False, "docs": False, "weights": False,
         "mix": 5},
        # one long document: few rows, the work lies along the cache
        {"name": "decode one of 131072", "op": "decode", "seqs": 1, "lo": 131072, "hi": 131072, "Hkv": 8, "group": 4,
         "D": 128, "page": 64, "heads_first": True, "fp8": False, "cap": 50.0, "bias": False, "docs": False,
         "weights": False, "mix": 6},
        # a large batch over an 8-bit cache: the rate of the memory
        {"name": "decode batch of 64 fp8", "op": "decode", "seqs": 64, "lo": 500, "hi": 16384, "Hkv": 8, "group": 8,
         "D": 128, "page": 32, "heads_first": False, "fp8": True, "cap": 0.0, "bias": False, "docs": False,
         "weights": False, "mix": 7},
        # every head its own keys, weights added up for the eviction that follows
        {"name": "decode with weights", "op": "decode", "seqs": 16, "lo": 1000, "hi": 4160, "Hkv": 16, "group": 1,
         "D": 128, "page": 64, "heads_first": True, "fp8": False, "cap": 0.0, "bias": False, "docs": False,
         "weights": True, "mix": 8},
        # all heads share their keys, odd pages, everything scored attention has, 8 bits, weights
        {"name": "decode shared keys odd pages", "op": "decode", "seqs": 7, "lo": 0, "hi": 20000, "Hkv": 1, "group": 32,
         "D": 64, "page": 24, "heads_first": False, "fp8": True, "cap": 30.0, "bias": True, "docs": True,
         "weights": True, "mix": 9},
        # the regular trim of a serving batch: a page's worth leaves
        {"name": "evict a page of 32", "op": "evict", "seqs": 32, "lo": 2000, "hi": 2112, "Hkv": 8, "D": 128, "page": 64,
         "heads_first": True, "fp8": False, "budget": 2048, "sinks": 4, "recent": 256, "mix": 10},
        # long prompts cut to what decoding keeps
        {"name": "evict 32768 to 4096", "op": "evict", "seqs": 4, "lo": 32768, "hi": 32768, "Hkv": 8, "D": 128, "page": 64,
         "heads_first": True, "fp8": False, "budget": 4096, "sinks": 4, "recent": 512, "mix": 11},
        # 8 bits, small heads, odd pages, uneven lengths
        {"name": "evict fp8 odd pages", "op": "evict", "seqs": 5, "lo": 300, "hi": 30000, "Hkv": 3, "D": 64, "page": 24,
         "heads_first": False, "fp8": True, "budget": 1111, "sinks": 1, "recent": 100, "mix": 12},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "evict"])
    D, fp8, Hkv = rng.choice([64, 128]), rng.random() < 0.5, rng.choice([1, 2, 3, 4, 8, 16])
    c = {"op": op, "Hkv": Hkv, "D": D, "page": rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]),
         "heads_first": rng.random() < 0.5, "fp8": fp8, "mix": rng.randrange(1 << 20)}
    row = Hkv * D                                    # values of a token's keys
    if op == "append":
        n = _spread(rng, 1, min(65536, (1 << 26) // row))
        seqs = min(n, _spread(rng, 1, 64))
        one = rng.random() < 0.3                     # single new tokens
        hi = 1 if one else max(1, n // seqs)
        return {**c, "seqs": seqs, "lo": hi if one else rng.choice([0, 1, max(1, hi // 2)]), "hi": hi,
                "old": _spread(rng, 1, 4000) if one or rng.random() < 0.3 else 0, "fused": rng.random() < 0.5}
    if op == "decode":
        seqs = _spread(rng, 1, 64)
        hi = _spread(rng, 1, max(2, min(131072, (1 << 28) // row // seqs)))
        weights = rng.random() < 0.3
        return {**c, "group": rng.choice([1, 2, 3, 4, 7, 8, 16, 32]), "seqs": seqs, "hi": hi,
                "lo": rng.choice([0, 1, max(1, hi // 4), hi]) if seqs > 1 else hi,
                "cap": rng.choice([15.0, 30.0, 50.0]) if rng.random() < 0.3 else 0.0, "bias": rng.random() < 0.25,
                "docs": rng.random() < 0.25, "weights": weights}
    seqs = _spread(rng, 1, 48)
    hi = _spread(rng, 16, max(17, min(65536, (1 << 27) // row // seqs)))
    budget = _spread(rng, 4, hi)
    return {**c, "seqs": seqs, "hi": hi, "lo": rng.choice([1, max(1, hi // 2), hi]) if seqs > 1 else hi, "budget": budget,
            "sinks": rng.choice([0, 1, 4]) if budget > 8 else 0, "recent": rng.choice([0, budget // 8, budget // 2])}


# ------------------------------------------------------------------ what a case consists of (host, from the case alone)
def _lengths(case):
    r = random.Random(case["mix"])
    return [case["hi"] if case["lo"] == case["hi"] else r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _starts(case):
    """First visible slot of each sequence: the start of its last document."""
    r = random.Random(case["mix"] + 1)
    return [r.randint(0, n // 2) if case["docs"] else 0 for n in _lengths(case)]


def work(case):
    n, D, Hkv, e = _lengths(case), case["D"], case["Hkv"], 1 if case["fp8"] else 2
    slot = 2 * D * e + (2 if case["fp8"] else 0)     # keys and values of a token and head
    if case["op"] == "append":
        return {"bytes": sum(n) * Hkv * (4 * D + slot + 8), "flops": sum(n) * Hkv * D * (4 if case["fp8"] else 0)}
    if case["op"] == "evict":
        b = case["budget"]
        over = [x for x in n if x > b]
        free = lambda x: max(1, x - case["sinks"] - case["recent"])  # noqa: E731
        # protected and kept slots behind the budget move; weights and positions are read, and written for what stays
        moved = sum(min(case["recent"], x - b) + max(0, x - b - case["recent"]) * max(0, free(b)) / free(x) for x in over)
        return {"bytes": Hkv * (2 * slot * moved + 8 * sum(n) + 8 * sum(min(x, b) for x in n)), "flops": Hkv * sum(n)}
    seen = sum(x - s for x, s in zip(n, _starts(case)))
    Hq = Hkv * case["group"]
    more = (8 if case["weights"] else 0) + (4 if case["bias"] else 0)
    return {"bytes": seen * Hkv * (slot + more) + 4 * case["seqs"] * Hq * (D + 1), "flops": 4.0 * D * Hq * seen}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    n, D, Hkv, page, B = _lengths(case), case["D"], case["Hkv"], case["page"], case["seqs"]
    op = case["op"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=_DEV) * std).to(torch.bfloat16)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=_DEV)

    new = n if op == "append" else [0] * B
    total = [x + (case["old"] if op == "append" else 0) for x in n]
    wide = max(1, max(-(-x // page) for x in total))
    used = sum(-(-x // page) for x in total)
    pages = used + 3                                 # a pool has pages that nobody holds
    order = torch.randperm(pages, generator=g, device=_DEV).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device=_DEV)   # entries behind a sequence's pages: none
    at = torch.arange(wide, device=_DEV)[None, :]
    held = i32([-(-x // page) for x in total])[:, None]
    table[at < held] = order[:used]

    def pool(make):                                  # [pages, page, heads, ...], whichever of the two lies inside
        if case["heads_first"]:
            return make(pages, Hkv, page).transpose(1, 2)
        return make(pages, page, Hkv)

    s = {"case": case, "table": table, "len": i32(total), "seen": i32([x + 17 * (x > 0) for x in total])}
    s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
    if case["fp8"]:
        for name in ("k", "v"):
            s[name + "c"] = pool(lambda a, b, c: (torch.randn(a, b, c, D, generator=g, device=_DEV) * 90.0)
                                 .clamp_(-_TOP, _TOP).to(torch.float8_e4m3fn))
            s[name + "e"] = pool(lambda a, b, c: torch.randint(119, 122, (a, b, c), generator=g, device=_DEV,
                                                               dtype=torch.uint8))
    else:
        s["kc"], s["vc"] = pool(lambda a, b, c: normal(a, b, c, D)), pool(lambda a, b, c: normal(a, b, c, D))
        s["ke"] = s["ve"] = None
    if op == "append":
        T = sum(new)
        if case["fused"]:                            # [T, 3 Hkv D]: queries, keys, values of one projection
            x = normal(T, 3 * Hkv * D, std=2.0)
            s["k"], s["v"] = x[:, Hkv * D:2 * Hkv * D].view(T, Hkv, D), x[:, 2 * Hkv * D:].view(T, Hkv, D)
        else:
            s["k"], s["v"] = normal(T, Hkv, D, std=2.0), normal(T, Hkv, D, std=0.3)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu"] = i32(cu)
        s["weight"] = pool(lambda a, b, c: torch.rand(a, b, c, generator=g, device=_DEV))
        s["pos"] = pool(lambda a, b, c: torch.zeros(a, b, c, dtype=torch.int32, device=_DEV))
        return s
    # positions of the tokens that are left after earlier evictions: in no order, some of the earliest among them
    s["pos"] = None
    if op == "evict" or case["bias"]:
        s["pos"] = pool(lambda a, b, c: torch.randint(0, max(1, max(total) + 17), (a, b, c), generator=g, device=_DEV,
                                                      dtype=torch.int32))
        p, j, held = _where(s)
        s["pos"][p[held], j[held]] = _numbers(s, g)[held]
    if op == "evict":
        # a heavy tail, steps that make ties, and tokens that nobody looked at
        w = lambda a, b, c: torch.exp(1.5 * torch.randn(a, b, c, generator=g, device=_DEV)).mul_(64).round_().div_(64)  # noqa: E731
        s["weight"] = pool(w)
        s["weight_out"] = torch.zeros_like(s["weight"])
        s["pos_out"] = torch.zeros_like(s["pos"])
        return s
    s["scale"] = 1.0 / math.sqrt(D)
    s["q"] = normal(B, Hkv * case["group"], D, std=3.0 if case["cap"] else 1.5)
    s["start"] = i32(_starts(case)) if case["docs"] else None
    s["slopes"] = None
    if case["bias"]:                                 # a geometric row of slopes, one per query head
        h = torch.arange(1, Hkv * case["group"] + 1, device=_DEV, dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * h / (Hkv * case["group"]))
    s["weight"] = s["weight_out"] = None
    if case["weights"]:
        s["weight"] = pool(lambda a, b, c: torch.rand(a, b, c, generator=g, device=_DEV))
        s["weight_out"] = torch.zeros_like(s["weight"])
    return s


def _numbers(s, g):
    """A position for every slot [B, L, Hkv]: its own number plus what has left before it, mixed for each head."""
    c = s["case"]
    L = s["table"].shape[1] * c["page"]
    n = s["len"].long()
    x = torch.rand(c["seqs"], L, c["Hkv"], generator=g, device=_DEV)
    x.masked_fill_(torch.arange(L, device=_DEV)[None, :, None] >= n[:, None, None], 2.0)
    rank = x.argsort(1).argsort(1)
    near = (rank < 8) & (n[:, None, None] > 16)      # all but eight of them have 17 tokens that left in front
    return torch.where(near, rank, rank + 17).to(torch.int32)


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _append_own(s):
    from packed_sequence_context_gb300 import thd_attn as T
    T.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["len"], cu_seqlens=s["cu"], k_exp=s["ke"], v_exp=s["ve"],
                   weight=s["weight"], pos=s["pos"], tokens_seen=s["seen"], dev_status=s["status"])
    return _appended(s)


def _appended(s):
    out = {"k": s["kc"], "v": s["vc"], "weight": s["weight"], "pos": s["pos"]}
    return {**out, "k_exp": s["ke"], "v_exp": s["ve"]} if s["case"]["fp8"] else out


def _decode_own(s):
    from packed_sequence_context_gb300 import thd_attn as T
    c = s["case"]
    o, lse, _ = T.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["len"], k_exp=s["ke"], v_exp=s["ve"],
                              softmax_scale=s["scale"], softcap=c["cap"], dist_slopes=s["slopes"], kv_start=s["start"],
                              pos=s["pos"], tokens_seen=s["seen"] if c["bias"] else None, weight=s["weight"],
                              weight_out=s["weight_out"], dev_status=s["status"])
    return {"o": o, "lse": lse, "weight": s["weight_out"]} if c["weights"] else {"o": o, "lse": lse}


def _evict_own(s):
    from packed_sequence_context_gb300 import thd_attn as T
    c = s["case"]
    left, _ = T.cache_evict(s["kc"], s["vc"], s["table"], s["len"], s["weight"], s["pos"], s["seen"], budget=c["budget"],
                            sinks=c["sinks"], recent=c["recent"], k_exp=s["ke"], v_exp=s["ve"],
                            weight_out=s["weight_out"], pos_out=s["pos_out"], dev_status=s["status"])
    return _evicted(s, left)


def _evicted(s, left):
    out = {"k": s["kc"], "v": s["vc"], "weight": s["weight_out"], "pos": s["pos_out"], "len": left}
    return {**out, "k_exp": s["ke"], "v_exp": s["ve"]} if s["case"]["fp8"] else out


# ------------------------------------------------------------------ plain forms
def _where(s):
    """Page and slot inside it of every slot number [B, L], and which of them are held."""
    page = s["case"]["page"]
    j = torch.arange(s["table"].shape[1] * page, device=_DEV)
    held = j[None, :] < s["len"][:, None]
    return s["table"][:, j // page].clamp(min=0).long(), (j % page)[None, :].expand(held.shape), held


def _bytes(x):
    """What indexing takes: 8-bit numbers as their bytes."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _take(x, *at):
    return _bytes(x)[at].view(x.dtype)


def _put(x, at, v):
    _bytes(x)[at] = _bytes(v)


def _append_plain(s):
    c, page = s["case"], s["case"]["page"]
    T = s["k"].shape[0]
    t = torch.arange(T, device=_DEV)
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    back = s["cu"].long()[b + 1] - t                 # rows to the sequence's end
    slot = s["len"].long()[b] - back
    p, at = s["table"][b, slot // page].long(), slot % page
    for name in ("k", "v"):
        x = s[name].float()
        if c["fp8"]:
            big = x.abs().amax(-1)
            m, e = torch.frexp(big)                  # big = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
            e = torch.where(big == 0, 0, e - 9 + (m > 0.875).int()).clamp(-60, 127)
            x = torch.ldexp(x, -e[..., None])
            s[name + "e"][p, at] = (e + 127).to(torch.uint8)
        _put(s[name + "c"], (p, at), x.to(s[name + "c"].dtype))
    s["weight"][p, at] = 0.0
    s["pos"][p, at] = (s["seen"].long()[b] - back).to(torch.int32)[:, None]
    return _appended(s)


def _rows(s, name):
    """Keys or values of all slots, [B, L, Hkv, D] in fp32."""
    p, at, _ = _where(s)
    x = _take(s[name + "c"], p, at).float()
    if s["case"]["fp8"]:
        x = torch.ldexp(x, s[name + "e"][p, at][..., None].int() - 127)
    return x


def _decode_plain(s):
    c, B, Hkv, G, D = s["case"], s["case"]["seqs"], s["case"]["Hkv"], s["case"]["group"], s["case"]["D"]
    p, at, seen = _where(s)
    if c["docs"]:
        seen = seen & (torch.arange(seen.shape[1], device=_DEV)[None, :] >= s["start"][:, None])
    y = s["q"].float().view(B, Hkv, G, D) @ _rows(s, "k").permute(0, 2, 3, 1) * s["scale"]   # [B, Hkv, G, L]
    if c["cap"]:
        y = torch.tanh(y / c["cap"]) * c["cap"]
    if c["bias"]:
        far = s["seen"][:, None, None] - 1 - s["pos"][p, at]
        y = y - s["slopes"].view(Hkv, G, 1) * far.permute(0, 2, 1)[:, :, None]
    y = y.masked_fill(~seen[:, None, None, :], float("-inf"))
    m = y.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    w = torch.exp(y - m)
    z = w.sum(-1, keepdim=True)
    w = w / torch.where(z == 0, 1.0, z)
    v = _rows(s, "v").masked_fill(~seen[:, :, None, None], 0.0).transpose(1, 2)
    out = {"o": (w @ v).reshape(B, Hkv * G, D).to(torch.bfloat16),
           "lse": (m + z.log()).reshape(B, Hkv * G).T.contiguous()}
    if c["weights"]:
        x = s["weight"][p, at] + w.sum(2).transpose(1, 2)
        s["weight_out"][p[seen], at[seen]] = x[seen]
        out["weight"] = s["weight_out"]
    return out


def _evict_plain(s):
    c, b = s["case"], s["case"]["budget"]
    p, at, held = _where(s)
    L, left = held.shape[1], s["len"].clamp(max=b)
    pos, weight = s["pos"][p, at], s["weight"][p, at]                       # [B, L, Hkv]
    first = torch.where((pos < c["sinks"]) | (pos >= s["seen"][:, None, None] - c["recent"]), float("inf"), weight)
    first = torch.where(held[:, :, None], first, float("-inf"))
    rank = first.sort(dim=1, descending=True, stable=True)[1].argsort(1)
    keep = (rank < left[:, None, None]) & held[:, :, None]
    front = (torch.arange(L, device=_DEV) < b)[None, :, None]
    # the i-th kept slot behind the budget goes into the i-th evicted slot in front of it
    to = (~keep & front & held[:, :, None]).transpose(1, 2)
    of = (keep & ~front).transpose(1, 2)
    bt, ht, jt = to.nonzero(as_tuple=True)
    bo, ho, jo = of.nonzero(as_tuple=True)
    pt, at_t, po, at_o = p[bt, jt], at[bt, jt], p[bo, jo], at[bo, jo]
    stay = (keep & front).nonzero(as_tuple=True)
    ps, at_s = p[stay[0], stay[1]], at[stay[0], stay[1]]
    for src, dst in (("weight", "weight_out"), ("pos", "pos_out")):
        s[dst][ps, at_s, stay[2]] = s[src][ps, at_s, stay[2]]
        s[dst][pt, at_t, ht] = s[src][po, at_o, ho]
    for x in [s["kc"], s["vc"]] + ([s["ke"], s["ve"]] if c["fp8"] else []):
        _put(x, (pt, at_t, ht), _take(x, po, at_o, ho))
    return _evicted(s, left)


_OWN = {"append": _append_own, "decode": _decode_own, "evict": _evict_own}
_PLAIN = {"append": _append_plain, "decode": _decode_plain, "evict": _evict_plain}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    return {"append": _append_exact, "decode": _decode_exact, "evict": _evict_exact}[case["op"]](prepare(case, seed))


def _slots(s, b):
    """(pages, slots in them) of sequence b, in order."""
    n, page = int(s["len"][b]), s["case"]["page"]
    pages = s["table"][b, :-(-n // page)].long()
    return (pages.repeat_interleave(page)[:n], torch.arange(page, device=_DEV).repeat(len(pages))[:n])


def _append_exact(s):
    c = s["case"]
    out = {"weight": s["weight"].double()}
    for name in ("k", "v"):
        out[name] = s[name + "c"].double()
    cu = s["cu"].tolist()
    for b in range(c["seqs"]):
        m = cu[b + 1] - cu[b]
        if not m:
            continue
        p, at = (x[-m:] for x in _slots(s, b))
        out["weight"][p, at] = 0.0
        for name in ("k", "v"):
            x = s[name][cu[b]:cu[b + 1]].double()
            if c["fp8"]:                             # the smallest power of two that brings the row under 448
                # (8-bit mantissas are powers of two or further from them than a logarithm's rounding)
                e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / _TOP) - 1e-6)
                x = (x / torch.exp2(e)).float().to(torch.float8_e4m3fn).double()
            out[name][p, at] = x
    return out


def _decode_exact(s):
    c, D, G, B, Hkv = s["case"], s["case"]["D"], s["case"]["group"], s["case"]["seqs"], s["case"]["Hkv"]
    f64 = {"dtype": torch.float64, "device": _DEV}
    o, lse = torch.zeros(B, Hkv * G, D, **f64), torch.full((Hkv * G, B), -math.inf, **f64)
    weight = s["weight_out"].double() if c["weights"] else None
    starts = _starts(c)
    for b in range(B):
        p, at = (x[starts[b]:] for x in _slots(s, b))
        if not len(p):
            continue
        for g in range(Hkv):
            k, v = _take(s["kc"], p, at, g).double(), _take(s["vc"], p, at, g).double()
            if c["fp8"]:
                k = k * torch.exp2(s["ke"][p, at, g].double() - 127)[:, None]
                v = v * torch.exp2(s["ve"][p, at, g].double() - 127)[:, None]
            heads = slice(g * G, (g + 1) * G)
            x = k @ s["q"][b, heads].double().T * s["scale"]               # [slots, G]
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["bias"]:
                x = x - s["slopes"][heads].double() * (int(s["seen"][b]) - 1 - s["pos"][p, at, g].double())[:, None]
            z = torch.logsumexp(x, 0)
            w = torch.exp(x - z)
            o[b, heads], lse[heads, b] = w.T @ v, z
            if c["weights"]:
                weight[p, at, g] = s["weight"][p, at, g].double() + w.sum(1)
    return {"o": o, "lse": lse, "weight": weight} if c["weights"] else {"o": o, "lse": lse}


def _evict_exact(s):
    """Sequence by sequence and head by head, with a selection by threshold."""
    c, b = s["case"], s["case"]["budget"]
    out = {n: s[x].double() for n, x in (("k", "kc"), ("v", "vc"), ("weight", "weight_out"))}
    for i in range(c["seqs"]):
        p, at = _slots(s, i)
        for g in range(c["Hkv"]):
            w, pos = s["weight"][p, at, g].double(), s["pos"][p, at, g]
            keep = torch.ones(len(p), dtype=torch.bool, device=_DEV)
            if len(p) > b:
                x = torch.where((pos < c["sinks"]) | (pos >= int(s["seen"][i]) - c["recent"]), math.inf, w)
                least = x.topk(b)[0][-1]             # the smallest value that stays; of its equals the first ones
                same = x == least
                keep = (x > least) | (same & (same.cumsum(0) <= b - (x > least).sum()))
            of = torch.arange(len(p), device=_DEV)[keep]
            to = of.clone()
            to[of >= b] = torch.arange(min(b, len(p)), device=_DEV)[~keep[:b]]
            for n, x in (("k", "kc"), ("v", "vc"), ("weight", "weight")):
                out[n][p[to], at[to], g] = _take(s[x], p[of], at[of], g).double()
    return out
