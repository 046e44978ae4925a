"""Attention of one new token over a paged cache and the append, in 64 bits and
without loops over heads or rows (torch, on any device): for calls too large for
the loops of the oracle, whose bounds the first takes over."""

import torch


def places(table_row, n, page, first=0):
    """(page, slot in it) of a sequence's slots first .. n - 1."""
    j = torch.arange(first, n, device=table_row.device)
    return table_row.long()[j // page], j % page


def rows(x, exp, p, at):
    """Rows [slots, heads, D] of a cache's keys or values, in 64 bits."""
    if exp is None:
        return x[p, at].double()
    y = x.view(torch.uint8)[p, at].view(x.dtype).double()
    return y * torch.exp2(exp[p, at].double() - 127)[..., None]


def decode(q, k, v, table, kv_len, *, scale, softcap=0.0, slopes=None, start=None, pos=None, seen=None, weight=None,
           k_exp=None, v_exp=None):
    """As the oracle's decode: kv_len, start and seen are lists, the rest tensors."""
    B, Hq, D = q.shape
    page, Hkv, e4m3 = k.shape[1], k.shape[2], k_exp is not None
    G, dev = Hq // Hkv, q.device
    f64 = {"dtype": torch.float64, "device": dev}
    o, tol_o = torch.zeros(B, Hq, D, **f64), torch.full((B, Hq, D), 1e-30, **f64)
    lse, tol_lse = torch.full((Hq, B), float("-inf"), **f64), torch.zeros(Hq, B, **f64)
    w = tol_w = None
    if weight is not None:
        w, tol_w = weight.double().clone(), torch.zeros(weight.shape, **f64)
    half = 2.0 ** -11 if e4m3 else 2.0 ** -16 if G <= 16 else 2.0 ** -8
    for b in range(B):
        n = int(kv_len[b])
        s0 = 0 if start is None else min(max(int(start[b]), 0), n)
        if s0 == n:
            continue
        p, at = places(table[b], n, page, s0)
        kk, vv = (rows(x, e, p, at).permute(1, 0, 2) for x, e in ((k, k_exp), (v, v_exp)))   # [Hkv, n, D]
        qq = q[b].double().view(Hkv, G, D)
        x = scale * (qq @ kk.transpose(1, 2))                                                # [Hkv, G, n]
        size = scale * (qq.abs() @ kk.abs().transpose(1, 2))
        y = softcap * torch.tanh(x / softcap) if softcap else x
        err = 2.0 ** -24 * (D + 12) * size + 2.0 ** -21 * (softcap + y.abs())
        if e4m3:
            err = err + 2.0 ** -39 * scale * qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[:, None]
        if slopes is not None:
            num = pos[p, at].double().T if pos is not None else torch.arange(s0, n, **f64).expand(Hkv, -1)
            far = slopes.double().view(Hkv, G, 1) * ((int(seen[b]) if seen is not None else n) - 1 - num)[:, None]
            y = y - far
            err = err + 2.0 ** -22 * far.abs()
        m = y.amax(-1, keepdim=True)
        e = torch.exp(y - m)
        err = err + 2.0 ** -23 * (m.abs() + (y - m).abs().clamp(max=150))
        z = e.sum(-1, keepdim=True)
        pr = e / z
        rel = err + 2.0 ** -21
        dz = (pr * rel).sum(-1, keepdim=True) + 2.0 ** -18
        o[b], lse[:, b] = (pr @ vv).reshape(Hq, D), (m + z.log()).reshape(Hq)
        tol_lse[:, b] = (dz + 2.0 ** -22 * (m + z.log()).abs() + 2.0 ** -22 * m.abs()).reshape(Hq)
        tol_o[b] += ((pr * (half + rel + dz)) @ vv.abs()).reshape(Hq, D) + 2.0 ** -8 * o[b].abs()
        if e4m3:
            of = torch.exp2(v_exp[p, at].double() - 127).T                                   # [Hkv, n]
            top = (pr * torch.where((vv != 0).any(-1), of, 2.0 ** -112)[:, None]).amax(-1, keepdim=True)
            tol_o[b] += (2.0 ** -32 * top * (vv / of[..., None]).abs().sum(1)[:, None]).reshape(Hq, D)
        if w is not None:
            w[p, at] += pr.sum(1).T
            tol_w[p, at] += (pr * (rel + dz + 2.0 ** -20) + 1e-30).sum(1).T
    if w is not None:
        tol_w += 2.0 ** -23 * w.abs() * (tol_w > 0)
    return {"o": o, "lse": lse, "weight": w, "tol_o": tol_o, "tol_lse": tol_lse, "tol_weight": tol_w}


def append(k, v, cu, table, kv_len, page, *, fp8, seen):
    """For rows k, v [T, Hkv, D] in front of cu[-1]: their pages and slots, stored numbers, exponents (of a row with an
    infinity or NaN: 255) and the tokens' numbers."""
    cu, kv_len, seen = (torch.as_tensor(x, device=k.device).long() for x in (cu, kv_len, seen))
    t = torch.arange(int(cu[-1]), device=k.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    back = cu[b + 1] - t
    slot = kv_len[b] - back
    out = {"p": table.long()[b, slot // page], "at": slot % page, "pos": seen[b] - back}
    for name, x in (("k", k), ("v", v)):
        x = x[:len(t)].double()
        if fp8:
            big = x.abs().amax(-1)
            e = torch.full_like(big, 67)
            while (more := big > 448.0 * torch.exp2(e - 127)).any() and not (e[more] > 300).any():
                e = e + more
            e = torch.where(big == 0, 127.0, torch.where(torch.isfinite(big), e, 255.0))
            x = torch.where((e == 255)[..., None], torch.nan, x * torch.exp2(127 - e)[..., None]).float()
            x = x.to(torch.float8_e4m3fn)
            out[name + "_exp"] = e.to(torch.uint8)
        else:
            x = x.to(torch.bfloat16)
        out[name] = x
    return out
