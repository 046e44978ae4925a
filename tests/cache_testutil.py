"""A paged cache for the tests: random pages, host copies for the oracle."""

import numpy as np
import torch

FP8 = torch.float8_e4m3fn


def layout(rng, lens, page, extra=2, wide=0):
    """(table [B, wide] int32 with -1 behind the held pages, number of pages)."""
    held = [-(-int(n) // page) for n in lens]
    total = sum(held) + extra
    order = rng.permutation(total).astype(np.int32)
    w = max(1, wide, max(held))
    table = np.full((len(lens), w), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    return table, total


def slotwise(pages, page, heads, dtype, heads_first, device="cuda", tail=()):
    """An uninitialised array [pages, page, heads, *tail], heads or slots inside."""
    if heads_first:
        return torch.empty((pages, heads, page, *tail), dtype=dtype, device=device).transpose(1, 2)
    return torch.empty((pages, page, heads, *tail), dtype=dtype, device=device)


class Cache:
    """Tensors of a cache filled with random rows; unheld slots hold NaN."""

    def __init__(self, lens, *, page=16, Hkv=2, D=64, fp8=False, heads_first=False, seed=0, extra=2, wide=0, spread=3):
        r = self.rng = np.random.default_rng(seed)
        self.lens, self.page, self.Hkv, self.D, self.fp8 = np.asarray(lens, np.int32), page, Hkv, D, fp8
        self.table_np, self.pages = layout(r, lens, page, extra, wide)
        self.table = torch.from_numpy(self.table_np).cuda()
        self.kv_len = torch.from_numpy(self.lens).cuda()
        mk = lambda dt, tail=(): slotwise(self.pages, page, Hkv, dt, heads_first, tail=tail)  # noqa: E731
        self.k_exp = self.v_exp = None
        self.k, self.v = mk(FP8 if fp8 else torch.bfloat16, (D,)), mk(FP8 if fp8 else torch.bfloat16, (D,))
        for name in ("k", "v"):
            t = getattr(self, name)
            x = r.standard_normal(t.shape, dtype=np.float32) * (80 if fp8 else 1)
            t.copy_(torch.from_numpy(np.clip(x, -448, 448)))
            if fp8:
                e = mk(torch.uint8)
                # the values' scales spread further than the keys': scores stay of one size
                s = spread if name == "v" else 1
                e.copy_(torch.from_numpy(r.integers(121 - s, 122 + s, e.shape).astype(np.uint8)))
                setattr(self, name + "_exp", e)
        held = np.zeros((self.pages, page), bool)
        for b, n in enumerate(self.lens):
            j = np.arange(n)
            held[self.table_np[b][j // page], j % page] = True
        self.held = held
        m = torch.from_numpy(~held).cuda()
        for t in (self.k, self.v):
            if fp8:
                t.view(torch.uint8)[m] = 0x7f
            else:
                t[m] = float("nan")
        if fp8:
            self.k_exp[m] = 255
            self.v_exp[m] = 255
        self.weight = mk(torch.float32)
        self.weight.copy_(torch.from_numpy(r.random(self.weight.shape, dtype=np.float32)))
        self.pos = mk(torch.int32)
        self.pos.copy_(torch.from_numpy(r.integers(0, 1 << 20, self.pos.shape).astype(np.int32)))

    def host(self):
        f = lambda t: t.float().double().cpu().numpy()  # noqa: E731
        i = lambda t: None if t is None else t.cpu().numpy().astype(np.int64)  # noqa: E731
        return {"k": f(self.k), "v": f(self.v), "k_exp": i(self.k_exp), "v_exp": i(self.v_exp)}

    def args(self):
        return self.k, self.v, self.table, self.kv_len

    def exps(self):
        return {"k_exp": self.k_exp, "v_exp": self.v_exp}


def same(a, b):
    """Equal numbers, NaN where NaN."""
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=True)
