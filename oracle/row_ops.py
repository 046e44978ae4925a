"""Plain fp64 CPU oracles of the row-wise operators around attention: rotary
positions with several axes, and dropout from a counter-based generator.
numpy only; shares no code with the GPU path."""

from __future__ import annotations

import numpy as np


def rope(x, positions, inv_freq, axis_of, *, adjacent=False, inverse=False):
    """x [T, H, D] float; positions int [n_axes, T].  Pair i is a complex
    number, multiplied by exp(i angle) with angle = position * frequency."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    out = x.copy()
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, half + i)
        angle = np.asarray(positions, np.float64)[int(axis_of[i])] * float(inv_freq[i])
        if inverse:
            angle = -angle
        z = (x[:, :, ia] + 1j * x[:, :, ib]) * np.exp(1j * angle)[:, None]
        out[:, :, ia], out[:, :, ib] = z.real, z.imag
    return out


def philox4x32(counter, key, rounds=10):
    """Philox 4x32 (Salmon et al., SC 2011) on uint64 arrays holding 32-bit
    words: counter (4 arrays) and key (2 ints) -> 4 arrays."""
    m = np.uint64(0xffffffff)
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)   # < 2^64
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c


def dropout_bits(ids, C, seed, offset):
    """The 16 random bits of every (row, column): [len(ids), C]."""
    ids = np.asarray(ids).astype(np.int64) & 0xffffffff
    groups = (C + 7) // 8
    shape = (len(ids), groups)
    w = philox4x32([np.broadcast_to(np.arange(groups, dtype=np.uint64)[None, :], shape),
                    np.broadcast_to(ids.astype(np.uint64)[:, None], shape),
                    np.full(shape, offset & 0xffffffff, np.uint64), np.full(shape, offset >> 32, np.uint64)],
                   (seed & 0xffffffff, seed >> 32))
    bits = np.empty(shape + (8,), np.int64)
    for k in range(4):
        bits[:, :, 2 * k] = w[k] & np.uint64(0xffff)
        bits[:, :, 2 * k + 1] = w[k] >> np.uint64(16)
    return bits.reshape(len(ids), 8 * groups)[:, :C]


def dropout_add(x, residual, ids, p, seed, offset):
    """(out, keep) of out = residual + keep x / (1 - p), p to 2^-16."""
    x = np.asarray(x, np.float64)
    drop = int(np.rint(65536 * p))
    keep = dropout_bits(ids, x.shape[1], seed, offset) >= drop
    out = np.where(keep, x * (65536.0 / (65536 - drop)), 0.0)
    return (out if residual is None else out + np.asarray(residual, np.float64)), keep
