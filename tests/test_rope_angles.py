"""The angles of rotary positions, at any 32-bit position and at frequencies on
both sides of 1: the host's part (turns per position as a 64-bit fraction,
rope_turn) on the CPU against 100-digit arithmetic, and sines and cosines on the
GPU against the exactly reduced angle.

GPU tolerance, fp32, on inputs (1, 0) and (0, 1): the angle lies within 1/8 turn
of a quarter and is rounded to 24 bits there, 2^-27 turns at most, and the turns
per position are off by 2^-64 at positions up to 2^31, 2^-33 turns.  Sine and
cosine, of at most pi / 4 either way and so with half a unit of at most 2^-25,
are off by two units in the last place, 2^-23, and the result by one rounding,
2^-25: below 2 pi (2^-27 + 2^-33) + 2^-23 + 2^-25 = 2.0e-7 < 2^-22."""

import os
import shutil
import subprocess
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest
import torch

from packed_sequence_context_gb300 import thd_attn as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _two_pi():
    getcontext().prec = 120

    def arctan_inverse(n):
        s = t = Decimal(1) / n
        k = 1
        while abs(t) > Decimal(10) ** -115:
            t = -t / (n * n)
            k += 2
            s += t / k
        return s
    return Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)))   # Machin


TWO_PI = _two_pi()
FREQUENCIES = [1.0, 0.5, 1e-4, 3e-8, 1.0 / 3, 10.0, 100.7, 1000.0, 1e6 / 7, 2.0 ** 40, 6.283185307179586, 0.15915494309189535,
               1e-300, 0.0]
FREQUENCIES += [-f for f in FREQUENCIES]

PROGRAM = r"""
#include <cinttypes>
#include <cstdio>
#include "rope.cuh"
int main() {
  double f;
  while (scanf("%lf", &f) == 1) printf("%" PRIu64 "\n", thd::rope_turn(f));
  return 0;
}
"""


def test_turns_per_position(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    (tmp_path / "turns.cu").write_text(PROGRAM)
    csrc = os.path.join(ROOT, "packed_sequence_context_gb300", "csrc")
    r = subprocess.run([nvcc, "-std=c++17", "-O3", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                        str(tmp_path / "turns.cu"), "-o", str(tmp_path / "turns")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rng = np.random.default_rng(5)
    fs = FREQUENCIES + [float(x) for x in np.exp(rng.uniform(-20, 27, 200)) * rng.choice([-1, 1], 200)]
    more = [1e308, -1e308, 2.0 ** 52 + 1, 2.0 ** 60 * 1.1]   # no precision is promised, only a number
    r = subprocess.run([str(tmp_path / "turns")], input="\n".join(repr(f) for f in fs + more), capture_output=True,
                       text=True, timeout=60)
    got = [int(x) for x in r.stdout.split()]
    assert len(got) == len(fs) + len(more) and all(0 <= x < 2 ** 64 for x in got)
    for f, x in zip(fs, got):
        off = (Fraction(x, 2 ** 64) - Fraction(f) / TWO_PI) % 1
        assert min(off, 1 - off) <= Fraction(1, 2 ** 64), f


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
def test_sines_at_any_position(thd_lib, inverse):
    rng = np.random.default_rng(6)
    pos = [0, 1, -1, 7, 131071, 10 ** 6, -(10 ** 6), 2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 3]
    pos += [int(x) for x in rng.integers(-2 ** 31, 2 ** 31, 60)]
    fs = [f for f in FREQUENCIES if f != 1e-300]
    rot = 2 * len(fs)
    x = torch.zeros(len(pos), 2, rot, device="cuda")
    x[:, 0, :len(fs)] = 1.0    # (1, 0) -> (cos, sin)
    x[:, 1, len(fs):] = 1.0    # (0, 1) -> (-sin, cos)
    y, _ = T.rope(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), np.array(fs), inverse=inverse)
    y = y.double().cpu().numpy()
    for t, p in enumerate(pos):
        for i, f in enumerate(fs):
            frac = p * Fraction(f) / TWO_PI % 1
            a = 2 * np.pi * float(frac if frac < Fraction(1, 2) else frac - 1) * (-1 if inverse else 1)
            want = [np.cos(a), np.sin(a), -np.sin(a), np.cos(a)]
            have = [y[t, 0, i], y[t, 0, len(fs) + i], y[t, 1, i], y[t, 1, len(fs) + i]]
            assert np.abs(np.subtract(have, want)).max() <= 2.0 ** -22, (p, f)
