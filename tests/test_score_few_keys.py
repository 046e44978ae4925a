"""CPU test of the keys scored attention's dQ walks for Delta (few_keys): a host
program built with nvcc runs the geometry the planner uses on random masks.
Against the masks' definition: they lie inside the tile's range, and every row
that sees 1 to 128 keys has all of them inside; where every row sees more than
384, there are none."""

import os
import shutil
import subprocess

import numpy as np
import pytest
from test_score_schedule import CSRC, ROOT, TILE, _draw

from oracle import score_oracle

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "common.cuh"
using namespace thd;
struct P { int causal; };

int main() {
  int ncase;
  if (scanf("%d", &ncase) != 1) return 1;
  for (int n = 0; n < ncase; ++n) {
    int prefix, docs, Lq, Lkv;
    P p;
    if (scanf("%d %d %d %d %d", &p.causal, &prefix, &docs, &Lq, &Lkv) != 5) return 1;
    std::vector<int2> rq(Lq + 1);
    for (int i = 0; docs && i < Lq; ++i) if (scanf("%d %d", &rq[i].x, &rq[i].y) != 2) return 1;
    SeqGeom g;
    g.q_off = g.kv_off = 0;
    g.Lq = Lq, g.Lkv = Lkv;
    g.koff = p.causal == 2 ? Lkv - Lq : 0;
    ScoreMods m{};
    m.rows_q = docs ? rq.data() : nullptr;
    m.prefix = prefix >= 0 && p.causal ? &prefix : nullptr;
    for (int t = 0; t < ceil_div(Lq, kTile); ++t) {
      const int2 rows = tile_rows(Lq, t), f = few_keys(p, m, g, 0, rows.x, rows.y);
      printf("%d %d %d %d %d %d\n", n, t, f.x, f.y, query_sees(p, m, g, 0, rows.x).x, query_sees(p, m, g, 0, rows.y).y);
    }
  }
  return 0;
}
"""


def test_few_keys_hold_every_row_of_few(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    (tmp_path / "few.cu").write_text(PROGRAM)
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", CSRC, "-I",
                        os.path.join(ROOT, "include"), str(tmp_path / "few.cu"), "-o", str(tmp_path / "few")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rng = np.random.default_rng(78)
    cases, text = [], []
    for _ in range(300):
        _, causal, prefix, docs, lq, _, lk, _ = _draw(rng)
        if rng.random() < 0.5:   # longer ones, for tiles that see many keys
            lq, lk = 3 * lq, 3 * lk
            docs = None if docs is None else tuple(np.repeat(d, 3) if rng.random() < 0.5 else
                                                   np.sort(rng.integers(0, 9, 3 * len(d))) for d in docs)
        cases.append((causal, prefix, docs, lq, lk))
        text.append(f"{causal} {prefix} {int(docs is not None)} {lq} {lk}")
        if docs is not None:
            lo, hi = np.searchsorted(docs[1], docs[0], "left"), np.searchsorted(docs[1], docs[0], "right")
            text += [f"{a} {z}" for a, z in zip(lo, hi)]
    r = subprocess.run([str(tmp_path / "few")], input="\n".join([str(len(cases)), *text]), capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0
    seen, kinds = {}, [0, 0, 0]
    for n, t, lo, hi, k_lo, k_hi in (map(int, ln.split()) for ln in r.stdout.splitlines()):
        causal, prefix, docs, lq, lk = cases[n]
        if n not in seen:
            seen[n], _ = score_oracle.visible(lq, lk, causal, max(prefix, 0), *(docs or (None, None)))
        see = seen[n][t * TILE:(t + 1) * TILE]
        if lo < hi:
            assert k_lo <= lo and hi <= k_hi
        count = see.sum(1)
        for i in np.flatnonzero((count > 0) & (count <= 128)):
            cols = np.flatnonzero(see[i])
            assert lo <= cols[0] and cols[-1] < hi
        if count.min() > 384:
            assert lo >= hi
        kinds[0 if lo >= hi else 2 if (lo, hi) == (k_lo, k_hi) else 1] += 1
    assert min(kinds) > 20, "no keys, some of them and all of them are drawn"
