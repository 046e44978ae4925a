"""CPU test of scored attention's work decomposition: a host program built
with nvcc runs the __host__ __device__ geometry the kernels and the planner
use (query_sees, key_seen_by, tile_rows, tiles_in) on random ragged metadata
with documents and prefixes.  Against the masks' definition: the two intervals
describe the same visible pairs, every visible pair lies in a visited tile of
both walks, visited tiles lie inside the sequence, and a tile is visited only
inside its item's range."""

import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import score_oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_sequence_context_gb300", "csrc")
TILE = 128

WALKER = r"""
#include <cstdio>
#include <vector>
#include "common.cuh"
using namespace thd;
struct P { int causal; };

int main() {
  int ncase;
  if (scanf("%d", &ncase) != 1) return 1;
  for (int n = 0; n < ncase; ++n) {
    int cp, prefix, docs, Lq, Pq, Lkv, Pkv;
    P p;
    if (scanf("%d %d %d %d %d %d %d %d", &cp, &p.causal, &prefix, &docs, &Lq, &Pq, &Lkv, &Pkv) != 8) return 1;
    std::vector<int2> rq(Lq + 1), rk(Lkv + 1);
    for (int i = 0; docs && i < Lq; ++i) if (scanf("%d %d", &rq[i].x, &rq[i].y) != 2) return 1;
    for (int i = 0; docs && i < Lkv; ++i) if (scanf("%d %d", &rk[i].x, &rk[i].y) != 2) return 1;
    SeqGeom g;
    g.q_off = g.kv_off = 0;
    g.Lq = Lq, g.Lkv = Lkv, g.cbq = Pq, g.cbkv = Pkv;
    g.koff = p.causal == 2 ? Lkv - Lq : 0;
    ScoreMods m{};
    m.rows_q = docs ? rq.data() : nullptr;
    m.rows_kv = docs ? rk.data() : nullptr;
    m.prefix = prefix >= 0 && p.causal ? &prefix : nullptr;
    printf("C %d\n", n);
    for (int i = 0; i < Lq; ++i) { const int2 s = query_sees(p, m, g, 0, i); printf("q %d %d\n", s.x, s.y); }
    for (int j = 0; j < Lkv; ++j) { const int2 s = key_seen_by(p, m, g, 0, j); printf("k %d %d\n", s.x, s.y); }
    for (int t = 0; t < ceil_div(g.cbq, kTile); ++t) {
      const int2 rows = tile_rows(Lq, t);
      if (rows.x > rows.y) continue;
      const int lo = query_sees(p, m, g, 0, rows.x).x, hi = query_sees(p, m, g, 0, rows.y).y;
      printf("F %d %d %d", t, lo, hi);
      const int2 n = tiles_in(lo, hi);
      for (int j = n.x; j < n.y; ++j) printf(" %d", j);
      printf("\n");
    }
    for (int t = 0; t < ceil_div(g.cbkv, kTile); ++t) {
      const int2 rows = tile_rows(Lkv, t);
      int kf, kl;
      bwd_kv_range(g, 0, t, kf, kl);
      if (kf != rows.x || kl != rows.y) return 2;
      if (kf > kl) continue;
      const int lo = key_seen_by(p, m, g, 0, kf).x, hi = key_seen_by(p, m, g, 0, kl).y;
      printf("K %d %d %d", t, lo, hi);
      const int2 n = tiles_in(lo, hi);
      for (int j = n.x; j < n.y; ++j) printf(" %d", j);
      printf("\n");
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    d = tmp_path_factory.mktemp("score_walk")
    (d / "walk.cu").write_text(WALKER)
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", CSRC, "-I",
                        os.path.join(ROOT, "include"), str(d / "walk.cu"), "-o", str(d / "walk")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "walk")


def _docs(rng, n):
    """Non-decreasing numbers with gaps."""
    if rng.random() < 0.3:
        return np.sort(rng.integers(0, 4, n))
    return np.cumsum(rng.random(n) < 3.0 / max(n, 1)) * int(rng.integers(1, 3))


def _draw(rng):
    cp = int(rng.integers(1, 5))
    unit = 2 * cp
    causal = int(rng.integers(0, 3))
    lq = int(rng.integers(1, 700))
    lk = lq if causal == 1 or rng.random() < 0.3 else int(rng.integers(1, 700))
    up = lambda x, m: -(-x // m) * m  # noqa: E731
    pad = unit * int(rng.choice([1, 8, 40]))
    pq, pk = up(lq, pad), up(lk, pad)
    prefix = int(rng.integers(0, lk + 50)) if rng.random() < 0.5 else -1
    docs = (_docs(rng, lq), _docs(rng, lk)) if rng.random() < 0.6 else None
    if docs is not None and lq == lk and rng.random() < 0.5:
        docs = (docs[0], docs[0])
    return cp, causal, prefix, docs, lq, pq, lk, pk


def test_intervals_and_walks_cover_the_masks(walker):
    rng = np.random.default_rng(77)
    cases = [_draw(rng) for _ in range(120)]
    text = [str(len(cases))]
    for cp, causal, prefix, docs, lq, pq, lk, pk in cases:
        text.append(f"{cp} {causal} {prefix} {int(docs is not None)} {lq} {pq} {lk} {pk}")
        if docs is not None:
            dq, dk = docs
            for own, other in ((dq, dk), (dk, dq)):
                lo, hi = np.searchsorted(other, own, "left"), np.searchsorted(other, own, "right")
                text += [f"{a} {z}" for a, z in zip(lo, hi)]
    r = subprocess.run([walker], input="\n".join(text), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0
    blocks = r.stdout.split("C ")[1:]
    assert len(blocks) == len(cases)
    for (cp, causal, prefix, docs, lq, pq, lk, pk), block in zip(cases, blocks):
        lines = [ln.split() for ln in block.splitlines()[1:]]
        see, _ = score_oracle.visible(lq, lk, causal, max(prefix, 0), *(docs or (None, None)))
        q = np.array([[int(a), int(z)] for k, a, z in (ln for ln in lines if ln[0] == "q")])
        k = np.array([[int(a), int(z)] for k, a, z in (ln for ln in lines if ln[0] == "k")])
        j, i = np.arange(lk), np.arange(lq)
        assert np.array_equal((j[None] >= q[:, :1]) & (j[None] < q[:, 1:]), see)
        assert np.array_equal(((i[None] >= k[:, :1]) & (i[None] < k[:, 1:])).T, see)
        assert np.all((0 <= q) & (q <= lk)) and np.all((0 <= k) & (k <= lq))
        done = np.zeros_like(see, dtype=int)
        done_k = np.zeros_like(done)
        for ln in lines:
            if ln[0] not in "FK":
                continue
            t, lo, hi = map(int, ln[1:4])
            own, other = (lq, lk) if ln[0] == "F" else (lk, lq)
            rows = np.arange(t * TILE, min((t + 1) * TILE, own))
            for jt in map(int, ln[4:]):
                a, z = jt * TILE, min((jt + 1) * TILE, other)
                assert 0 <= a < z and z > lo and a < hi
                if ln[0] == "F":
                    done[np.ix_(rows, np.arange(a, z))] += 1
                else:
                    done_k[np.ix_(np.arange(a, z), rows)] += 1
        assert np.all(done[see] == 1) and np.all(done <= 1)
        assert np.all(done_k[see] == 1) and np.all(done_k <= 1)
