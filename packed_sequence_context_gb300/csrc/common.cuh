// Internal declarations shared by the translation units of libthdattn.so:
// workspace layout, the per-work-item geometry of the emulated ring, and the
// host-side launchers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/thd_attn.h"

namespace thd {

constexpr int kTile = 128;          // rows of a query tile and of a key/value tile
constexpr int kPlanThreads = 1024;  // threads of the single-CTA planner
constexpr int kCostBins = 4096;     // counting-sort bins for the longest-first order

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ inline int imax(int a, int b) { return a > b ? a : b; }

// ---------------------------------------------------------------- score modifications
// What thd_attn_score_* adds to plain attention.  A kernel instantiation is
// told which of it costs work per score by its kMod: 0 is plain attention;
// with kScored set, each query sees the keys of one interval (causal, prefix
// and document masks together); kModCap and kModDist add the tanh cap and the
// distance bias.
// kModBounded (forward, with a cap of at most kBoundedCap): a row's largest y is
// within that of its largest bias, so 2^(y - largest bias) needs no running
// maximum.
// kModParts (dK/dV): a key tile's walk is shared among bwd_parts work items.
constexpr int kScored = 1, kModCap = 2, kModDist = 4, kModBounded = 8, kModParts = 16;
constexpr float kBoundedCap = 80.f;  // softcap log2(e) at most this: 2^-80 <= P <= 2^80

struct ScoreMods {
  float cap_a;            // softcap * log2(e)
  float cap_c;            // 2 log2(e) softmax_scale / softcap: 2^(cap_c s) = e^(2 scale s / softcap)
  // tanh(scale s / softcap) as s times a polynomial in s^2: three terms while
  // |s| <= cap_near, five while |s| <= cap_far (0: never)
  float cap_n[3], cap_near;
  float cap_f[5], cap_far;
  float cap_sat;          // |s| past which dK/dV takes 1 - tanh^2 apart from tanh
  const float* slopes;    // [Hq], or null
  const int2* rows_q;     // per query row: the keys [x, y) of its document, or null
  const int2* rows_kv;    // per key row: the queries [x, y) of its document, or null
  const int32_t* prefix;  // [B], or null
  const int2* ranges;     // per schedule entry: the keys (queries) [x, y) its queries (keys) may see
};

// ---------------------------------------------------------------- workspace
// Effective metadata written by the planner (after the pad decision):
//   eff[0][*] = cu_q, eff[1][*] = pad_q, eff[2][*] = cu_kv, eff[3][*] = pad_kv
struct WsLayout {
  size_t eff = 0;       // int32 [4][B+1]
  size_t tile_off = 0;  // int32 [B+1]
  size_t counters = 0;  // int32 [64]: [0] number of schedule entries
  size_t items = 0;     // int4 [item_cap]
  // backward only: the query-tile schedule of the dQ pass (its own planner
  // outputs), Delta = rowsum(dO * O) and lse in log2 units
  size_t tile_off_q = 0;  // int32 [B+1]
  size_t counters_q = 0;  // int32 [64]
  size_t items_q = 0;     // int4 [item_cap_q]
  size_t delta = 0;       // fp32 [Hq][T_q]
  size_t lse2 = 0;        // fp32 [Hq][T_q], lse * log2(e)
  // scored attention only: the schedules' ranges and the documents' extents
  size_t ranges = 0;    // int2 [item_cap]
  size_t ranges_q = 0;  // int2 [item_cap_q], backward
  size_t doc_err = 0;   // int32
  size_t rows_q = 0;    // int2 [T_q], with documents
  size_t rows_kv = 0;   // int2 [T_kv], with documents, backward
  size_t part = 0;      // fp32 [2 parts][T_kv][Hkv][D], dK and dV of a key tile's parts (bwd_parts > 1)
  int parts = 1;
  size_t total = 0;
  int item_cap = 0;
  int item_cap_q = 0;
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Scored dK/dV: how many work items share a key tile's walk over its queries
// (each takes every bwd_parts-th step and leaves fp32 dK, dV that a last kernel
// adds up).  An SM works on one item, and a causal sequence's first key tile
// sees twice the mean number of queries: unshared, the pass takes the longest
// walk or, if that is more, the mean walk times items / SMs.  Sharing divides
// the first and costs the join (8 us) and the parts' way to memory and back; of
// 1, 2, .. 16 the rule takes what that makes least, at 2 us a step (a query tile
// of one head), as long as every part keeps 12 steps.  Backward measured, cap
// 50, heads of 128, one item a tile against the rule's, us: 32,768 tokens of
// 4 + 1 heads 4161 / 3308, 8192 of 16 + 4 1120 / 922, 4096 of 8 + 2 359 / 209,
// 4096 of 32 + 1 2278 / 647; 4096 of 8 + 8 it leaves alone, 207 (two parts 239).
constexpr double kBwdSms = 152;
inline int bwd_parts(int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D) {
  const double items = (double)(T_kv / kTile + 1) * Hkv;
  const double steps = (double)(T_q / (B > 0 ? B : 1) / kTile + 1) * (Hq / Hkv);
  const double shared = items * steps / (2 * kBwdSms);  // all SMs at work
  int best = 1;
  double least = 2 * (steps > shared ? steps : shared);
  for (int parts = 2; parts <= 16 && steps / parts >= 12; parts *= 2) {
    const double walk = steps / parts > shared ? steps / parts : shared;
    const double t = 2 * walk + 8 + items * parts * kTile * D * 16 / 5e6;
    if (t < least) best = parts, least = t;
  }
  return best;
}

inline WsLayout ws_layout(int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int cp, bool bwd,
                          bool scored = false, bool docs = false, int most_parts = 16) {
  WsLayout w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  w.eff = take(sizeof(int32_t) * 4 * (size_t)(B + 1));
  w.tile_off = take(sizeof(int32_t) * (size_t)(B + 1));
  w.counters = take(sizeof(int32_t) * 64);
  // query schedule: rank-local query tiles; key schedule: chunk-aligned key
  // tiles.  Both are bounded by rows/128 + (one partial tile per chunk).
  const int64_t cap_q = T_q / kTile + (int64_t)cp * B + 1;
  const int64_t cap_kv = T_kv / kTile + (int64_t)2 * cp * B + 1;
  w.item_cap = (int)(bwd ? cap_kv : cap_q);
  w.items = take(sizeof(int32_t) * 4 * (size_t)w.item_cap);
  if (bwd) {
    w.item_cap_q = (int)cap_q;
    w.tile_off_q = take(sizeof(int32_t) * (size_t)(B + 1));
    w.counters_q = take(sizeof(int32_t) * 64);
    w.items_q = take(sizeof(int32_t) * 4 * (size_t)cap_q);
    w.delta = take(sizeof(float) * (size_t)Hq * (size_t)T_q);
    w.lse2 = take(sizeof(float) * (size_t)Hq * (size_t)T_q);
  }
  if (scored) {
    w.ranges = take(sizeof(int32_t) * 2 * (size_t)w.item_cap);
    if (bwd) {
      w.ranges_q = take(sizeof(int32_t) * 2 * (size_t)w.item_cap_q);
      w.parts = bwd_parts(B, T_q, T_kv, Hq, Hkv, D);
      if (w.parts > most_parts) w.parts = most_parts;
      if (w.parts > 1) w.part = take(sizeof(float) * 2 * (size_t)w.parts * (size_t)T_kv * Hkv * D);
    }
  }
  if (docs) {
    w.doc_err = take(sizeof(int32_t));
    w.rows_q = take(sizeof(int32_t) * 2 * (size_t)T_q);
    if (bwd) w.rows_kv = take(sizeof(int32_t) * 2 * (size_t)T_kv);
  }
  w.total = off;
  return w;
}

// ---------------------------------------------------------------- geometry
// One sequence's view after the pad decision.
struct SeqGeom {
  int q_off, kv_off;  // buffer row of position 0
  int Lq, Lkv;        // valid lengths
  int cbq, cbkv;      // chunk lengths (padded / (2 cp))
  int koff;           // causal masks: query i sees key j iff j <= i + koff
};

// Causal modes (the `causal` argument of the entry points).
constexpr int kCausalNone = THD_CAUSAL_NONE;
constexpr int kCausalTopLeft = THD_CAUSAL_TOP_LEFT;          // j <= i; equal query and key lengths
constexpr int kCausalBottomRight = THD_CAUSAL_BOTTOM_RIGHT;  // j <= i + Lkv - Lq: last query sees last key

// `whole` (scored attention): the sequence is one chunk of one rank.
__device__ inline SeqGeom seq_geom(const int32_t* eff, int B, int b, int cp, int causal, bool whole) {
  const int32_t* cu_q = eff;
  const int32_t* pad_q = eff + (B + 1);
  const int32_t* cu_kv = eff + 2 * (B + 1);
  const int32_t* pad_kv = eff + 3 * (B + 1);
  SeqGeom g;
  g.q_off = pad_q[b];
  g.kv_off = pad_kv[b];
  g.Lq = cu_q[b + 1] - cu_q[b];
  g.Lkv = cu_kv[b + 1] - cu_kv[b];
  g.cbq = pad_q[b + 1] - pad_q[b];
  g.cbkv = pad_kv[b + 1] - pad_kv[b];
  if (!whole) {
    g.cbq /= 2 * cp;
    g.cbkv /= 2 * cp;
  }
  g.koff = causal == kCausalBottomRight ? g.Lkv - g.Lq : 0;
  return g;
}

// Position (within the sequence) of rank r's rank-local query row p:
// rows [0, cb) are chunk r, rows [cb, 2cb) chunk 2cp-1-r.
__host__ __device__ inline int local_to_pos(int p, int r, int cb, int cp) {
  return p < cb ? r * cb + p : (2 * cp - 1 - r) * cb + (p - cb);
}

// Largest valid query position among rank-local rows [128 t, 128 t + 128)
// of rank r, or -1 when the tile holds no valid query.
__host__ __device__ inline int fwd_tile_qmax(const SeqGeom& g, int r, int t, int cp) {
  const int p0 = t * kTile, p1 = imin(p0 + kTile, 2 * g.cbq);
  int qmax = -1;
  // first half (chunk r)
  int a0 = p0, a1 = imin(p1, g.cbq);
  if (a0 < a1) {
    int last = imin(local_to_pos(a1 - 1, r, g.cbq, cp), g.Lq - 1);
    if (local_to_pos(a0, r, g.cbq, cp) <= last) qmax = imax(qmax, last);
  }
  // second half (chunk 2cp-1-r)
  a0 = imax(p0, g.cbq);
  a1 = p1;
  if (a0 < a1) {
    int last = imin(local_to_pos(a1 - 1, r, g.cbq, cp), g.Lq - 1);
    if (local_to_pos(a0, r, g.cbq, cp) <= last) qmax = imax(qmax, last);
  }
  return qmax;
}

// Number of 128-row key tiles of chunk c that a query tile with largest
// valid position qmax visits (tiles whose first key is past every query, or
// past the valid length, are skipped).
__host__ __device__ inline int fwd_chunk_tiles(const SeqGeom& g, int c, int qmax, bool causal) {
  if (qmax < 0) return 0;
  const int limit = causal ? imin(g.Lkv, qmax + g.koff + 1) : g.Lkv;
  const int start = c * g.cbkv;
  if (start >= limit) return 0;
  return imin(ceil_div(g.cbkv, kTile), ceil_div(limit - start, kTile));
}

// Ring step i of rank r holds the KV of rank s = (r - i) mod cp; its chunks
// are s and 2cp-1-s (in that order).
__host__ __device__ inline int ring_src(int r, int i, int cp) { return ((r - i) % cp + cp) % cp; }
__host__ __device__ inline int ring_chunk(int s, int e, int cp) { return e == 0 ? s : 2 * cp - 1 - s; }

// Key tiles one forward work item visits over ring steps [step_lo, step_hi).
__host__ __device__ inline int fwd_item_tiles(const SeqGeom& g, int r, int t, int cp, bool causal, int step_lo,
                                              int step_hi) {
  const int qmax = fwd_tile_qmax(g, r, t, cp);
  int n = 0;
  for (int i = step_lo; i < step_hi; ++i) {
    const int s = ring_src(r, i, cp);
    for (int e = 0; e < 2; ++e) n += fwd_chunk_tiles(g, ring_chunk(s, e, cp), qmax, causal);
  }
  return n;
}

// ---- scored attention: the keys one query sees, and the queries that see one
// key, are intervals of positions inside the sequence:
//   query i: keys [lo, hi), hi = Lkv, under a causal mask min(Lkv, i + koff + 1)
//     or the prefix length if that is more; then cut to the keys [x, y) of its
//     document;
//   key j: queries [lo, hi), lo = 0, under a causal mask j - koff unless j is
//     in the prefix, hi = Lq; then cut to the queries of its document.
// Document numbers do not decrease inside a sequence, so lo and hi do not
// decrease with the position either (empty intervals included: hi >= lo), and
// a tile's interval runs from the lo of its first row to the hi of its last.
//
// A sequence is walked as a whole, in order: its query and key tiles are rows
// [128 t, 128 t + 128) of it, not of a rank's chunks.  Outputs do not depend on
// that beyond rounding (every rank's rows lie in the one buffer, and scored
// attention has no single ring step to expose), while chunks of a few dozen
// rows leave most of a tile empty.  By four ranks' chunks and as a whole, us, when
// that changed: a packed batch of 8 sequences of 488 to 3792, 16 heads of 128, cap
// 50, 384 and 238; 12 padded sequences of 154 to 1409 with a bias, forward and
// backward, 1310 and 750; one sequence of 28 113 and 36.
template <class P>
__host__ __device__ inline int2 query_sees(const P& p, const ScoreMods& mods, const SeqGeom& g, int b, int pos) {
  int lo = 0, hi = g.Lkv;
  if (p.causal) {
    hi = imin(hi, imax(pos + g.koff + 1, 0));
    if (mods.prefix) hi = imax(hi, imin(mods.prefix[b], g.Lkv));
  }
  if (mods.rows_q) {
    const int2 d = mods.rows_q[(int64_t)g.q_off + pos];
    lo = d.x;
    hi = imax(imin(hi, d.y), lo);
  }
  return make_int2(lo, hi);
}
template <class P>
__host__ __device__ inline int2 key_seen_by(const P& p, const ScoreMods& mods, const SeqGeom& g, int b, int pos) {
  int lo = 0, hi = g.Lq;
  if (p.causal && !(mods.prefix && pos < mods.prefix[b])) lo = imin(imax(pos - g.koff, 0), g.Lq);
  if (mods.rows_kv) {
    const int2 d = mods.rows_kv[(int64_t)g.kv_off + pos];
    lo = imax(lo, d.x);
    hi = imin(hi, d.y);
  }
  return make_int2(lo, imax(lo, hi));
}

// The keys [x, y) of the rows first .. last of a query tile that see few keys: a
// row that sees 1 to 128 has its interval inside, rows that see more may.  The
// first row's document counts unless that row sees more than kFewKeys, the last
// row's unless that one does (inside a document a row sees at least as many keys
// as the one before, at most one more under a causal mask), those between always.
constexpr int kFewKeys = 256;
template <class P>
__host__ __device__ inline int2 few_keys(const P& p, const ScoreMods& mods, const SeqGeom& g, int b, int first,
                                         int last) {
  const int2 a = query_sees(p, mods, g, b, first), z = query_sees(p, mods, g, b, last);
  const int a_end = mods.rows_q ? mods.rows_q[(int64_t)g.q_off + first].y : g.Lkv;
  return make_int2(a.y - a.x <= kFewKeys ? a.x : a_end, z.y - z.x <= kFewKeys ? z.y : z.x);
}

// First and last valid position of tile t of a sequence of L (first > last: none).
__host__ __device__ inline int2 tile_rows(int L, int t) { return make_int2(t * kTile, imin((t + 1) * kTile, L) - 1); }

// Tiles [x, y) that hold a position of [lo, hi).
__host__ __device__ inline int2 tiles_in(int lo, int hi) {
  return lo < hi ? make_int2(lo / kTile, ceil_div(hi, kTile)) : make_int2(0, 0);
}

// Query rows of one rank.
template <int kMod>
__host__ __device__ inline int rank_rows(const SeqGeom& g) {
  return kMod != 0 ? g.cbq : 2 * g.cbq;
}

// ---- one query tile's walk (forward and the dQ pass).  P is any params
// struct with items, eff, B, Hq, Hkv, cp, causal, step_lo, step_hi.
struct QItem {
  SeqGeom g;
  int b, r, t, h, kvh, qmax;
  int k_lo, k_hi;      // scored: the keys the tile's queries may see
  int few_lo, few_hi;  // scored: the keys of a walk for Delta (see few_keys)
};

// Work item w -> (schedule entry, query head).  Items are ordered by groups
// of p.group_kv kv heads (outermost: while a group runs, its keys and values
// are what the CTAs read, so they stay in L2), then by schedule entry
// (longest first), then by the group's query heads (innermost: query heads
// that share a kv head run side by side).  Ungrouped (one group, group_kv ==
// Hkv) it is entry-major with every head innermost.  n_entries = schedule
// length.
// kGrouped is a compile-time choice: a runtime branch between the two maps
// here measured 8% slower in the forward kernel.
template <bool kGrouped, int kMod, class P>
__device__ inline QItem q_item(const P& p, int n_entries, int w) {
  QItem it;
  int x;  // schedule entry
  if constexpr (kGrouped) {
    const int hg = p.group_kv * (p.Hq / p.Hkv);  // query heads per group
    const int per = n_entries * hg;               // items per group
    const int grp = w / per, rem = w - grp * per;
    x = rem / hg;
    it.h = grp * hg + rem % hg;
  } else {  // one group: entry-major, heads innermost
    (void)n_entries;
    x = w / p.Hq;
    it.h = w % p.Hq;
  }
  const int4 e = p.items[x];
  it.b = e.x;
  it.r = kMod != 0 ? 0 : e.y;
  it.t = e.z;
  it.kvh = it.h / (p.Hq / p.Hkv);
  it.g = seq_geom(p.eff, p.B, it.b, p.cp, p.causal, kMod != 0);
  if constexpr (kMod != 0) {
    const int2 k = p.mods.ranges[x];
    it.k_lo = k.x;
    it.k_hi = k.y;
    it.few_lo = e.y;
    it.few_hi = e.w;
  } else {
    it.qmax = fwd_tile_qmax(it.g, it.r, it.t, p.cp);
  }
  return it;
}

// Calls f(c, j) for every key tile the item visits, in ring order: step i
// holds the KV of rank s = (r - i) mod cp, chunks s then 2cp-1-s.  Scored: the
// sequence's tiles as chunk 0 (those that hold one of `keys`), the last first:
// under a causal mask and a bias the nearest keys hold the maximum, which then
// hardly moves (32,768 tokens, bias alone 4.6 -> 4.1 ms).
template <int kMod, class P, typename F>
__device__ inline void for_each_kv_tile(const QItem& it, const P& p, int2 keys, F&& f) {
  if constexpr (kMod != 0) {
    const int2 n = tiles_in(keys.x, keys.y);
    for (int j = n.y; j-- > n.x;) f(0, j);
    return;
  }
  for (int i = p.step_lo; i < p.step_hi; ++i) {
    const int s = ring_src(it.r, i, p.cp);
    for (int e = 0; e < 2; ++e) {
      const int c = ring_chunk(s, e, p.cp);
      const int n = fwd_chunk_tiles(it.g, c, it.qmax, p.causal != 0);
      for (int j = 0; j < n; ++j) f(c, j);
    }
  }
}

template <int kMod, class P, typename F>
__device__ inline void for_each_kv_tile(const QItem& it, const P& p, F&& f) {
  for_each_kv_tile<kMod>(it, p, kMod != 0 ? make_int2(it.k_lo, it.k_hi) : make_int2(0, 0), f);
}

// Columns (keys) of tile (c, j) any query of the item may see, rounded up to
// the MMA granularity of 16: the N of the item's S product and the K of the
// product that contracts over keys.
template <int kMod, class P>
__device__ inline int q_tile_ncols(const QItem& it, const P& p, int c, int j) {
  const int j0 = c * it.g.cbkv + j * kTile;
  int n;
  if constexpr (kMod != 0) {
    n = imin(kTile, it.k_hi - j0);
  } else {
    n = imin(kTile, imin((c + 1) * it.g.cbkv - j0, it.g.Lkv - j0));
    if (p.causal) n = imin(n, it.qmax + it.g.koff - j0 + 1);
  }
  return 16 * ceil_div(imax(n, 1), 16);
}

// ---- backward: key tile (chunk c, tile jk) of sequence b, and the query
// tiles (chunk qc, tile jq) that attend to it, walked in ring order: the KV of
// owner s is held by rank r = (s + i) mod cp at step i; rank r's query chunks
// are r and 2cp-1-r.
__host__ __device__ inline int chunk_owner(int c, int cp) { return c < cp ? c : 2 * cp - 1 - c; }

// [first, last] valid key positions of key tile (c, jk), or first > last.
__host__ __device__ inline void bwd_kv_range(const SeqGeom& g, int c, int jk, int& first, int& last) {
  first = c * g.cbkv + jk * kTile;
  last = imin(c * g.cbkv + imin((jk + 1) * kTile, g.cbkv), g.Lkv) - 1;
}
// Does query tile (qc, jq) hold a query that sees key position kv_first?
__host__ __device__ inline bool bwd_q_tile_visits(const SeqGeom& g, int qc, int jq, int kv_first, int kv_last,
                                                  bool causal) {
  if (kv_first > kv_last) return false;
  const int q0 = qc * g.cbq + jq * kTile;
  const int qlast = imin(qc * g.cbq + imin((jq + 1) * kTile, g.cbq), g.Lq) - 1;
  if (q0 > qlast) return false;
  return causal ? (qlast + g.koff >= kv_first) : true;
}
__host__ __device__ inline int bwd_item_qtiles(const SeqGeom& g, int c, int jk, int cp, bool causal) {
  int kf, kl;
  bwd_kv_range(g, c, jk, kf, kl);
  if (kf > kl) return 0;
  const int s = chunk_owner(c, cp);
  const int nq = ceil_div(g.cbq, kTile);
  int n = 0;
  for (int i = 0; i < cp; ++i) {
    const int r = (s + i) % cp;
    for (int e = 0; e < 2; ++e) {
      const int qc = e == 0 ? r : 2 * cp - 1 - r;
      for (int jq = 0; jq < nq; ++jq) n += bwd_q_tile_visits(g, qc, jq, kf, kl, causal) ? 1 : 0;
    }
  }
  return n;
}

// ---------------------------------------------------------------- planner
struct PlanParams {
  const int32_t* cu_q;
  const int32_t* cu_kv;
  const int32_t* pad_q;   // may be null
  const int32_t* pad_kv;  // may be null
  int B, cp, causal, pad_mode;
  int64_t rows_q, rows_kv;  // buffer rows
  int mode;                 // 0: partition only, 1: query-tile schedule, 2: key-tile schedule,
                            // 3: both (key tiles into items, query tiles into items_q)
  int step_lo, step_hi;     // ring steps the forward items cover (for the cost)
  int32_t* eff;             // [4][B+1]
  int32_t* cu_rank;         // optional partition outputs (q side)
  int32_t* cu_rank_padded;
  int32_t* cu_rank_half;
  int32_t* token_map;
  int64_t token_map_cap;
  int32_t* tile_off;  // [B+1]
  int32_t* counters;  // [64]
  int4* items;
  int item_cap;
  int32_t* tile_off_q;  // mode 3: the query-tile schedule's outputs
  int32_t* counters_q;
  int4* items_q;
  int item_cap_q;
  // scored attention: the schedules take each entry's range from the masks
  int2* ranges;
  int2* ranges_q;
  ScoreMods mods;
  int32_t* doc_err;  // set by the document kernel; cleared by a mode 0 run
  int32_t* dev_status;
};

// ---------------------------------------------------------------- kernels
struct FwdParams {
  const uint16_t* q;
  void* o;        // bf16 [T_q][Hq][D] (fused) or fp32 (one ring step)
  float* lse;     // [Hq][T_q]
  const int32_t* eff;
  const int4* items;
  const int32_t* counters;
  int32_t* claim;  // dynamic hand-out counter (zeroed by the planner)
  int32_t* dev_status;
  int B, Hq, Hkv, cp, causal;
  int group_kv;  // kv heads per locality group (divides Hkv)
  int64_t T_q;
  float scale_log2;  // softmax_scale * log2(e)
  int step_lo, step_hi;
  int test_stall;  // test hook: every thread waits for a barrier nothing completes
  ScoreMods mods;  // scored attention
};

struct BwdParams {
  const uint16_t* q;
  const uint16_t* dout;
  const float* lse2;   // [Hq][T_q], lse * log2(e)
  const float* delta;  // [Hq][T_q]: Delta = rowsum(dO * O)
  uint16_t* dk;
  uint16_t* dv;
  const int32_t* eff;
  const int4* items;
  const int32_t* counters;
  int32_t* claim;  // dynamic hand-out counter (zeroed by the planner)
  int32_t* dev_status;
  int B, Hq, Hkv, cp, causal;
  int group_kv;  // kv heads per locality group (divides Hkv)
  int64_t T_q, dkv_rows;
  float scale, scale_log2;
  int test_stall;  // test hook: every thread waits for a barrier nothing completes
  ScoreMods mods;  // scored attention
  float* part;     // scored, parts > 1: fp32 [2 parts][T_kv][Hkv][D], dK's parts, then dV's
  int parts;       // scored: work items that share a key tile's walk
  int64_t T_kv;
};

struct DqParams {
  const uint16_t* q;
  const uint16_t* dout;
  const float* lse2;   // [Hq][T_q], lse * log2(e)
  const float* delta;  // [Hq][T_q]: Delta = rowsum(dO * O)
  float* delta_out;    // scored: the same buffer, for the corrected Delta
  uint16_t* dq;       // bf16 [dq_rows][Hq][D]
  const int32_t* eff;
  const int4* items;  // the query-tile schedule
  const int32_t* counters;
  int32_t* claim;  // dynamic hand-out counter (zeroed by the planner)
  int32_t* dev_status;
  int B, Hq, Hkv, cp, causal;
  int group_kv;  // kv heads per locality group (divides Hkv)
  int64_t T_q, dq_rows;
  float scale, scale_log2;
  int step_lo, step_hi;  // always the whole ring
  int test_stall;  // test hook: every thread waits for a barrier nothing completes
  ScoreMods mods;  // scored attention
};

// host launchers (each returns a cudaError_t)
cudaError_t launch_plan(const PlanParams& p, cudaStream_t st);
cudaError_t launch_fwd(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool step_mode,
                       bool dyn, int grid, cudaStream_t st);
cudaError_t launch_fwd_dual(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool step_mode,
                            int grid, cudaStream_t st);
cudaError_t launch_bwd(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                       const CUtensorMap& tv, int D, bool grouped, int grid, cudaStream_t st);
cudaError_t launch_dq(const DqParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool grouped,
                      int grid, cudaStream_t st);
// scored attention: the same kernels with the score modifications `mod`
cudaError_t launch_score_fwd(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, int mod,
                             int grid, cudaStream_t st);
cudaError_t launch_score_fwd_dual(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, int mod,
                                  int grid, cudaStream_t st);
cudaError_t launch_score_bwd(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                             const CUtensorMap& tv, int D, bool grouped, int mod, int grid, cudaStream_t st);
cudaError_t launch_bwd_join(const float* part, int parts, uint16_t* dk, uint16_t* dv, float scale, const int32_t* eff,
                            int B, int64_t T_kv, int Hkv, int D, const int32_t* dev_status, cudaStream_t st);
cudaError_t launch_score_bwd_parts(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo,
                                   const CUtensorMap& tk, const CUtensorMap& tv, int D, int mod, int grid,
                                   cudaStream_t st);
cudaError_t launch_score_dq(const DqParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool grouped,
                            int mod, int grid, cudaStream_t st);
cudaError_t launch_docs(const int32_t* doc_q, const int32_t* doc_kv, const int32_t* eff, int B, int64_t T_q,
                        int64_t T_kv, int2* rows_q, int2* rows_kv, int32_t* doc_err, const int32_t* dev_status,
                        cudaStream_t st);
cudaError_t launch_lse_merge(float* o_acc, float* lse_acc, const float* o_part, const float* lse_part, int64_t T,
                             int H, int D, cudaStream_t st);
cudaError_t launch_lse_merge_bf16(float* o_acc, float* lse_acc, const uint16_t* o_part, const float* lse_part,
                                  int64_t T, int H, int D, cudaStream_t st);
cudaError_t launch_tail_zero(uint16_t* dq, uint16_t* dk, uint16_t* dv, int64_t dq_rows, int64_t dkv_rows, int Hq,
                             int Hkv, int D, const int32_t* pad_q_end, const int32_t* pad_kv_end,
                             const int32_t* dev_status, cudaStream_t st);
cudaError_t launch_bwd_prep(const uint16_t* o, const uint16_t* dout, const float* lse, float* delta, float* lse2,
                            const int32_t* eff, int B, int64_t T_q, int Hq, int D, const int32_t* dev_status,
                            cudaStream_t st);

int num_sms();
bool take_test_stall(int kernel_id);
int test_fwd_kernel();
void prof_before(int kernel_id, cudaStream_t st);
void prof_after(int kernel_id, cudaStream_t st);
void count_launch();

}  // namespace thd
