// Attention of one new token per sequence over a paged key-value cache
// (thd_attn_decode in the header): per sequence, kv head and run of at most 8, 16 or
// 32 of its query heads one work item, whose slots are read once.
//
// What bounds it: HBM.  A slot's keys and values are 4 D bytes (2 D in e4m3)
// for 4 D G flops, G query heads a kv head: G to 2 G flops a byte, far under what
// the tensor cores need to become the limit, so the products run as warp-level
// matrix instructions (m16n8k16) in which the slots are the 16 rows and the
// query heads the 8 columns: S^T = K q^T, O^T = V^T P^T.  No row of the
// instruction is padding, only heads short of 8 are.  e4m3 rows become fp16
// operands in registers (their instructions of 32 elements are made of the same
// steps on this GPU, and cost more).
//
// Work: every item's slots are cut into units of 64; a block takes a contiguous
// run of all items' units, as long as every other block's, whatever the
// sequences' lengths (they are read on the device: a captured graph stays
// balanced while they grow).  Where a block's run begins or ends inside an item
// it leaves an fp32 partial, which the join kernel adds up in the order of the
// blocks; both run in one wave and nothing is summed by atomics.
//
// Inside a block each warp walks its own tiles (every kWarps-th of the run's)
// through its own ring of stages in shared memory, filled with 16-byte
// asynchronous copies that take each row from wherever its page lies (any page
// size, any order of pages, slots and heads), and keeps its own running maximum
// and sum: no barrier between warps until the item's end, during which the next
// item's first copies are under way.
//
// Measured on one GB300, heads of 128, of the rate of a plain copy: bf16, 524,288
// slots of 8 kv heads 293 us (108%), 38 sequences of 8192 with 8, 16 or 32 heads
// a kv head 178, 180, 184 us (105, 104, 102%); e4m3, 1,048,576 slots 308 us (103%),
// 38 sequences with 8, 16, 32 heads 104, 115, 172 us (91, 82, 55%: from 16
// heads on the conversions, softmax and products of a warp's tile take longer than
// its bytes, and with 32 two warps a scheduler hide too little of that: it issues
// in 29% of the cycles, the tensor pipe works in 27%).  Items of one or two units
// cost a block what long ones do at their beginning and end: 4096 sequences of 16
// slots 281 us (14%), 1024 of 64 86 (46%), 256 of 128 36 (54%).  A call begins and ends in about 10 us (lengths, table and first
// rows are three loads one after the other; the join 2.5 us).
#include <cfloat>

#include <cuda_fp16.h>

#include "cache.cuh"
#include "ptx.cuh"

namespace thd {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecTile = 8192;  // bytes of a stage: a tile's keys, then its values
constexpr int kUnit = 64;       // slots
constexpr int kLead = 3;        // units that an item's beginning and end cost (1: +4% for 32 ragged sequences)
constexpr int kMinUnits = 2;    // of a block, while there are few

constexpr float kSlack = 8.f;   // see the running maximum
constexpr float kRaise = 7.f;   // fp16 probabilities are 2^7 times as large: 2^15 at most, 2^-31 at least
constexpr float kLeastScale = -112.f;  // log2 of the least scale of a row: a stored exponent of 15
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

int decode_heads(int G) { return G <= 8 ? 8 : G <= 16 ? 16 : 32; }
int decode_blocks(int B, int Hkv, int G, int64_t capacity) {
  const int64_t items = (int64_t)B * Hkv * ((G + decode_heads(G) - 1) / decode_heads(G));
  const int64_t total = items * ((capacity + kUnit - 1) / kUnit + kLead), n = (total + kMinUnits - 1) / kMinUnits;
  return n < kDecodeMaxGrid ? (int)n : kDecodeMaxGrid;
}

// ------------------------------------------------------------------ PTX
THD_DEV void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
THD_DEV void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// A 16-byte asynchronous copy, and one that fills with zeros (reading nothing) unless `on`.
THD_DEV void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
THD_DEV void cp16_if(uint32_t dst, const void* src, bool on) { cp_async_16(dst, src, on ? 16 : 0); }
THD_DEV uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool kHalf>
THD_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 numbers as two pairs of fp16, exactly.
THD_DEV void e4m3x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
template <bool kHalf>
THD_DEV uint32_t pack2(float lo, float hi) {
  if (kHalf) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
THD_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
THD_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// 2^(e - 127) of a stored exponent; 255: NaN.
THD_DEV float scale_of(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x400000u : e << 23);
}

// ------------------------------------------------------------------ the cut into units
struct Range {
  int n, s;  // slots of a sequence, the first visible one
};
THD_DEV Range range_of(const DecodeParams& p, int b) {
  bool bad;
  Range r;
  r.n = slots_of(p.c, b, bad);
  r.s = p.start ? p.start[b] : 0;
  r.s = r.s < 0 ? 0 : r.s > r.n ? r.n : r.s;
  return r;
}
THD_DEV int units_of(const Range& r) { return (r.n - r.s + kUnit - 1) / kUnit; }
// What an item counts in the cut: its units, and kLead in front of them for its
// beginning and end (queries, first loads, the join of the warps).
THD_DEV int cost_of(const Range& r) {
  const int n = units_of(r);
  return n > 0 ? n + kLead : 0;
}

// Blocks that share `total` units, and what the c-th of them takes: [c total /
// blocks, (c + 1) total / blocks).
THD_DEV int64_t blocks_for(int64_t total, int grid) {
  const int64_t n = (total + kMinUnits - 1) / kMinUnits;
  return n < grid ? n : grid;
}
// A quotient of numbers >= 0: most fit 32 bits, where dividing takes a third of the time.
THD_DEV int64_t quotient(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
THD_DEV int64_t owner_of(int64_t unit, int64_t total, int64_t blocks) { return quotient((unit + 1) * blocks - 1, total); }

// ------------------------------------------------------------------ the walk
// What a block works on at a time: slots [k0, k1) of a sequence, for query heads
// h0 .. of kv head g.
struct Segment {
  int b, g, h0, k0, k1;
  int i0;      // units of the item in front of it
  bool last;   // the item ends with it
  int64_t at;  // where the item's cost begins in the cut
};

template <bool kFp8, int D, int NT>
struct DecShape {
  static constexpr int kRow = D * (kFp8 ? 1 : 2);      // bytes
  static constexpr int kKeys = kDecTile / 2 / kRow;    // slots of a tile: 16, 32 or 64
  static constexpr int kSub = kKeys / 16;
  static constexpr int kPieces = kRow / 16;
  static constexpr int kHeads = 8 * NT;
  // Stages of a warp and blocks of an SM: 8 warps with 16 KB each keep enough
  // bytes in flight for bf16 (a third stage: 301 -> 311 us for 524,288 slots); where
  // the conversions of e4m3 leave a warp little time to wait, 12 do better (8 heads
  // 350 -> 329 us for 1,048,576 slots, 16 heads 121 -> 115 for 38 x 8192)
  static constexpr int kStages = 2;
  static constexpr int kPerSm = kFp8 && NT <= 2 ? 3 : 2;
  // slots worked on at a time, in sixteens: more of them overlap better, fewer
  // leave the registers to the heads (e4m3, 32 heads: 182 us at 16 slots, 171 at 32)
  static constexpr int kStep = NT == 1 || kSub < 2 ? kSub : 2;
  // bf16 probabilities as two numbers each (to 2^-16 instead of 2^-8): a second
  // product of every tile, which up to 16 heads' time does not show (at 32 heads 38
  // sequences of 8192 slots take 211 us instead of 190)
  static constexpr bool kTwo = !kFp8 && NT <= 2;
  // whether a warp's part of O fits one stage, so that the other may be filled meanwhile
  static constexpr bool kAhead = kHeads * D * 4 <= kDecTile;
  // shared memory, bytes
  static constexpr int kRing = kStages * kDecTile;  // a warp's
  static constexpr int kMeta = kStages * kKeys * 12; // a warp's: the rows' scales, positions
  static constexpr int kQ = D * kHeads * 2;
  static constexpr size_t kSmem = (size_t)kDecWarps * (kRing + kMeta) + kQ + sizeof(float) * (kHeads * (2 + 3 * kDecWarps));
  static_assert(kHeads * D * 4 <= kRing, "a warp's partial fits its ring");
};

// A tile's keys or values: row r's 16-byte piece c lies at piece c ^ x(r) of the
// row, x(r) = r mod 8 (rows of 64 bytes: r / 2 mod 4), so that eight rows' equal
// pieces lie in eight different bank groups.  Where a lane's row is fixed but for
// multiples of 8, or its piece but for even numbers, what varies is an exclusive
// or of address bits 4 to 7 and a constant.
template <int kPieces>
THD_DEV uint32_t swz(int r, int c) {
  return (uint32_t)(r * kPieces * 16 + ((c ^ (kPieces >= 8 ? r & 7 : (r >> 1) & 3)) << 4));
}

template <bool kFp8, int D, int NT>
__global__ void __launch_bounds__(kDecThreads, DecShape<kFp8, D, NT>::kPerSm) decode_kernel(const DecodeParams p) {
  using S = DecShape<kFp8, D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t s_seg[kDecThreads + 1];
  __shared__ int s_at[kDecWarps];  // where a warp's part of O lies in its ring
  const CacheView& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  follow();
  uint8_t* const ring = smem + warp * S::kRing;
  uint8_t* const meta = smem + kDecWarps * S::kRing + warp * S::kMeta;
  uint8_t* const s_q = smem + kDecWarps * (S::kRing + S::kMeta);
  float* const s_hs = reinterpret_cast<float*>(s_q + S::kQ);  // [kHeads] score multiplier, then slopes
  float* const s_sl = s_hs + S::kHeads;
  float* const s_ml = s_sl + S::kHeads;                       // [kDecWarps][3][kHeads]

  // the block table on its way to L2 while the lengths come: a line a thread
  {
    const int64_t bytes = (c.B - 1) * c.table_stride * 4 + c.capacity / c.page.d * 4;
    const int64_t line = ((int64_t)blockIdx.x * kDecThreads + tid) * 128;
    if (line < bytes)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(c.table) + line));
  }
  // units in front of each sequence
  const int per = (c.B + kDecThreads - 1) / kDecThreads;
  const int b_lo = tid * per < c.B ? tid * per : c.B, b_hi = b_lo + per < c.B ? b_lo + per : c.B;
  {
    int64_t sum = 0;
    for (int b = b_lo; b < b_hi; ++b) sum += cost_of(range_of(p, b));
    s_seg[tid + 1] = sum;
    if (tid == 0) s_seg[0] = 0;
    __syncthreads();
    if (warp == 0) {
      int64_t run = 0;
#pragma unroll
      for (int k = 0; k < kDecWarps; ++k) {
        int64_t v = s_seg[1 + 32 * k + lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, v, d);
          if (lane >= d) v += y;
        }
        v += run;
        s_seg[1 + 32 * k + lane] = v;
        run = __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
  }
  const int HG = c.Hkv * p.blocks;  // items of a sequence
  const int64_t total = s_seg[kDecThreads] * HG;
  const int64_t blocks = blocks_for(total, (int)gridDim.x);
  int64_t u = 0, u_end = 0;
  if (blockIdx.x < blocks) {
    u = quotient(blockIdx.x * total, blocks);
    u_end = quotient((blockIdx.x + 1) * total, blocks);
  }

  // the first item
  int b = 0, item = 0, ic = 0;  // ic: where in the item's cost
  if (u < u_end) {
    const int64_t ub = quotient(u, HG);
    int seg = 0;
    for (int step = kDecThreads / 2; step > 0; step >>= 1)
      if (s_seg[seg + step] <= ub) seg += step;
    b = seg * per;
    int64_t before = s_seg[seg];
    for (; b < c.B; ++b) {
      const int n = cost_of(range_of(p, b));
      if (ub < before + n) {
        const int64_t r = u - before * HG;
        item = (int)quotient(r, n);
        ic = (int)(r - (int64_t)item * n);
        break;
      }
      before += n;
    }
  }

  // the next run of an item's units in this block's share
  auto next = [&](Segment& x) {
    while (u < u_end && b < c.B) {
      const Range rg = range_of(p, b);
      const int units = units_of(rg), cost = units + kLead;
      const int step = u_end - u < cost - ic ? (int)(u_end - u) : cost - ic;
      x.b = b;
      x.g = item / p.blocks;
      x.h0 = (item % p.blocks) * S::kHeads;
      x.i0 = ic > kLead ? ic - kLead : 0;
      const int take = ic + step - kLead - x.i0;  // 0 or less: nothing but a part of what the item counts in front
      x.last = x.i0 + take == units;
      x.k0 = rg.s + x.i0 * kUnit;
      x.k1 = rg.n - x.k0 < take * kUnit ? rg.n : x.k0 + take * kUnit;
      x.at = u - ic;
      u += step;
      ic = 0;
      if (u < u_end && ++item == HG) {
        item = 0;
        do ++b;
        while (b < c.B && units_of(range_of(p, b)) == 0);
      }
      if (take > 0) return true;
    }
    return false;
  };

  const int64_t v_minus_k = c.v - c.k;
  const uint32_t ring_a = smem_u32(ring);

  // ---- a tile's copies
  constexpr int kRpl = S::kKeys > 32 ? S::kKeys / 32 : 1;  // rows a lane finds the place of
  int pid[kRpl], pid_after[kRpl];  // pages of the rows of the next tile to issue, and of the one after it
  // exponents on their way to shared memory: loaded when a tile's copies are
  // issued, looked at a tile later (combining them sooner would wait for them)
  uint32_t pend_k[kRpl], pend_v[kRpl];
  int pend_stage = -1;
  auto fetch_pid = [&](const Segment& x, int t) {
#pragma unroll
    for (int r = 0; r < kRpl; ++r) {
      const int row = lane + 32 * r, j = x.k0 + t * S::kKeys + row;
      pid[r] = pid_after[r];
      pid_after[r] = row < S::kKeys && j < x.k1 ? c.table[x.b * c.table_stride + place_of(c, j).page] : 0;
    }
  };
  auto flush = [&]() {
    if (kFp8 && pend_stage >= 0) {
#pragma unroll
      for (int r = 0; r < kRpl; ++r)
        if (lane + 32 * r < S::kKeys)
          reinterpret_cast<float2*>(meta + pend_stage * 12 * S::kKeys)[lane + 32 * r] =
              make_float2(scale_of(pend_k[r]), pend_v[r] == 255u ? NAN : (float)((int)pend_v[r] - 127));
    }
    pend_stage = -1;
  };
  auto issue = [&](const Segment& x, int t, int stage) {
    const int j0 = x.k0 + t * S::kKeys, k1 = x.k1, g = x.g;
    const uint32_t slot0 = place_of(c, j0).slot;
    constexpr int kRowsPer = 32 / S::kPieces;  // rows of one warp-wide copy: 512 bytes
    const int piece = lane % S::kPieces, row0 = lane / S::kPieces;
    const uint32_t dst = ring_a + stage * kDecTile + swz<S::kPieces>(row0, piece), meta_a = smem_u32(meta) + stage * 12 * S::kKeys;
    // of the i-th copy: row i kRowsPer + row0
    auto at_row = [&](int i) { return dst ^ (S::kPieces >= 8 ? ((i * kRowsPer) & 7) << 4 : 0); };
    pend_stage = stage;
    const int page0 = __shfl_sync(0xffffffffu, pid[0], 0);
    if (slot0 + S::kKeys <= c.page.d && j0 + S::kKeys <= k1 && page0 >= 0 && page0 < c.num_pages) {
      // the whole tile in one page
      const uint8_t* from = c.k + at(c.row, page0, slot0 + row0, g) + 16 * piece;
      const uint8_t* from_v = from + v_minus_k;
      const int64_t step = kRowsPer * c.row.slot;
#pragma unroll
      for (int i = 0; i < S::kKeys / kRowsPer; ++i) {
        cp16(at_row(i) + i * 512, from);
        cp16(at_row(i) + i * 512 + kDecTile / 2, from_v);
        from += step;
        from_v += step;
      }
#pragma unroll
      for (int r = 0; r < kRpl; ++r) {
        const int row = lane + 32 * r;
        if (row < S::kKeys) {
          if (kFp8) {
            const int64_t e = at(c.exp, page0, slot0 + row, g);
            pend_k[r] = c.k_exp[e];
            pend_v[r] = c.v_exp[e];
          }
          if (p.pos) cp_async_4(meta_a + S::kKeys * 8 + row * 4, p.pos + at(p.pos_at, page0, slot0 + row, g));
        }
      }
      return;
    }
    int64_t off[kRpl];
#pragma unroll
    for (int r = 0; r < kRpl; ++r) {
      const int row = lane + 32 * r, j = j0 + row;
      off[r] = -1;
      pend_k[r] = pend_v[r] = 127u;
      if (row < S::kKeys && j < k1) {
        const uint32_t slot = place_of(c, j).slot;
        if (pid[r] < 0 || pid[r] >= c.num_pages) {
          raise(p.status, THD_DEV_ERR_PAGE);
        } else {
          off[r] = at(c.row, pid[r], slot, g);
          if (kFp8) {
            const int64_t e = at(c.exp, pid[r], slot, g);
            pend_k[r] = c.k_exp[e];
            pend_v[r] = c.v_exp[e];
          }
          if (p.pos) cp_async_4(meta_a + S::kKeys * 8 + row * 4, p.pos + at(p.pos_at, pid[r], slot, g));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < S::kKeys / kRowsPer; ++i) {
      const int row = i * kRowsPer + row0;
      const int64_t o = __shfl_sync(0xffffffffu, off[kRpl > 1 ? (i * kRowsPer) / 32 : 0], row & 31);
      const uint8_t* const from = c.k + (o < 0 ? 0 : o + 16 * piece);
      cp16_if(at_row(i) + i * 512, from, o >= 0);
      cp16_if(at_row(i) + i * 512 + kDecTile / 2, from + v_minus_k, o >= 0);
    }
  };

  // ---- an item's queries: a warp takes every kDecWarps-th head
  constexpr int kPairs = D / 64, kQHeads = S::kHeads / kDecWarps;  // of a lane, of a warp
  uint32_t q_next[kQHeads][kPairs];
  auto fetch_q = [&](const Segment& x) {
#pragma unroll
    for (int i = 0; i < kQHeads; ++i) {
      const int n = warp + i * kDecWarps;
      const uint32_t* const row = reinterpret_cast<const uint32_t*>(p.q + x.b * p.q_stride + (int64_t)(x.g * p.G + x.h0 + n) * D);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) q_next[i][k] = x.h0 + n < p.G ? row[lane + 32 * k] : 0u;
    }
  };

  Segment cur;
  const bool any = next(cur);
  if (any) {
    fetch_q(cur);
    fetch_pid(cur, warp);
    fetch_pid(cur, warp + kDecWarps);
#pragma unroll
    for (int x = 0; x < S::kStages; ++x) {
      const int t = warp + x * kDecWarps;
      flush();
      if (cur.k0 + t * S::kKeys < cur.k1) issue(cur, t, x);
      fetch_pid(cur, t + 2 * kDecWarps);
      cp_commit();
    }
  }

  // while those come: rows without a visible slot, bad lengths, what the join reads
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    bool bad;
    slots_of(c, b, bad);
    if (bad && tid == 0) raise(p.status, THD_DEV_ERR_KV_LEN);
    if (units_of(range_of(p, b)) == 0) {
      for (int i = tid; i < p.Hq * D / 8; i += kDecThreads)
        reinterpret_cast<uint4*>(p.o + (int64_t)b * p.Hq * D)[i] = make_uint4(0, 0, 0, 0);
      for (int h = tid; h < p.Hq; h += kDecThreads) p.lse[(int64_t)h * c.B + b] = -INFINITY;
      if (p.by_item)
        for (int i = tid; i < c.Hkv * p.blocks; i += kDecThreads) p.joins[b * c.Hkv * p.blocks + i].count = 0;
    }
  }
  if (tid == 0 && !p.by_item) p.joins[blockIdx.x].count = 0;
  if (!any) return;

  int stage = 0;
  for (;;) {
    const int b = cur.b, g = cur.g, h0 = cur.h0, k0 = cur.k0, k1 = cur.k1;
    const int heads = p.G - h0 < S::kHeads ? p.G - h0 : S::kHeads;
    const int tiles = (k1 - k0 + S::kKeys - 1) / S::kKeys;
    const int seen = p.slopes ? (p.seen ? p.seen[b] : c.kv_len[b]) : 0;
#pragma unroll
    for (int i = 0; i < kQHeads; ++i) {
      const int n = warp + i * kDecWarps;
      uint32_t(&w)[kPairs] = q_next[i];
      float mul = 1.f;
      if (kFp8) {
        // fp16 queries: the largest of a head is brought to [2^14, 2^15) by a
        // power of two, so elements down to 2^-28 of it keep bf16's precision
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) big = __vmaxu2(big, w[k] & 0x7fff7fffu);
        big = max(big >> 16, big & 0xffffu);
        big = __reduce_max_sync(0xffffffffu, big);
        int e = (int)(big >> 7);                  // exponent field of the largest
        e = e == 0 ? 1 : e;
        const int up = 127 + 14 - e;              // 2^up times the head; in two steps, each a normal number
        const float m1 = __uint_as_float((uint32_t)(127 + up / 2) << 23);
        const float m2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
        mul = (1.f / m1) * (1.f / m2);
        if (e == 255) mul = NAN;                  // an infinity or NaN among the elements
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          const float lo = __uint_as_float(w[k] << 16) * m1 * m2, hi = __uint_as_float(w[k] & 0xffff0000u) * m1 * m2;
          w[k] = pack2<true>(lo, hi);
        }
      }
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        const int d = 2 * (lane + 32 * k), ks = d >> 4, in = d & 15;
        // fragment order of the matrix instruction's second operand; next to
        // e4m3 keys a step's elements are counted as the keys' bytes arrive
        const int reg = kFp8 ? (in & 3) >> 1 : in >> 3, quad = kFp8 ? in >> 2 : (in & 7) >> 1;
        *reinterpret_cast<uint32_t*>(s_q + ((((ks * NT + (n >> 3)) * 32 + (n & 7) * 4 + quad) * 2 + reg) * 4)) = w[k];
      }
      if (lane == 0) {
        s_hs[n] = mul * (p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e);
        s_sl[n] = p.slopes && n < heads ? p.slopes[cur.g * p.G + cur.h0 + n] * kLog2e : 0.f;
      }
    }
    __syncthreads();

    // ---- tiles: running maximum (base 2) and sum of each head, O^T
    // nm: the maximum, negated; before the first score the largest float, so that
    // no difference is infinity less infinity
    // mo: the maximum of score + log2 of the value's scale, what O is relative to;
    // up: from a probability to what the product takes, but for its value's scale
    float nm[NT][2], mo[NT][2], l[NT][2], up[NT][2], o[D / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) nm[nt][e] = FLT_MAX, mo[nt][e] = -FLT_MAX, l[nt][e] = 0.f, up[nt][e] = 1.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][nt][e] = 0.f;

    for (int t = warp; t < tiles; t += kDecWarps) {
      cp_wait<S::kStages - 1>();
      __syncwarp();
#pragma unroll 1
      for (int r0 = 0; r0 < S::kKeys && k0 + t * S::kKeys + r0 < k1; r0 += 16 * S::kStep) {  // rows of the tile at a time
        const float2* const scales = reinterpret_cast<const float2*>(meta + stage * 12 * S::kKeys) + r0;
        const uint32_t* const numbers = reinterpret_cast<const uint32_t*>(meta + stage * 12 * S::kKeys + 8 * S::kKeys) + r0;
        float s[S::kStep][NT][4];
#pragma unroll
        for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[sub][nt][e] = 0.f;
        // lanes' rows and pieces of a load's four 8x8 matrices: rows 0-7 and 8-15
        // of the first 16 bytes, then of the second; of bf16 values, which are
        // loaded transposed, the two pieces of rows 0-7, then of rows 8-15
        constexpr int kSubBytes = 16 * S::kRow;
        const uint32_t tile_a = ring_a + stage * kDecTile + r0 * S::kRow;
        const uint32_t kt = tile_a + swz<S::kPieces>(lane & 15, lane >> 4);
        const uint32_t vt = kFp8 ? kt : tile_a + swz<S::kPieces>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
        constexpr int kSteps = kFp8 ? 2 : 1;  // steps of 16 elements in 32 bytes
#pragma unroll
        for (int kp = 0; kp < S::kPieces / 2; ++kp) {
          uint2 bq[kSteps][NT];
#pragma unroll
          for (int x = 0; x < kSteps; ++x)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              bq[x][nt] = *reinterpret_cast<const uint2*>(s_q + (((kp * kSteps + x) * NT + nt) * 32 + lane) * 8);
#pragma unroll
          for (int sub = 0; sub < S::kStep; ++sub) {
            uint32_t r[4];
            ldsm4(r, (kt ^ (kp << 5)) + sub * kSubBytes);
            if (kFp8) {
              uint32_t a0[4], a1[4];
              e4m3x4(r[0], a0[0], a0[2]);
              e4m3x4(r[1], a0[1], a0[3]);
              e4m3x4(r[2], a1[0], a1[2]);
              e4m3x4(r[3], a1[1], a1[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816<true>(s[sub][nt], a0, bq[0][nt].x, bq[0][nt].y);
                mma16816<true>(s[sub][nt], a1, bq[kSteps - 1][nt].x, bq[kSteps - 1][nt].y);
              }
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<false>(s[sub][nt], r, bq[0][nt].x, bq[0][nt].y);
            }
          }
        }
        // scores in base 2
        const int j0 = k0 + t * S::kKeys + r0;
        float lv[S::kStep][2];  // log2 of the values' scales
        float2 hs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) hs[nt] = *reinterpret_cast<const float2*>(s_hs + nt * 8 + 2 * t4);
#pragma unroll
        for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float2 sc;
            if (kFp8) {
              sc = scales[sub * 16 + half * 8 + gid];
              lv[sub][half] = sc.y;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float &y0 = s[sub][nt][2 * half], &y1 = s[sub][nt][2 * half + 1];
              if (kFp8) fmul2(y0, y1, y0, y1, sc.x, sc.x);
              fmul2(y0, y1, y0, y1, hs[nt].x, hs[nt].y);
            }
          }
        if (p.cap > 0.f) {
#pragma unroll
          for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[sub][nt][e] = p.cap * kLog2e * tanhf(s[sub][nt][e]);
        }
        if (p.slopes) {
#pragma unroll
          for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int row = sub * 16 + half * 8 + gid;
              const float far = (float)(int)((uint32_t)seen - 1u - (p.pos ? numbers[row] : (uint32_t)(j0 + row)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float2 sl = *reinterpret_cast<const float2*>(s_sl + nt * 8 + 2 * t4);
                s[sub][nt][2 * half] = fmaf(-sl.x, far, s[sub][nt][2 * half]);
                s[sub][nt][2 * half + 1] = fmaf(-sl.y, far, s[sub][nt][2 * half + 1]);
              }
            }
        }
        if (j0 + 16 * S::kStep > k1) {  // slots behind the last
#pragma unroll
          for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (j0 + sub * 16 + half * 8 + gid >= k1) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[sub][nt][2 * half] = s[sub][nt][2 * half + 1] = -INFINITY;
              }
        }
        if (p.weight_out) {
#pragma unroll
          for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int j = j0 + sub * 16 + half * 8 + gid;
              if (j < k1) {
                float* const to = p.scores + (((int64_t)b * c.Hkv + g) * c.capacity + j) * p.G + h0 + 2 * t4;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (nt * 8 + 2 * t4 + e < heads) to[nt * 8 + e] = s[sub][nt][2 * half + e];
              }
            }
        }
        // The maximum moves only when a score passes it by more than kSlack: until
        // then the lanes need not know one another's scores.  Probabilities then
        // reach 2^8, which any bf16, fp16 or fp32 sum takes.
        float mx[NT][2], mxo[NT][2];
        bool moved = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[nt][e] = mxo[nt][e] = -INFINITY;
#pragma unroll
            for (int sub = 0; sub < S::kStep; ++sub) {
              mx[nt][e] = fmax3(mx[nt][e], s[sub][nt][e], s[sub][nt][2 + e]);
              if (kFp8) mxo[nt][e] = fmax3(mxo[nt][e], s[sub][nt][e] + lv[sub][0], s[sub][nt][2 + e] + lv[sub][1]);
            }
            moved |= mx[nt][e] + nm[nt][e] > kSlack;
            if (kFp8) moved |= mxo[nt][e] > mo[nt][e] + kSlack;
          }
        if (__any_sync(0xffffffffu, moved)) {
          // A row of zeros adds nothing to O whatever its scale says, so it must not
          // set what O is relative to: rows that would raise that are looked at, and
          // count as of the least scale if they are zeros.
          if (kFp8) {
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) far |= mxo[nt][e] > mo[nt][e] + kSlack;
            if (__any_sync(0xffffffffu, far)) {
              constexpr int kRows = 16 * S::kStep;
              uint32_t zeros[(kRows + 31) / 32];
              bool some = false;
#pragma unroll
              for (int k = 0; k < kRows; k += 32) {
                const uint4* const x =
                    reinterpret_cast<const uint4*>(ring + stage * kDecTile + kDecTile / 2 + (r0 + k + lane) * S::kRow);
                bool zero = k + lane < kRows;
                for (int i = 0; zero && i < S::kPieces; ++i)
                  zero = ((x[i].x | x[i].y | x[i].z | x[i].w) & 0x7f7f7f7fu) == 0;
                zeros[k / 32] = __ballot_sync(0xffffffffu, zero);
                some |= zeros[k / 32] != 0;
              }
              if (some) {
#pragma unroll
                for (int sub = 0; sub < S::kStep; ++sub)
#pragma unroll
                  for (int half = 0; half < 2; ++half) {
                    const int row = sub * 16 + half * 8 + gid;
                    // (a row marked as no number stays one)
                    if ((zeros[sub / 2] >> (row & 31) & 1u) && lv[sub][half] == lv[sub][half]) lv[sub][half] = kLeastScale;
                  }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    mxo[nt][e] = -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < S::kStep; ++sub)
                      mxo[nt][e] = fmax3(mxo[nt][e], s[sub][nt][e] + lv[sub][0], s[sub][nt][2 + e] + lv[sub][1]);
                  }
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float al[2], alo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) {
                mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], d));
                if (kFp8) mxo[nt][e] = fmaxf(mxo[nt][e], __shfl_xor_sync(0xffffffffu, mxo[nt][e], d));
              }
              const float nm2 = fminf(nm[nt][e], -mx[nt][e]);
              al[e] = ex2(nm2 - nm[nt][e]);
              nm[nt][e] = nm2;
              alo[e] = al[e];
              if (kFp8) {
                const float mo2 = fmaxf(mo[nt][e], mxo[nt][e]);
                alo[e] = ex2(mo[nt][e] - mo2);
                mo[nt][e] = mo2;
                up[nt][e] = ex2(kRaise - nm2 - mo2);
              }
              l[nt][e] *= al[e];
            }
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              fmul2(o[d][nt][0], o[d][nt][1], o[d][nt][0], o[d][nt][1], alo[0], alo[1]);
              fmul2(o[d][nt][2], o[d][nt][3], o[d][nt][2], o[d][nt][3], alo[0], alo[1]);
            }
          }
        }
        // probabilities: summed in fp32, and for the product rounded to bf16 next
        // to bf16 values (twice, the second time what the first left), to fp16
        // next to e4m3 ones (2^-11, and 2^-32 of the largest)
        uint32_t pb[S::kStep][NT][2], pr[S::kTwo ? S::kStep : 1][NT][2];
#pragma unroll
        for (int sub = 0; sub < S::kStep; ++sub) {
          float vs[2];
          if (kFp8) vs[0] = ex2(lv[sub][0]), vs[1] = ex2(lv[sub][1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[2][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float y0, y1;
              fadd2(y0, y1, s[sub][nt][2 * half], s[sub][nt][2 * half + 1], nm[nt][0], nm[nt][1]);
              y0 = ex2(y0);
              y1 = ex2(y1);
              fadd2(l[nt][0], l[nt][1], l[nt][0], l[nt][1], y0, y1);
              if (kFp8) {
                fmul2(y0, y1, y0, y1, up[nt][0], up[nt][1]);
                fmul2(y0, y1, y0, y1, vs[half], vs[half]);
              }
              w[half][0] = y0;
              w[half][1] = y1;
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t first = pack2<kFp8>(w[half][0], w[half][1]);
              pb[sub][nt][half] = movm_t(first);
              if (S::kTwo) {
                float r0, r1;
                fadd2(r0, r1, w[half][0], w[half][1], -__uint_as_float(first << 16), -__uint_as_float(first & 0xffff0000u));
                pr[S::kTwo ? sub : 0][nt][half] = movm_t(pack2<false>(r0, r1));
              }
            }
          }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int dp = 0; dp < S::kPieces / 2; ++dp)
#pragma unroll
          for (int sub = 0; sub < S::kStep; ++sub) {
            uint32_t r[4];
            if (kFp8) {
              // matrices: slots 0-7 and 8-15 of 16 elements, then of the next 16;
              // a register has elements 2 gid and 2 gid + 1 of two slots
              ldsm4t(r, (vt ^ (dp << 5)) + kDecTile / 2 + sub * kSubBytes);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t a[4];
                e4m3x4(__byte_perm(r[2 * x], 0, 0x3120), a[0], a[1]);
                e4m3x4(__byte_perm(r[2 * x + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<true>(o[(kFp8 ? 2 * dp + x : 0)][nt], a, pb[sub][nt][0], pb[sub][nt][1]);
              }
            } else {
              ldsm4t(r, (vt ^ (dp << 5)) + kDecTile / 2 + sub * kSubBytes);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816<false>(o[dp][nt], r, pb[sub][nt][0], pb[sub][nt][1]);
                if (S::kTwo) mma16816<false>(o[dp][nt], r, pr[S::kTwo ? sub : 0][nt][0], pr[S::kTwo ? sub : 0][nt][1]);
              }
            }
          }
      }
      __syncwarp();  // the stage is read
      flush();
      const int tn = t + S::kStages * kDecWarps;
      if (tn < tiles) {
        issue(cur, tn, stage);
        fetch_pid(cur, tn + 2 * kDecWarps);
      }
      cp_commit();
      stage ^= 1;
    }

    // ---- what the next item begins with is on its way during this one's end:
    // its queries, its pages and the warp's first tile, into the stage that is free
    Segment after;
    const bool more = next(after);
    if (more) {
      fetch_q(after);
      fetch_pid(after, warp);
      fetch_pid(after, warp + kDecWarps);
    }

    // ---- the item's end: the warps' sums, then their O, through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        if (gid == 0) {
          float* const to = s_ml + warp * 3 * S::kHeads + nt * 8 + 2 * t4 + e;
          to[0] = kFp8 ? mo[nt][e] : -nm[nt][e];
          to[S::kHeads] = -nm[nt][e];
          to[2 * S::kHeads] = l[nt][e];
        }
      }
    // the warp's part of O goes through the other stage (or both)
    if (lane == 0) s_at[warp] = S::kAhead ? (stage ^ 1) * kDecTile : 0;
    __syncthreads();
    float* const mine = reinterpret_cast<float*>(ring + s_at[warp]);
    if (S::kAhead) {
      if (more) {
        if (after.k0 + warp * S::kKeys < after.k1) issue(after, warp, stage);
        fetch_pid(after, warp + 2 * kDecWarps);
      }
      cp_commit();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, s_ml[w * 3 * S::kHeads + nt * 8 + 2 * t4 + e]);
        f[e] = ex2((kFp8 ? mo[nt][e] : -nm[nt][e]) - top);
        if (kFp8) f[e] *= 1.f / 128;
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at_d = d * 16 + (kFp8 ? 2 * gid + (e >> 1) : gid + 8 * (e >> 1));
          const int n = nt * 8 + 2 * t4 + (e & 1);
          mine[n * D + (at_d ^ (n >> 1 & 3) << 3)] =  // eight words apart for the four lanes of a row
              o[d][nt][e] * f[e & 1];
        }
    }
    __syncthreads();
    const bool whole = cur.i0 == 0 && cur.last;
    if (tid == 0 && cur.last && (!whole || p.by_item)) {
      // the item's last block names its parts: the first block's is in that
      // one's second slot, the others' in their first
      const int64_t first = whole ? 0 : owner_of(cur.at + kLead, total, blocks);
      p.joins[p.by_item ? b * HG + g * p.blocks + h0 / S::kHeads : blockIdx.x] =
          DecodeJoin{b, g * p.G + h0, heads, (int)first, whole ? 0 : (int)(blockIdx.x - first) + 1};
    }
    const int64_t slot = 2 * (int64_t)blockIdx.x + (cur.i0 > 0 ? 0 : 1);
    for (int i = tid; i < heads * (D / 4); i += kDecThreads) {
      const int n = i / (D / 4), d = 4 * (i % (D / 4));
      float top = -FLT_MAX, topo = -FLT_MAX, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        topo = fmaxf(topo, s_ml[w * 3 * S::kHeads + n]);
        top = fmaxf(top, s_ml[w * 3 * S::kHeads + S::kHeads + n]);
      }
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        sum += s_ml[w * 3 * S::kHeads + 2 * S::kHeads + n] * ex2(s_ml[w * 3 * S::kHeads + S::kHeads + n] - top);
      }
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(smem + w * S::kRing + s_at[w] + (n * D + (d ^ (n >> 1 & 3) << 3)) * 4);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      if (whole) {
        const float f = sum == 0.f ? 0.f : ex2(topo - top) / sum;
        const int h = g * p.G + h0 + n;
        uint2 y;
        y.x = pack2<false>(x.x * f, x.y * f);
        y.y = pack2<false>(x.z * f, x.w * f);
        *reinterpret_cast<uint2*>(p.o + ((int64_t)b * p.Hq + h) * D + d) = y;
        if (d == 0) {
          const float lse2 = top + log2f(sum);
          p.lse[(int64_t)h * c.B + b] = lse2 * kLn2;
          if (p.weight_out) p.lse2[(int64_t)b * p.Hq + h] = lse2;
        }
      } else {
        *reinterpret_cast<float4*>(p.part + (slot * S::kHeads + n) * D + d) = x;
        if (d == 0) {
          float* const to = p.part_ml + (slot * S::kHeads + n) * 3;
          to[0] = topo, to[1] = top, to[2] = sum;
        }
      }
    }
    if (!more) return;
    __syncthreads();  // the rings are read
    cur = after;
#pragma unroll
    for (int x = S::kAhead ? 1 : 0; x < S::kStages; ++x) {
      const int t = warp + x * kDecWarps;
      flush();
      if (cur.k0 + t * S::kKeys < cur.k1) issue(cur, t, stage ^ x);
      fetch_pid(cur, t + 2 * kDecWarps);
      cp_commit();
    }
  }
}

// ------------------------------------------------------------------ the join
// The parts of an item that several blocks shared: a block of 128 threads for
// each (item or block that ended one, head or several), four parts at a time, a head's row across
// the lanes.  The sums run over the parts in order, four interleaved.
constexpr int kJoinThreads = 128;

template <int D, bool kSeveral>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeParams p, int kheads) {
  constexpr int kLanes = D / 4, kParts = kJoinThreads / kLanes;
  __shared__ float4 s_x[kJoinThreads];
  __shared__ float s_ml[kDecodeMaxGrid][3], s_top[kJoinThreads / 32][2], s_sum[kParts];
  const int tid = threadIdx.x;
  follow();
  depend();
  const DecodeJoin j = p.joins[blockIdx.x];
  if (j.count == 0) return;
  for (int n = blockIdx.y; n < j.heads; n += kSeveral ? (int)gridDim.y : j.heads) {
    // part k's row
    auto row_of = [&](int k) { return (2 * (int64_t)(j.first + k) + (k == 0 ? 1 : 0)) * kheads + n; };
    // the first rows are on their way while the maxima are found
    constexpr int kAhead = 8;
    const int lane = tid % kLanes, mine = tid / kLanes;
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (mine + i * kParts < j.count)
        ahead[i] = *reinterpret_cast<const float4*>(p.part + row_of(mine + i * kParts) * D + 4 * lane);
    float topo = -FLT_MAX, top = -FLT_MAX;
    for (int k = tid; k < j.count; k += kJoinThreads) {
      const float* ml = p.part_ml + row_of(k) * 3;
      s_ml[k][0] = ml[0], s_ml[k][1] = ml[1], s_ml[k][2] = ml[2];
      topo = fmaxf(topo, ml[0]);
      top = fmaxf(top, ml[1]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      topo = fmaxf(topo, __shfl_xor_sync(0xffffffffu, topo, d));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    if ((tid & 31) == 0) s_top[tid >> 5][0] = topo, s_top[tid >> 5][1] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) topo = fmaxf(topo, s_top[w][0]), top = fmaxf(top, s_top[w][1]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int k, const float4& y) {
      const float f = ex2(s_ml[k][0] - topo);
      sum += s_ml[k][2] * ex2(s_ml[k][1] - top);
      acc.x += y.x * f, acc.y += y.y * f, acc.z += y.z * f, acc.w += y.w * f;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (mine + i * kParts < j.count) add(mine + i * kParts, ahead[i]);
#pragma unroll 8
    for (int k = mine + kAhead * kParts; k < j.count; k += kParts)
      add(k, *reinterpret_cast<const float4*>(p.part + row_of(k) * D + 4 * lane));
    s_x[tid] = acc;
    if (lane == 0) s_sum[mine] = sum;
    __syncthreads();
    if (tid < kLanes) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float z = 0.f;
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const float4 y = s_x[k * kLanes + tid];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        z += s_sum[k];
      }
      const float f = z == 0.f ? 0.f : ex2(topo - top) / z;
      uint2 y;
      y.x = pack2<false>(x.x * f, x.y * f);
      y.y = pack2<false>(x.z * f, x.w * f);
      const int64_t row = (int64_t)j.b * p.Hq + j.h + n;
      *reinterpret_cast<uint2*>(p.o + row * D + 4 * tid) = y;
      if (tid == 0) {
        const float lse2 = top + log2f(z);
        p.lse[(int64_t)(j.h + n) * p.c.B + j.b] = lse2 * kLn2;
        if (p.weight_out) p.lse2[row] = lse2;
      }
    }
    if (kSeveral) __syncthreads();  // the sums are read
  }
}

// ------------------------------------------------------------------ the weights
// From the scores and the finished log-sum-exps, 4 G + 8 bytes a slot and kv head,
// the scores mostly from L2: `share` blocks for each (sequence, kv head), every
// one of them runs of 1024 slots, four a thread.  Where the numbers lie and what
// they were is found while the kernels in front still run.
constexpr int kWeightThreads = 256, kWeightSlots = 4;

__global__ void __launch_bounds__(kWeightThreads) decode_weights_kernel(const DecodeParams p, int share) {
  __shared__ float s_lse[kDecodeMaxGroup];
  const CacheView& c = p.c;
  const int tid = threadIdx.x, pair = (int)(blockIdx.x / share), b = pair / c.Hkv, g = pair % c.Hkv;
  follow();
  const Range rg = range_of(p, b);
  const float* const scores = p.scores + ((int64_t)b * c.Hkv + g) * c.capacity * p.G;
  constexpr int kRun = kWeightThreads * kWeightSlots;
  bool waited = false;
  for (int64_t j0 = rg.s + (int64_t)(blockIdx.x % share) * kRun; j0 < rg.n; j0 += (int64_t)share * kRun) {
    int64_t a[kWeightSlots];
    float w[kWeightSlots];
#pragma unroll
    for (int x = 0; x < kWeightSlots; ++x) {
      const int64_t j = j0 + x * kWeightThreads + tid;
      a[x] = -1;
      if (j < rg.n) {
        const Place to = place_of(c, (int)j);
        const int page = page_of(c, b, to.page);
        if (page >= 0) a[x] = at(p.weight_at, page, to.slot, g);
      }
    }
#pragma unroll
    for (int x = 0; x < kWeightSlots; ++x) w[x] = a[x] < 0 ? 0.f : p.weight_in[a[x]];
    if (!waited) {
      waited = true;
      depend();
      for (int n = tid; n < p.G; n += kWeightThreads) {
        const float z = p.lse2[(int64_t)b * p.Hq + g * p.G + n];
        s_lse[n] = z == -INFINITY ? INFINITY : z;
      }
      __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < kWeightSlots; ++x) {
      if (a[x] < 0) continue;
      const float* const s = scores + (j0 + x * kWeightThreads + tid) * p.G;
      float sum = 0.f;
      if (p.G % 4 == 0) {
#pragma unroll 4
        for (int n = 0; n < p.G; n += 4) {
          const float4 y = *reinterpret_cast<const float4*>(s + n);
          sum += ex2(y.x - s_lse[n]) + ex2(y.y - s_lse[n + 1]) + (ex2(y.z - s_lse[n + 2]) + ex2(y.w - s_lse[n + 3]));
        }
      } else {
        for (int n = 0; n < p.G; ++n) sum += ex2(s[n] - s_lse[n]);
      }
      w[x] += sum;
    }
#pragma unroll
    for (int x = 0; x < kWeightSlots; ++x)
      if (a[x] >= 0) p.weight_out[a[x]] = w[x];
  }
  if (!waited) depend();  // no block of a kernel ends before what it follows: the next one counts on that
}

// ------------------------------------------------------------------ launch
template <bool kFp8, int D, int NT>
static cudaError_t launch_decode_t(DecodeParams& p, cudaStream_t st) {
  using S = DecShape<kFp8, D, NT>;
  static bool allowed[64] = {};  // of this instantiation
  cudaError_t e = allow_smem(decode_kernel<kFp8, D, NT>, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  const int wave = S::kPerSm * num_sms(), most = decode_blocks(p.c.B, p.c.Hkv, p.G, p.c.capacity);
  p.grid = wave < most ? wave : most;
  p.by_item = (int64_t)p.c.B * p.c.Hkv * p.blocks <= p.grid;
  prof_before(THD_KERNEL_DECODE, st);
  decode_kernel<kFp8, D, NT><<<(unsigned)p.grid, kDecThreads, S::kSmem, st>>>(p);
  count_launch();
  e = cudaGetLastError();
  prof_after(THD_KERNEL_DECODE, st);
  return e;
}

template <bool kFp8>
static cudaError_t launch_decode_d(DecodeParams& p, int heads, cudaStream_t st) {
  if (p.c.D == 64)
    return heads == 8 ? launch_decode_t<kFp8, 64, 1>(p, st)
                      : heads == 16 ? launch_decode_t<kFp8, 64, 2>(p, st) : launch_decode_t<kFp8, 64, 4>(p, st);
  return heads == 8 ? launch_decode_t<kFp8, 128, 1>(p, st)
                    : heads == 16 ? launch_decode_t<kFp8, 128, 2>(p, st) : launch_decode_t<kFp8, 128, 4>(p, st);
}

cudaError_t launch_decode(DecodeParams p, cudaStream_t st) {
  const int heads = decode_heads(p.G);
  cudaError_t e = p.c.k_exp ? launch_decode_d<true>(p, heads, st) : launch_decode_d<false>(p, heads, st);
  if (e != cudaSuccess) return e;
  if (p.c.capacity > kUnit) {  // an item of one unit is one block's
    const int64_t items = (int64_t)p.c.B * p.c.Hkv * p.blocks;
    // a head a block up to 16; of 32, as many blocks as 16 an SM (most find nothing
    // to do: 304 x 32 of them take 6 us more), each with several heads
    const int64_t x = p.by_item ? items : p.grid, most = 16LL * num_sms() / x > 8 ? 16LL * num_sms() / x : 8;
    const bool several = heads > 16 && most < heads;
    const dim3 grid((unsigned)x, (unsigned)(several ? most : heads));
    prof_before(THD_KERNEL_DECODE_JOIN, st);
    auto* const join = p.c.D == 64 ? (several ? decode_join_kernel<64, true> : decode_join_kernel<64, false>)
                                   : (several ? decode_join_kernel<128, true> : decode_join_kernel<128, false>);
    e = launch_following(join, grid, kJoinThreads, 0, st, (const DecodeParams)p, (int)heads);
    prof_after(THD_KERNEL_DECODE_JOIN, st);
    if (e != cudaSuccess) return e;
  }
  if (p.weight_out) {
    // as many blocks as eight an SM, or the slots, ask for
    const int64_t pairs = (int64_t)p.c.B * p.c.Hkv, run = kWeightThreads * kWeightSlots;
    const int64_t most = (p.c.capacity + run - 1) / run, want = (8LL * num_sms() + pairs - 1) / pairs;
    const int64_t share = most < want ? most : want;
    if (pairs * share >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
    prof_before(THD_KERNEL_DECODE_WEIGHTS, st);
    e = launch_following(decode_weights_kernel, dim3((unsigned)(pairs * share)), kWeightThreads, 0, st, (const DecodeParams)p,
                         (int)share);
    prof_after(THD_KERNEL_DECODE_WEIGHTS, st);
  }
  return e;
}

}  // namespace thd
