// Attention of one new token per sequence over a paged key-value cache
// (thd_attn_decode in the header): per sequence, kv head and run of at most 8, 16 or
// 32 of its query heads one work item, whose slots are read once.
//
// What bounds it: HBM.  A slot's keys and values are 4 D bytes (2 D in e4m3)
// for 4 D G flops, G query heads a kv head: G to 2 G flops a byte, far under what
// the tensor cores need to become the limit, so the products run as warp-level
// matrix instructions (m16n8k16) in which the slots are the 16 rows and the
// query heads the 8 columns: S^T = K q^T, O^T = V^T P^T.  No row of the
// instruction is padding, only heads short of 8 are.
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
// and sum: no barrier between warps until the item's end.
#include <cuda_fp16.h>

#include "cache.cuh"
#include "ptx.cuh"

namespace thd {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecStages = 3;
constexpr int kDecTile = 8192;  // bytes of a stage: a tile's keys, then its values
constexpr int kUnit = 64;       // slots
constexpr int kMinUnits = 2;    // of a block, while there are few

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

int decode_heads(int G) { return G <= 8 ? 8 : G <= 16 ? 16 : 32; }

// ------------------------------------------------------------------ PTX
THD_DEV void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
THD_DEV void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
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
// Two e4m3 numbers (low half) as two fp16, exactly.
THD_DEV uint32_t e4m3x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(x));
  return y;
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
THD_DEV void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
THD_DEV void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// Blocks that share `total` units, and what the c-th of them takes: [c total /
// blocks, (c + 1) total / blocks).
THD_DEV int64_t blocks_for(int64_t total, int grid) {
  const int64_t n = (total + kMinUnits - 1) / kMinUnits;
  return n < grid ? n : grid;
}
THD_DEV int64_t owner_of(int64_t unit, int64_t total, int64_t blocks) { return ((unit + 1) * blocks - 1) / total; }

// ------------------------------------------------------------------ the walk
template <bool kFp8, int D, int NT>
struct DecShape {
  static constexpr int kRow = D * (kFp8 ? 1 : 2);      // bytes
  static constexpr int kKeys = kDecTile / 2 / kRow;    // slots of a tile: 16, 32 or 64
  static constexpr int kSub = kKeys / 16;
  static constexpr int kPieces = kRow / 16;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPitch = D + 4;                 // floats of a head's row in the join of the warps
  // shared memory, bytes
  static constexpr int kRing = kDecStages * kDecTile;  // a warp's
  static constexpr int kMeta = kDecStages * kKeys * 8; // a warp's: exponents and positions
  static constexpr int kQ = D * kHeads * 2;
  static constexpr size_t kSmem = (size_t)kDecWarps * (kRing + kMeta) + kQ + sizeof(float) * (kHeads * (2 + 3 * kDecWarps));
  static_assert(kHeads * kPitch * 4 <= kRing, "a warp's partial fits its ring");
};

// Byte offset of 16-byte piece c of row r in a tile's keys or values: pieces
// are permuted so that eight rows' equal pieces lie in eight different bank
// groups.
template <int kPieces>
THD_DEV uint32_t swz(int r, int c) {
  if (kPieces >= 8) return (uint32_t)(r * kPieces * 16 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * kPieces * 16 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <bool kFp8, int D, int NT>
__global__ void __launch_bounds__(kDecThreads) decode_kernel(const DecodeParams p) {
  using S = DecShape<kFp8, D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_seg[kDecThreads + 1];
  const CacheView& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  grid_dep_launch();
  uint8_t* const ring = smem + warp * S::kRing;
  uint8_t* const meta = smem + kDecWarps * S::kRing + warp * S::kMeta;
  uint8_t* const s_q = smem + kDecWarps * (S::kRing + S::kMeta);
  float* const s_hs = reinterpret_cast<float*>(s_q + S::kQ);  // [kHeads] score multiplier, then slopes
  float* const s_sl = s_hs + S::kHeads;
  float* const s_ml = s_sl + S::kHeads;                       // [kDecWarps][3][kHeads]

  // units in front of each sequence; rows without a visible slot; bad lengths
  const int per = (c.B + kDecThreads - 1) / kDecThreads;
  const int b_lo = tid * per < c.B ? tid * per : c.B, b_hi = b_lo + per < c.B ? b_lo + per : c.B;
  {
    int64_t sum = 0;
    for (int b = b_lo; b < b_hi; ++b) sum += units_of(range_of(p, b));
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
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    bool bad;
    slots_of(c, b, bad);
    if (bad && tid == 0) raise(p.status, THD_DEV_ERR_KV_LEN);
    if (units_of(range_of(p, b)) == 0) {
      for (int i = tid; i < p.Hq * D / 8; i += kDecThreads)
        reinterpret_cast<uint4*>(p.o + (int64_t)b * p.Hq * D)[i] = make_uint4(0, 0, 0, 0);
      for (int h = tid; h < p.Hq; h += kDecThreads) p.lse[(int64_t)h * c.B + b] = -INFINITY;
    }
  }
  if (blockIdx.x == 0) {
    int64_t at_b = s_seg[tid];
    for (int b = b_lo; b < b_hi; ++b) {
      p.units[b] = at_b;
      at_b += units_of(range_of(p, b));
    }
    if (tid == kDecThreads - 1) p.units[c.B] = s_seg[kDecThreads];
  }
  const int HG = c.Hkv * p.blocks;  // items of a sequence
  const int64_t total = s_seg[kDecThreads] * HG;
  const int64_t blocks = blocks_for(total, (int)gridDim.x);
  if (blockIdx.x >= blocks) return;
  int64_t u = blockIdx.x * total / blocks;
  const int64_t u_end = (blockIdx.x + 1) * total / blocks;

  // the first item
  int b, item = 0, i0 = 0;
  {
    const int64_t ub = u / HG;
    int seg = 0;
    for (int step = kDecThreads / 2; step > 0; step >>= 1)
      if (s_seg[seg + step] <= ub) seg += step;
    b = seg * per;
    int64_t before = s_seg[seg];
    for (; b < c.B; ++b) {
      const int n = units_of(range_of(p, b));
      if (ub < before + n) {
        const int64_t r = u - before * HG;
        item = (int)(r / n);
        i0 = (int)(r % n);
        break;
      }
      before += n;
    }
  }

  const uint32_t ps = (uint32_t)c.page_size;
  const uint32_t ring_a = smem_u32(ring);
  while (u < u_end && b < c.B) {
    const Range rg = range_of(p, b);
    const int units = units_of(rg);
    const int64_t take64 = u_end - u;
    const int take = take64 < units - i0 ? (int)take64 : units - i0;
    const int g = item / p.blocks, h0 = (item % p.blocks) * S::kHeads;  // kv head; first query head of its group
    const int heads = p.G - h0 < S::kHeads ? p.G - h0 : S::kHeads;
    const int k0 = rg.s + i0 * kUnit;
    const int k1 = rg.n - k0 < take * kUnit ? rg.n : k0 + take * kUnit;
    const int tiles = (k1 - k0 + S::kKeys - 1) / S::kKeys;
    const int seen = p.slopes ? (p.seen ? p.seen[b] : rg.n) : 0;

    // ---- a tile's copies
    constexpr int kRpl = S::kKeys > 32 ? S::kKeys / 32 : 1;  // rows a lane finds the place of
    int pid[kRpl];
    uint32_t pend[kRpl];  // exponents on their way to shared memory
    int pend_stage = -1;
    auto fetch_pid = [&](int t) {
#pragma unroll
      for (int r = 0; r < kRpl; ++r) {
        const int row = lane + 32 * r, j = k0 + t * S::kKeys + row;
        pid[r] = row < S::kKeys && j < k1 ? c.table[b * c.table_stride + (uint32_t)j / ps] : 0;
      }
    };
    auto flush = [&]() {
      if (kFp8 && pend_stage >= 0) {
#pragma unroll
        for (int r = 0; r < kRpl; ++r)
          if (lane + 32 * r < S::kKeys)
            reinterpret_cast<uint32_t*>(meta)[pend_stage * 2 * S::kKeys + lane + 32 * r] = pend[r];
      }
      pend_stage = -1;
    };
    auto issue = [&](int t, int stage) {
      int64_t off[kRpl];
#pragma unroll
      for (int r = 0; r < kRpl; ++r) {
        const int row = lane + 32 * r, j = k0 + t * S::kKeys + row;
        off[r] = -1;
        pend[r] = 127u | 127u << 8;
        if (row < S::kKeys && j < k1) {
          const uint32_t slot = (uint32_t)j % ps;
          if (pid[r] < 0 || pid[r] >= c.num_pages) {
            raise(p.status, THD_DEV_ERR_PAGE);
          } else {
            off[r] = at(c.row, pid[r], slot, g);
            if (kFp8) {
              const int64_t e = at(c.exp, pid[r], slot, g);
              pend[r] = (uint32_t)c.k_exp[e] | (uint32_t)c.v_exp[e] << 8;
            }
            if (p.pos)
              cp_async_4(smem_u32(meta) + (stage * 2 * S::kKeys + S::kKeys + row) * 4, p.pos + at(p.pos_at, pid[r], slot, g));
          }
        }
      }
      const uint32_t dst = ring_a + stage * kDecTile;
      constexpr int kRowsPer = 32 / S::kPieces;  // rows of one warp-wide copy
      const int piece = lane % S::kPieces;
#pragma unroll
      for (int i = 0; i < S::kKeys / kRowsPer; ++i) {
        const int row = i * kRowsPer + lane / S::kPieces;
        const int64_t o = __shfl_sync(0xffffffffu, off[kRpl > 1 ? (i * kRowsPer) / 32 : 0], row & 31);
        const uint32_t a = dst + swz<S::kPieces>(row, piece);
        const int64_t from = o < 0 ? 0 : o + 16 * piece;
        cp_async_16(a, c.k + from, o < 0 ? 0 : 16);
        cp_async_16(a + kDecTile / 2, c.v + from, o < 0 ? 0 : 16);
      }
      pend_stage = stage;
    };

    // ---- the first copies, then the queries, which all warps share
    fetch_pid(warp);
#pragma unroll
    for (int s = 0; s < kDecStages - 1; ++s) {
      const int t = warp + s * kDecWarps;
      flush();
      if (t < tiles) {
        issue(t, s);
        fetch_pid(t + kDecWarps);
      }
      cp_commit();
    }
    for (int n = warp; n < S::kHeads; n += kDecWarps) {
      constexpr int kPairs = D / 64;  // of a lane
      uint32_t w[kPairs];
#pragma unroll
      for (int k = 0; k < kPairs; ++k)
        w[k] = n < heads ? reinterpret_cast<const uint32_t*>(p.q + b * p.q_stride + (int64_t)(g * p.G + h0 + n) * D)[lane + 32 * k] : 0u;
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
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          const float lo = __uint_as_float(w[k] << 16) * m1 * m2, hi = __uint_as_float(w[k] & 0xffff0000u) * m1 * m2;
          w[k] = pack2<true>(lo, hi);
        }
      }
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        const int d = 2 * (lane + 32 * k), ks = d >> 4, in = d & 15;
        // fragment order of the matrix instruction's second operand; the e4m3
        // form counts the elements of a step as its keys' bytes arrive
        const int reg = kFp8 ? (in & 3) >> 1 : in >> 3, quad = kFp8 ? in >> 2 : (in & 7) >> 1;
        *reinterpret_cast<uint32_t*>(s_q + ((((ks * NT + (n >> 3)) * 32 + (n & 7) * 4 + quad) * 2 + reg) * 4)) = w[k];
      }
      if (lane == 0) {
        s_hs[n] = mul * (p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e);
        s_sl[n] = p.slopes && n < heads ? p.slopes[g * p.G + h0 + n] * kLog2e : 0.f;
      }
    }
    __syncthreads();
    float hs[NT][2], sl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) hs[nt][e] = s_hs[nt * 8 + 2 * t4 + e], sl[nt][e] = s_sl[nt * 8 + 2 * t4 + e];

    // ---- tiles: running maximum (base 2) m and sum l of each head, O^T
    // mo: the maximum of score + log2 of the value's scale, what O is relative to
    float m[NT][2], mo[NT][2], l[NT][2], o[D / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nt][e] = mo[nt][e] = -INFINITY, l[nt][e] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][nt][e] = 0.f;

    int stage = 0;
    for (int t = warp; t < tiles; t += kDecWarps) {
      cp_wait<kDecStages - 2>();
      __syncwarp();
      const uint32_t kt = ring_a + stage * kDecTile, vt = kt + kDecTile / 2;
      const uint32_t* const mt = reinterpret_cast<const uint32_t*>(meta) + stage * 2 * S::kKeys;
      float s[S::kSub][NT][4];
#pragma unroll
      for (int sub = 0; sub < S::kSub; ++sub)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[sub][nt][e] = 0.f;
      // lanes' rows and pieces of the four 8x8 matrices of a load: rows 0-7 and
      // 8-15 of the first 16 bytes, then of the second
      const int lrow = lane & 15, lpc = lane >> 4;
#pragma unroll
      for (int kp = 0; kp < S::kPieces / 2; ++kp) {
        constexpr int kSteps = kFp8 ? 2 : 1;  // steps of 16 elements in 32 bytes
        uint2 bq[kSteps][NT];
#pragma unroll
        for (int x = 0; x < kSteps; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            bq[x][nt] = *reinterpret_cast<const uint2*>(s_q + (((kp * kSteps + x) * NT + nt) * 32 + lane) * 8);
#pragma unroll
        for (int sub = 0; sub < S::kSub; ++sub) {
          uint32_t r[4];
          ldsm4(r, kt + swz<S::kPieces>(sub * 16 + lrow, 2 * kp + lpc));
          if (kFp8) {
            const uint32_t a0[4] = {e4m3x2(r[0]), e4m3x2(r[1]), e4m3x2(r[0] >> 16), e4m3x2(r[1] >> 16)};
            const uint32_t a1[4] = {e4m3x2(r[2]), e4m3x2(r[3]), e4m3x2(r[2] >> 16), e4m3x2(r[3] >> 16)};
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
      const int j0 = k0 + t * S::kKeys;
      float lv[S::kSub][2];  // log2 of the values' scales
      float mx[NT][2], mxo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[nt][e] = mxo[nt][e] = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < S::kSub; ++sub)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = sub * 16 + half * 8 + gid, j = j0 + row;
          const bool ok = j < k1;
          float ksc = 1.f, far = 0.f;
          if (kFp8) {
            const uint32_t e = mt[row];
            ksc = scale_of(e & 0xffu);
            lv[sub][half] = (e >> 8) == 255u ? NAN : (float)((int)(e >> 8) - 127);
          }
          if (p.slopes) far = (float)(int)((uint32_t)seen - 1u - (p.pos ? mt[S::kKeys + row] : (uint32_t)j));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[e] = s[sub][nt][2 * half + e] * hs[nt][e];
              if (kFp8) y[e] *= ksc;
              if (p.cap > 0.f) y[e] = p.cap * kLog2e * tanhf(y[e]);
              if (p.slopes) y[e] = fmaf(-sl[nt][e], far, y[e]);
              y[e] = ok ? y[e] : -INFINITY;
              s[sub][nt][2 * half + e] = y[e];
              mx[nt][e] = fmaxf(mx[nt][e], y[e]);
              if (kFp8) mxo[nt][e] = fmaxf(mxo[nt][e], y[e] + lv[sub][half]);
            }
            if (p.weight_out && j < k1) {
              float* const to = p.scores + (((int64_t)b * c.Hkv + g) * c.capacity + j) * p.G + h0 + nt * 8 + 2 * t4;
              if (nt * 8 + 2 * t4 < heads) to[0] = y[0];
              if (nt * 8 + 2 * t4 + 1 < heads) to[1] = y[1];
            }
          }
        }
      bool moved = false;
      float al[NT][2], alo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], d));
            if (kFp8) mxo[nt][e] = fmaxf(mxo[nt][e], __shfl_xor_sync(0xffffffffu, mxo[nt][e], d));
          }
          const float m2 = fmaxf(m[nt][e], mx[nt][e]);
          moved |= m2 > m[nt][e];
          al[nt][e] = m2 > m[nt][e] ? ex2(m[nt][e] - m2) : 1.f;
          m[nt][e] = m2;
          if (kFp8) {
            const float o2 = fmaxf(mo[nt][e], mxo[nt][e]);
            moved |= o2 > mo[nt][e];
            alo[nt][e] = o2 > mo[nt][e] ? ex2(mo[nt][e] - o2) : 1.f;
            mo[nt][e] = o2;
          } else {
            alo[nt][e] = al[nt][e];
            mo[nt][e] = m2;
          }
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l[nt][0] *= al[nt][0];
          l[nt][1] *= al[nt][1];
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            o[d][nt][0] *= alo[nt][0];
            o[d][nt][1] *= alo[nt][1];
            o[d][nt][2] *= alo[nt][0];
            o[d][nt][3] *= alo[nt][1];
          }
        }
      }
      // probabilities: summed in fp32, rounded to 16 bits (bf16 next to bf16
      // values, fp16 next to e4m3) for the product, as the packed kernels do
      uint32_t pb[S::kSub][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float base[2], baseo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          base[e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
          baseo[e] = mo[nt][e] == -INFINITY ? 0.f : mo[nt][e];
        }
#pragma unroll
        for (int sub = 0; sub < S::kSub; ++sub)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float y = s[sub][nt][2 * half + e];
              w[e] = ex2(y - base[e]);
              l[nt][e] += w[e];
              if (kFp8) w[e] = ex2(y + lv[sub][half] - baseo[e]);
            }
            pb[sub][nt][half] = movm_t(pack2<kFp8>(w[0], w[1]));
          }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int dp = 0; dp < S::kPieces / 2; ++dp)
#pragma unroll
        for (int sub = 0; sub < S::kSub; ++sub) {
          uint32_t r[4];
          if (kFp8) {
            // matrices: slots 0-7 and 8-15 of 16 elements, then of the next 16;
            // a register has elements 2 gid and 2 gid + 1 of two slots
            ldsm4t(r, vt + swz<S::kPieces>(sub * 16 + lrow, 2 * dp + lpc));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t y0 = __byte_perm(r[2 * x], 0, 0x3120), y1 = __byte_perm(r[2 * x + 1], 0, 0x3120);
              const uint32_t a[4] = {e4m3x2(y0), e4m3x2(y0 >> 16), e4m3x2(y1), e4m3x2(y1 >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(o[(kFp8 ? 2 * dp + x : 0)][nt], a, pb[sub][nt][0], pb[sub][nt][1]);
            }
          } else {
            // matrices: elements 0-7 and 8-15 of slots 0-7, then of slots 8-15
            ldsm4t(r, vt + swz<S::kPieces>(sub * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * dp + ((lane >> 3) & 1)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[dp][nt], r, pb[sub][nt][0], pb[sub][nt][1]);
          }
        }
      __syncwarp();  // the stage is read
      flush();
      const int tn = t + (kDecStages - 1) * kDecWarps;
      if (tn < tiles) {
        int ns = stage + kDecStages - 1;
        ns = ns >= kDecStages ? ns - kDecStages : ns;
        issue(tn, ns);
        fetch_pid(tn + kDecWarps);
      }
      cp_commit();
      stage = stage + 1 == kDecStages ? 0 : stage + 1;
    }
    cp_wait<0>();

    // ---- the item's end: the warps' sums, then their O, through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        if (gid == 0) {
          float* const to = s_ml + warp * 3 * S::kHeads + nt * 8 + 2 * t4 + e;
          to[0] = mo[nt][e];
          to[S::kHeads] = m[nt][e];
          to[2 * S::kHeads] = l[nt][e];
        }
      }
    __syncthreads();
    float* const mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, s_ml[w * 3 * S::kHeads + nt * 8 + 2 * t4 + e]);
        f[e] = top == -INFINITY ? 1.f : ex2(mo[nt][e] - top);
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at_d = d * 16 + (kFp8 ? 2 * gid + (e >> 1) : gid + 8 * (e >> 1));
          mine[(nt * 8 + 2 * t4 + (e & 1)) * S::kPitch + at_d] = o[d][nt][e] * f[e & 1];
        }
    }
    __syncthreads();
    const bool whole = take == units;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (i0 > 0 ? 0 : 1);
    for (int i = tid; i < heads * (D / 4); i += kDecThreads) {
      const int n = i / (D / 4), d = 4 * (i % (D / 4));
      float top = -INFINITY, topo = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        topo = fmaxf(topo, s_ml[w * 3 * S::kHeads + n]);
        top = fmaxf(top, s_ml[w * 3 * S::kHeads + S::kHeads + n]);
      }
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float mw = s_ml[w * 3 * S::kHeads + S::kHeads + n];
        sum += s_ml[w * 3 * S::kHeads + 2 * S::kHeads + n] * (top == -INFINITY ? 1.f : ex2(mw - top));
      }
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(smem + w * S::kRing + (n * S::kPitch + d) * 4);
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
    // on to the next item
    u += take;
    i0 = 0;
    if (u < u_end && ++item == HG) {
      item = 0;
      do ++b;
      while (b < c.B && units_of(range_of(p, b)) == 0);
    }
    __syncthreads();  // the rings are read
  }
}

// ------------------------------------------------------------------ the join
// The parts of the items that several blocks shared, a block for each (sequence,
// query head); behind them, blocks that turn the scores into weights.
constexpr int kJoinThreads = 256;

THD_DEV float joined_lse2(const DecodeParams& p, int64_t u0, int64_t u1, int64_t total, int64_t blocks, int kheads, int n,
                          int lane) {
  const int64_t c0 = owner_of(u0, total, blocks), c1 = owner_of(u1 - 1, total, blocks);
  float top = -INFINITY;
  for (int64_t x = c0 + lane; x <= c1; x += 32)
    top = fmaxf(top, p.part_ml[((2 * x + (x * total / blocks > u0 ? 0 : 1)) * kheads + n) * 3 + 1]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int64_t x = c0 + lane; x <= c1; x += 32) {
    const float* ml = p.part_ml + ((2 * x + (x * total / blocks > u0 ? 0 : 1)) * kheads + n) * 3;
    sum += ml[2] * ex2(ml[1] - base);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return base + log2f(sum);
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeParams p, int kheads, int weight_blocks) {
  constexpr int kLanes = D / 4, kParts = kJoinThreads / kLanes;
  __shared__ float4 s_x[kJoinThreads];
  __shared__ float s_lse[kDecodeMaxGroup];
  const CacheView& c = p.c;
  const int tid = threadIdx.x;
  grid_dep_wait();
  const int HG = c.Hkv * p.blocks;
  const int64_t total = p.units[c.B] * HG;
  if (total == 0) return;
  const int64_t blocks = blocks_for(total, p.grid);
  const int64_t joins = (int64_t)c.B * p.Hq;
  if (blockIdx.x < joins) {
    const int b = (int)(blockIdx.x / p.Hq), h = (int)(blockIdx.x % p.Hq);
    const int g = h / p.G, n = (h % p.G) % kheads, item = g * p.blocks + (h % p.G) / kheads;
    const int64_t units = p.units[b + 1] - p.units[b];
    const int64_t u0 = p.units[b] * HG + item * units, u1 = u0 + units;
    if (units == 0) return;
    const int64_t c0 = owner_of(u0, total, blocks), c1 = owner_of(u1 - 1, total, blocks);
    if (c0 == c1) return;  // one block's: written
    const int lane = tid % kLanes, mine = tid / kLanes;
    float topo = -INFINITY, top = -INFINITY;
    for (int64_t x = c0; x <= c1; ++x) {
      const float* ml = p.part_ml + ((2 * x + (x * total / blocks > u0 ? 0 : 1)) * kheads + n) * 3;
      topo = fmaxf(topo, ml[0]);
      top = fmaxf(top, ml[1]);
    }
    const float base = top == -INFINITY ? 0.f : top, baseo = topo == -INFINITY ? 0.f : topo;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int64_t x = c0 + mine; x <= c1; x += kParts) {
      const int64_t slot = (2 * x + (x * total / blocks > u0 ? 0 : 1)) * kheads + n;
      const float* ml = p.part_ml + slot * 3;
      const float4 y = *reinterpret_cast<const float4*>(p.part + slot * D + 4 * lane);
      const float f = ex2(ml[0] - baseo);
      sum += ml[2] * ex2(ml[1] - base);
      acc.x += y.x * f, acc.y += y.y * f, acc.z += y.z * f, acc.w += y.w * f;
    }
    __shared__ float s_sum[kParts];
    s_x[tid] = acc;
    if (lane == 0) s_sum[mine] = sum;
    __syncthreads();
    if (tid < kLanes) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float s = 0.f;
      for (int k = 0; k < kParts; ++k) {
        const float4 y = s_x[k * kLanes + tid];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        s += s_sum[k];
      }
      const float f = s == 0.f ? 0.f : ex2(baseo - base) / s;
      uint2 y;
      y.x = pack2<false>(x.x * f, x.y * f);
      y.y = pack2<false>(x.z * f, x.w * f);
      *reinterpret_cast<uint2*>(p.o + ((int64_t)b * p.Hq + h) * D + 4 * tid) = y;
      if (tid == 0) p.lse[(int64_t)h * c.B + b] = (base + log2f(s)) * kLn2;
    }
    return;
  }
  // weights: the units of (sequence, kv head) pairs, cut evenly
  const int64_t w = blockIdx.x - joins, all = p.units[c.B] * c.Hkv;
  int64_t u = w * all / weight_blocks;
  const int64_t u_end = (w + 1) * all / weight_blocks;
  while (u < u_end) {
    const int64_t ub = u / c.Hkv;
    int lo = 0, hi = c.B - 1;  // the sequence: the last with units in front of it <= ub, and units of its own
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.units[mid] <= ub) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const int64_t units = p.units[b + 1] - p.units[b], r = u - p.units[b] * c.Hkv;
    const int g = (int)(r / units);
    const int64_t i0 = r % units;
    const int64_t take = u_end - u < units - i0 ? u_end - u : units - i0;
    for (int n = tid >> 5; n < p.G; n += kJoinThreads / 32) {
      const int item = g * p.blocks + n / kheads;
      const int64_t v0 = p.units[b] * HG + item * units;
      float z;
      if (owner_of(v0, total, blocks) == owner_of(v0 + units - 1, total, blocks))
        z = p.lse2[(int64_t)b * p.Hq + g * p.G + n];
      else
        z = joined_lse2(p, v0, v0 + units, total, blocks, kheads, n % kheads, tid & 31);
      if ((tid & 31) == 0) s_lse[n] = z == -INFINITY ? INFINITY : z;
    }
    __syncthreads();
    const Range rg = range_of(p, b);
    const int k0 = rg.s + (int)i0 * kUnit;
    const int k1 = rg.n - k0 < take * kUnit ? rg.n : k0 + (int)take * kUnit;
    for (int j = k0 + tid; j < k1; j += kJoinThreads) {
      const int page = page_of(c, b, (uint32_t)j / (uint32_t)c.page_size);
      if (page < 0) continue;
      const float* s = p.scores + (((int64_t)b * c.Hkv + g) * c.capacity + j) * p.G;
      float x = 0.f;
      for (int n = 0; n < p.G; ++n) x += ex2(s[n] - s_lse[n]);
      const int64_t a = at(p.weight_at, page, (uint32_t)j % (uint32_t)c.page_size, g);
      p.weight_out[a] = p.weight_in[a] + x;
    }
    __syncthreads();
    u += take;
  }
}

// ------------------------------------------------------------------ launch
template <bool kFp8, int D, int NT>
static cudaError_t launch_decode_t(const DecodeParams& p, cudaStream_t st) {
  using S = DecShape<kFp8, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<kFp8, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  if (e != cudaSuccess) return e;
  prof_before(THD_KERNEL_DECODE, st);
  decode_kernel<kFp8, D, NT><<<p.grid, kDecThreads, S::kSmem, st>>>(p);
  count_launch();
  e = cudaGetLastError();
  prof_after(THD_KERNEL_DECODE, st);
  return e;
}

template <bool kFp8>
static cudaError_t launch_decode_d(const DecodeParams& p, int heads, cudaStream_t st) {
  if (p.c.D == 64)
    return heads == 8 ? launch_decode_t<kFp8, 64, 1>(p, st)
                      : heads == 16 ? launch_decode_t<kFp8, 64, 2>(p, st) : launch_decode_t<kFp8, 64, 4>(p, st);
  return heads == 8 ? launch_decode_t<kFp8, 128, 1>(p, st)
                    : heads == 16 ? launch_decode_t<kFp8, 128, 2>(p, st) : launch_decode_t<kFp8, 128, 4>(p, st);
}

cudaError_t launch_decode(DecodeParams p, cudaStream_t st) {
  const int heads = decode_heads(p.G);
  int64_t grid = 2LL * num_sms();  // two blocks an SM, one wave
  if (grid > kDecodeMaxGrid) grid = kDecodeMaxGrid;
  p.grid = (int)grid;
  cudaError_t e = p.c.k_exp ? launch_decode_d<true>(p, heads, st) : launch_decode_d<false>(p, heads, st);
  if (e != cudaSuccess) return e;
  // an item of one unit is one block's, and without weights nothing is left to do
  if (p.c.capacity <= kUnit && !p.weight_out) return cudaSuccess;
  const int wb = p.weight_out ? 4 * num_sms() : 0;
  const int64_t joins = (int64_t)p.c.B * p.Hq;
  if (joins + wb >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(joins + wb));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_before(THD_KERNEL_DECODE_JOIN, st);
  e = p.c.D == 64 ? cudaLaunchKernelEx(&cfg, decode_join_kernel<64>, p, heads, wb)
                  : cudaLaunchKernelEx(&cfg, decode_join_kernel<128>, p, heads, wb);
  count_launch();
  prof_after(THD_KERNEL_DECODE_JOIN, st);
  return e;
}

}  // namespace thd
