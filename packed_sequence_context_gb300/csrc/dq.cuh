// dQ of attention over packed THD tensors, query-stationary, walked in the
// same P2P ring order as the forward and executed for every emulated rank on
// one GB300.
//
// [P2] TransformerEngine issue #3487 ("Steps/Code to reproduce bug": BF16
// attention backward on this layout with four-rank P2P context parallelism;
// "Describe the bug": THD dQ tail-zeroing).  [P1] TransformerEngine issue
// #2208 (traceback through AttnFuncWithCPAndKVP2P): at ring step i rank r
// holds the KV of rank s = (r - i) mod cp and accumulates its dQ partial from
// it.  The key/value-stationary kernel produces dK and dV; this one recomputes
// S and dP for its own query tile and keeps dQ on chip for the whole walk, so
// dQ needs no atomics and no fp32 accumulator in global memory.
//
// One work item = (rank r, sequence b, query head h, rank-local 128-row query
// tile t), the forward's schedule.  For each key tile (chunk c, tile j) the
// item visits:
//   S  = Q K^T   (TMEM S buffer g % 2)     dP = dO V^T   (TMEM dP, released
//                                           as soon as the dS warps hold it)
//   P  = 2^(S scale log2(e) - lse log2(e))  dS = P (dP - Delta)  -> bf16 into S
//   dQ += dS K   (A = dS from TMEM, B = the K tile read MN-major)
// and dQ * scale is written as bf16 at the end of the item.
//
// Scored attention, Delta: rowsum(dO O) comes from O in bf16, an error of up to
// 2^-9 |dO| |O| that dS = P (dP - Delta) takes over whole; it shows in rows whose
// weight lies on a few keys, most where dP - Delta itself is nearly 0.  The row
// sum off of P (dP - Delta), which is 0 for the exact Delta, corrects it: every
// item adds it up and leaves the exact Delta for the dK/dV kernel.  For dQ itself:
// heads of 64 leave room in TMEM for M = sum of P (1 - tanh^2) K, one product more
// a tile, and dQ - off M is exact in every row (32,768 tokens of 16 + 4 heads:
// masks 3.2 -> 4.15 ms, bias 4.0 -> 4.95, cap 4.55 -> 5.0, and without the walks
// below cap and bias 5.9 -> 5.6).  Heads of 128 leave none; there an
// item walks the keys of rows that see few of them a first time, for Delta alone:
// those of short walks and of documents that begin or end inside its tile
// (few_keys), or all of its keys where the head's slope is at least kSteepSlope
// either way.
// Others keep Delta from O, as plain attention does for every row: a walk for
// Delta takes two thirds of dQ's time again, and how far the scores themselves
// gather a row's weight is only known after it.  From kSteepSlope on Delta's
// error outgrows that of dS's own rounding.  Emulated against fp64, 512 rows
// behind 512 keys, D = 128: relative error of dQ, and of its worst row, with Delta
// from O (corrected it is 2.4e-3 and 0.4% in every line):
//   no bias 2.4e-3, 0.4%; slope 1/32 2.5e-3, 1.7%; 1/8 3.0e-3, 4%; 1/4 3.0e-3,
//   7%; 3/8 3.3e-3, 6%; 0.7 4.0e-3, 40%; 2 6.0e-3, 8 times the row's norm
//   documents of 512 rows 2.6e-3, 1%; 64 3.0e-3, 8%; 8 3.9e-3, the row's norm
//   scores of standard deviation 3 under a cap 3.1e-3, 58%; 6 4.2e-3, 3 times
// (the worst rows' gradients are nearly 0: their weight lies on one key).
// What the walk for steep slopes costs: 12 padded sequences of 154 to 1409, 5 of
// 32 heads, dQ 268 -> 291 us.
//
// CTA layout (one CTA per SM, persistent over the schedule): the dS warps, then
// four warps with a role each.
//   dS warps  two warpgroups (384 threads in all), with a cap or a bias four (640):
//             thread = query row, a half (quarter) of the key columns; and the
//             dQ epilogue (as much of the head dimension)
//   role 0    producer: gathers the item's Q and dO rows (cp.async) and
//             issues the K tile TMA loads into a 3-slot ring
//   role 1    TMEM allocator, S = Q K^T and dQ += dS K issuer (one thread)
//   role 2    producer of the V tiles (2-slot ring)
//   role 3    dP = dO V^T issuer (one thread)
// TMEM: S buffers [0,128) and [128,256), dP [256,384), dQ [384, 384+D).  A K
// slot is read by S of its tile and by dQ of that tile, so it frees after the
// dQ product; S buffer b is overwritten by an S issued after the dQ that read
// its dS, by the same thread (the tensor pipe runs one thread's MMAs in issue
// order).
//
// 32,768 tokens, 16 + 4 heads of 128: plain 3.8 ms (1741 TFLOPS of the three
// products), masks 3.75, cap 50 4.9 (1336), every score saturated 5.8; with the two
// walks of 2 of the 16 heads, bias 4.4, cap and bias 6.05.  The row sum of
// P (dP - Delta) is 4% of that.  Two warpgroups against four (before the
// row sum, and before sequences were walked as a whole): cap 5.1 / 4.6, cap and
// bias 6.2 / 5.2; bias alone, padded batch of 154 to 1409, 520 / 486 us,
// sequences of 256 164 / 170; masks alone, 32,768 tokens, 3.8 / 4.0 ms.  With a
// cap the tensor pipe is 59% busy and the schedulers issue in 65% of the cycles.
// 32,768 tokens in sequences of 256 (keys walked twice): masks 260 us, cap 317; of
// 512 246 and 320.
#pragma once

#include "common.cuh"
#include "ptx.cuh"
#include "sched.cuh"
#include "score.cuh"

namespace thd {

template <int D, int kMod>
struct DqCfg {
  static constexpr int kKStages = 3;
  static constexpr int kVStages = 2;
  static constexpr int kQBytes = kTile * D * 2;  // one [128, D] bf16 tile
  static constexpr int kKVBytes = kTile * D * 2;
  static constexpr int kSmem = 1024 + 2 * kQBytes + (kKStages + kVStages) * kKVBytes;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColDP = 256, kColDQ = 384;
  // scored, where TMEM has room for it: M = sum of P (1 - tanh^2) K beside dQ
  static constexpr bool kMass = kMod != 0 && D == 64;
  static constexpr uint32_t kColM = kColDQ + D;
  // dS warpgroups: two, each with half of the columns of a tile; four with a
  // quarter each where a cap or a bias makes dS long enough for its latencies
  // to show (two warps per scheduler, in step, left it idle half of the time)
  static constexpr int kGroups = (kMod & (kModCap | kModDist)) != 0 ? 4 : 2;
  static constexpr int kWarps = 4 * kGroups;  // dS warps; the four others follow
  static constexpr int kThreads = 32 * kWarps + 128;
  // where packed dS of key columns 16 ks.. sits in the S buffer: inside the S
  // columns of the warpgroup that writes it (another may still be reading its own)
  __host__ __device__ static constexpr uint32_t ds_col(int ks) {
    return kGroups == 2 ? 64 * (ks >> 2) + 8 * (ks & 3) : 32 * (ks >> 1) + 8 * (ks & 1);
  }
  static constexpr uint32_t kMassOff = kGroups == 2 ? 32 : 16;  // packed P (1 - tanh^2) beside it
  // register split (setmaxnreg) for the instantiation shorter sequences take:
  // dQ +2-3% on batches of 0.1-8K-token sequences, -0.9% on one long sequence
  static constexpr uint32_t kLaunchRegs = kGroups == 2 ? 168 : 96;   // per thread, what 65,536 allow
  static constexpr uint32_t kComputeRegs = kGroups == 2 ? 192 : 104;  // per thread, dS warps
  static constexpr uint32_t kOtherRegs = kGroups == 2 ? 112 : 64;     // per thread, the others
  static_assert(32 * kWarps * kComputeRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
                "register split above the launch budget");
};

// An item's walks over its keys: the first one's, and whether it is the last (the
// one that makes dQ, over all of them; else it is for Delta alone, see above).
constexpr float kSteepSlope = 0.375f;
__device__ inline int2 all_keys(const QItem& it) { return make_int2(it.k_lo, it.k_hi); }
template <int D, int kMod>
__device__ inline int2 first_keys(const DqParams& p, const QItem& it, bool& last) {
  last = true;
  if constexpr (kMod == 0) return make_int2(0, 0);
  if constexpr (DqCfg<D, kMod>::kMass) return all_keys(it);
  int2 k = make_int2(it.few_lo, it.few_hi);
  if constexpr ((kMod & kModDist) != 0)
    if (fabsf(p.mods.slopes[it.h]) >= kSteepSlope) k = all_keys(it);
  last = k.x >= k.y;
  return last ? all_keys(it) : k;
}

template <int D, bool kGrouped, int kMod>
__global__ void __launch_bounds__((DqCfg<D, kMod>::kThreads), 1)
    dq_kernel(const DqParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = DqCfg<D, kMod>;
  // the register split also carries the longer dS of a score function
  constexpr bool kSplit = !kGrouped || C::kGroups == 4;
  constexpr int KS = C::kKStages, VS = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sDO = smem + C::kQBytes;
  uint8_t* sK = smem + 2 * C::kQBytes;
  uint8_t* sV = sK + KS * C::kKVBytes;
  __shared__ __align__(8) uint64_t bar_k_full[KS];
  __shared__ __align__(8) uint64_t bar_k_empty[KS];
  __shared__ __align__(8) uint64_t bar_v_full[VS];
  __shared__ __align__(8) uint64_t bar_v_empty[VS];
  __shared__ __align__(8) uint64_t bar_s_full[2];
  __shared__ __align__(8) uint64_t bar_ds_ready[2];
  __shared__ __align__(8) uint64_t bar_dp_full;
  __shared__ __align__(8) uint64_t bar_dp_free;  // the dS warps have read dP into registers
  __shared__ __align__(8) uint64_t bar_q_full;
  __shared__ __align__(8) uint64_t bar_q_empty;
  __shared__ __align__(8) uint64_t bar_dq_done;
  __shared__ __align__(8) uint64_t bar_eps[4];  // scored: the dS warps of one quarter of the rows
  __shared__ float s_eps[kMod != 0 ? C::kGroups - 1 : 1][kMod != 0 ? kTile : 1];
  __shared__ __align__(8) uint64_t bar_drain;
  __shared__ __align__(8) uint64_t bar_drain2;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ ItemRing ring;  // items handed out to this CTA, in claim order

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int role = warp - C::kWarps;  // of the four warps after the dS warps: 0 Q, dO, K; 1 S, dQ; 2 V; 3 dP
  if (*p.dev_status != 0) return;  // metadata rejected: outputs untouched
  const int n_entries = p.counters[0];
  const int n_items = n_entries * p.Hq;

  if (tid == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&bar_k_full[s], 1);
      mbar_init(&bar_k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&bar_v_full[s], 1);
      mbar_init(&bar_v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar_s_full[s], 1);
      mbar_init(&bar_ds_ready[s], C::kWarps);  // one arrival per dS warp
    }
    mbar_init(&bar_dp_full, 1);
    mbar_init(&bar_dp_free, C::kWarps);  // one arrival per dS warp
    mbar_init(&bar_q_full, 32);
    mbar_init(&bar_q_empty, 2);  // the S issuer's last read of Q and the dP issuer's last read of dO
    mbar_init(&bar_dq_done, 1);
    for (int s = 0; s < 4; ++s) mbar_init(&bar_eps[s], C::kGroups);
    mbar_init(&bar_drain, 1);
    mbar_init(&bar_drain2, 1);
    item_ring_init(&ring, 3 + C::kWarps);  // warps 9, 10, 11 (one thread each) and the dS warps
    s_abort = 0;
    fence_mbar_init();
  }
  if (role == 1) {
    tmem_alloc(&s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (role == 0 && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Test hook (thd_test_arm_stall): every thread waits on a barrier nothing
  // completes, so the bounded wait runs out, the CTA takes the abort path
  // before any copy or MMA is issued, frees its TMEM and reports
  // THD_ERR_TIMEOUT.  The drain barrier is free for this: in this mode no
  // role runs, so nothing ever commits to it.
  if (p.test_stall) {
    mbar_wait(&bar_drain, 0, &s_abort);
  } else if (role >= 0) {
    if constexpr (kSplit) regs_lower<C::kOtherRegs>();
    if (role == 0) {
      // ------------------------------------------------------------ Q, dO and K producer (whole warp)
      int ks = 0;
      uint32_t kph = 0, n_fill = 0, q_iter = 0;
      bool ok = true;
      int w = item_first();
      for (uint32_t kit = 0; ok; ++kit) {
        // publish this item (or the end marker) to the other roles, and claim
        // the next one while this one is loaded
        int wnext = 0;
        if (lane == 0) {
          ok = item_publish(&ring, kit, w, &s_abort);
          if (ok && w < n_items) wnext = item_claim(p.claim);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok || w >= n_items) break;
        const QItem it = q_item<kGrouped, kMod>(p, n_entries, w);
        // the item's rank-local query rows of Q and dO, once the previous
        // item's last products that read them have completed; rows without a
        // valid query are zero
        if (!mbar_wait(&bar_q_empty, (q_iter & 1u) ^ 1u, &s_abort)) break;
        const uint32_t qdst = smem_u32(sQ), ddst = smem_u32(sDO);
#pragma unroll
        for (int rr = 0; rr < 4; ++rr) {
          const int row = lane + 32 * rr;
          const int prow = it.t * kTile + row;
          const bool in_rank = prow < rank_rows<kMod>(it.g);
          const int pos = in_rank ? local_to_pos(prow, it.r, it.g.cbq, p.cp) : 0;
          const bool valid = in_rank && pos < it.g.Lq;
          const int64_t off = valid ? (((int64_t)it.g.q_off + pos) * p.Hq + it.h) * D : 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            cp_async_16(qdst + sw128_offset(row, 8 * c, kTile), p.q + off + (valid ? 8 * c : 0), valid ? 16u : 0u);
            cp_async_16(ddst + sw128_offset(row, 8 * c, kTile), p.dout + off + (valid ? 8 * c : 0), valid ? 16u : 0u);
          }
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
        mbar_arrive(&bar_q_full);
        ++q_iter;
        bool last;
        for (int2 keys = first_keys<D, kMod>(p, it, last);; keys = all_keys(it), last = true) {
          for_each_kv_tile<kMod>(it, p, keys, [&](int c, int j) {
            if (!ok) return;
            if (!mbar_wait(&bar_k_empty[ks], kph ^ 1u, &s_abort)) {
              ok = false;
              return;
            }
            if (lane == 0) {
              const int row = it.g.kv_off + c * it.g.cbkv + j * kTile;
              mbar_arrive_expect_tx(&bar_k_full[ks], C::kKVBytes);
#pragma unroll
              for (int hb = 0; hb < D / 64; ++hb)
                tma_load_3d(smem_u32(sK + ks * C::kKVBytes + hb * 16384), &tmK, &bar_k_full[ks], hb * 64, it.kvh, row);
            }
            ++n_fill;
            if (++ks == KS) {
              ks = 0;
              kph ^= 1u;
            }
          });
          if (last) break;
        }
        w = __shfl_sync(0xffffffffu, wnext, 0);
      }
      if (lane == 0) {
        for (int s = 0; s < KS; ++s) {
          const uint32_t fills = n_fill > (uint32_t)s ? (n_fill - 1 - s) / KS + 1 : 0;
          if (fills > 0) drain_wait(&bar_k_full[s], (fills - 1) & 1u);
        }
      }
      __syncwarp();
    } else if (role == 2) {
      // ------------------------------------------------------------ value producer
      if (lane == 0) {
        int vs = 0;
        uint32_t vph = 0, n_fill = 0;
        bool ok = true;
        for (uint32_t kit = 0; ok; ++kit) {
          int w;
          if (!item_take_one(&ring, kit, w, &s_abort) || w >= n_items) break;
          const QItem it = q_item<kGrouped, kMod>(p, n_entries, w);
          bool last;
          for (int2 keys = first_keys<D, kMod>(p, it, last);; keys = all_keys(it), last = true) {
            for_each_kv_tile<kMod>(it, p, keys, [&](int c, int j) {
              if (!ok) return;
              if (!mbar_wait(&bar_v_empty[vs], vph ^ 1u, &s_abort)) {
                ok = false;
                return;
              }
              const int row = it.g.kv_off + c * it.g.cbkv + j * kTile;
              mbar_arrive_expect_tx(&bar_v_full[vs], C::kKVBytes);
#pragma unroll
              for (int hb = 0; hb < D / 64; ++hb)
                tma_load_3d(smem_u32(sV + vs * C::kKVBytes + hb * 16384), &tmV, &bar_v_full[vs], hb * 64, it.kvh, row);
              ++n_fill;
              if (++vs == VS) {
                vs = 0;
                vph ^= 1u;
              }
            });
            if (last) break;
          }
        }
        for (int s = 0; s < VS; ++s) {
          const uint32_t fills = n_fill > (uint32_t)s ? (n_fill - 1 - s) / VS + 1 : 0;
          if (fills > 0) drain_wait(&bar_v_full[s], (fills - 1) & 1u);
        }
      }
      __syncwarp();
    } else if (role == 1) {
      // ------------------------------------------------------------ S = Q K^T and dQ += dS K issuer
      // Two issuing threads, as in the forward: a barrier wait in one does not
      // leave the tensor pipe idle while the other has products to issue.
      // This one issues, per tile g of an item, S(g) and then dQ(g-1) once the
      // dS warps have written dS(g-1) (ds_ready): S(g+1) thus follows dQ(g-1)
      // at once and is ready one tile ahead.  S(g) goes into S buffer g % 2,
      // whose dS(g-2) the dQ(g-2) issued before it by this same thread reads:
      // the tensor pipe runs one thread's MMAs in issue order, so no wait.
      if (lane == 0) {
        constexpr uint32_t idesc_dq = idesc_bf16(128, D, false, true);
        const uint64_t qdesc = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t kdesc = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t kmn = sdesc_sw128(smem_u32(sK), 16384, 1024);  // K read MN-major
        int ks = 0;
        uint32_t kph = 0, g = 0, q_iter = 0;
        bool ok = true;
        // issue dQ += dS K for tile gg (its dS in S buffer gg % 2, its K in ring slot gg % KS)
        // (a pass for Delta alone has none: its S is read, and the slot is free)
        auto issue_dq = [&](uint32_t gg, int ncols, bool first, bool delta_pass) -> bool {
          const uint32_t b = gg & 1u;
          if (!mbar_wait(&bar_ds_ready[b], (gg >> 1) & 1u, &s_abort)) return false;
          tc_fence_after();
          const int kslot = (int)(gg % KS);
          const uint64_t kd = kmn + (uint64_t)((kslot * C::kKVBytes) >> 4);
          if (!delta_pass)
            for (int kk = 0; kk < ncols / 16; ++kk)
              mma_ts(tmem + C::kColDQ, tmem + b * 128u + C::ds_col(kk), kd + (uint64_t)(kk * (2048 >> 4)), idesc_dq,
                     (first && kk == 0) ? 0u : 1u);
          if constexpr (C::kMass)
            for (int kk = 0; kk < ncols / 16; ++kk)
              mma_ts(tmem + C::kColM, tmem + b * 128u + C::ds_col(kk) + C::kMassOff, kd + (uint64_t)(kk * (2048 >> 4)),
                     idesc_dq, (first && kk == 0) ? 0u : 1u);
          tc_commit(&bar_k_empty[kslot]);  // the K slot's last reader
          return true;
        };
        for (uint32_t kit = 0; ok; ++kit) {
          int w;
          if (!item_take_one(&ring, kit, w, &s_abort) || w >= n_items) break;
          const QItem it = q_item<kGrouped, kMod>(p, n_entries, w);
          int n = 0;
          for_each_kv_tile<kMod>(it, p, [&](int, int) { ++n; });
          if (!mbar_wait(&bar_q_full, q_iter & 1u, &s_abort)) break;
          ++q_iter;
          tc_fence_after();
          if (n == 0) {
            tc_commit(&bar_q_empty);
            continue;
          }
          bool last;
          for (int2 keys = first_keys<D, kMod>(p, it, last); ok; keys = all_keys(it), last = true) {
            int j = 0, prev_cols = 0;
            for_each_kv_tile<kMod>(it, p, keys, [&](int c, int jt) {
              if (!ok) return;
              const int ncols = q_tile_ncols<kMod>(it, p, c, jt);
              const uint32_t b = g & 1u;
              if (!mbar_wait(&bar_k_full[ks], kph, &s_abort)) {
                ok = false;
                return;
              }
              tc_fence_after();
              const uint32_t idesc_s = idesc_bf16(128, ncols, false, false);
              const uint64_t kd = kdesc + (uint64_t)((ks * C::kKVBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                mma_ss(tmem + b * 128u, qdesc + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
              }
              tc_commit(&bar_s_full[b]);
              if (last && j == n - 1) tc_commit(&bar_q_empty);  // the item's last read of Q
              if (++ks == KS) {
                ks = 0;
                kph ^= 1u;
              }
              if (j > 0 && !issue_dq(g - 1, prev_cols, j == 1, !last)) {
                ok = false;
                return;
              }
              prev_cols = ncols;
              ++g;
              ++j;
            });
            if (ok && !issue_dq(g - 1, prev_cols, n == 1, !last)) ok = false;
            if (last) break;
          }
          if (!ok) break;
          tc_commit(&bar_dq_done);
        }
        tc_commit(&bar_drain);
        drain_wait(&bar_drain, 0);
      }
      __syncwarp();
    } else if (role == 3) {
      // ------------------------------------------------------------ dP = dO V^T issuer
      // Per tile g: once the dS warps have read dP of tile g-1 into registers
      // (dp_free: early in their work on g-1), dP of tile g -- so it is ready
      // when they come to g.
      if (lane == 0) {
        const uint64_t dodesc = sdesc_sw128(smem_u32(sDO), 16, 1024);
        const uint64_t vdesc = sdesc_sw128(smem_u32(sV), 16, 1024);
        int vs = 0;
        uint32_t vph = 0, g = 0, q_iter = 0;
        bool ok = true;
        for (uint32_t kit = 0; ok; ++kit) {
          int w;
          if (!item_take_one(&ring, kit, w, &s_abort) || w >= n_items) break;
          const QItem it = q_item<kGrouped, kMod>(p, n_entries, w);
          int n = 0;
          for_each_kv_tile<kMod>(it, p, [&](int, int) { ++n; });
          if (!mbar_wait(&bar_q_full, q_iter & 1u, &s_abort)) break;
          ++q_iter;
          tc_fence_after();
          if (n == 0) {
            tc_commit(&bar_q_empty);
            continue;
          }
          bool last;
          for (int2 keys = first_keys<D, kMod>(p, it, last); ok; keys = all_keys(it), last = true) {
            int j = 0;
            for_each_kv_tile<kMod>(it, p, keys, [&](int c, int jt) {
              if (!ok) return;
              const int ncols = q_tile_ncols<kMod>(it, p, c, jt);
              // the dP buffer is free once the dS warps have read tile g-1's dP
              if ((g > 0 && !mbar_wait(&bar_dp_free, (g - 1) & 1u, &s_abort)) ||
                  !mbar_wait(&bar_v_full[vs], vph, &s_abort)) {
                ok = false;
                return;
              }
              tc_fence_after();
              const uint32_t idesc_p = idesc_bf16(128, ncols, false, false);
              const uint64_t vd = vdesc + (uint64_t)((vs * C::kKVBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                mma_ss(tmem + C::kColDP, dodesc + off, vd + off, idesc_p, kk > 0 ? 1u : 0u);
              }
              tc_commit(&bar_dp_full);
              tc_commit(&bar_v_empty[vs]);
              if (last && j == n - 1) tc_commit(&bar_q_empty);  // the item's last read of dO
              if (++vs == VS) {
                vs = 0;
                vph ^= 1u;
              }
              ++g;
              ++j;
            });
            if (last) break;
          }
        }
        tc_commit(&bar_drain2);
        drain_wait(&bar_drain2, 0);
      }
      __syncwarp();
    }
  } else {
    if constexpr (kSplit) regs_raise<C::kComputeRegs>();
    // ------------------------------------------------------------ dS + epilogue
    // Thread (part, row) owns query row `row` (its TMEM lane) and the 32-column
    // chunks [kCh part, kCh part + kCh) of every tile, plus as many 32-column
    // chunks of dQ.
    constexpr int kCh = 4 / C::kGroups;
    const int part = warp >> 2;
    const int row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    constexpr int kChO = D / 32 >= C::kGroups ? D / 32 / C::kGroups : 1;  // chunks of dQ (parts past D have none)
    const float sl2 = p.scale_log2;
    // dQ rows start at multiples of 128 bytes: 32-byte stores when dQ is 32-byte aligned
    const bool dq_v8 = (reinterpret_cast<uintptr_t>(p.dq) & 31u) == 0;
    uint32_t g = 0, n_item = 0, n_eps = 0;
    bool ok = true;
    for (uint32_t kit = 0; ok; ++kit) {
      int w;
      if (!item_take_warp(&ring, kit, w, &s_abort)) {
        ok = false;
        break;
      }
      if (w >= n_items) break;
      const QItem it = q_item<kGrouped, kMod>(p, n_entries, w);
      const int prow = it.t * kTile + row;
      const bool in_rank = prow < rank_rows<kMod>(it.g);
      const int pos = in_rank ? local_to_pos(prow, it.r, it.g.cbq, p.cp) : 0;
      const bool valid = in_rank && pos < it.g.Lq;
      const int64_t grow = (int64_t)it.g.q_off + pos;
      // this row's lse (log2 units) and Delta; rows without a valid query mask
      // every key, so their values never matter
      float dlt = valid ? p.delta[(int64_t)it.h * p.T_q + grow] : 0.f;
      const float lse2 = valid ? p.lse2[(int64_t)it.h * p.T_q + grow] : 0.f;
      // scored: the keys this row sees, and its score function
      int2 sees = make_int2(0, 0);
      int cap = kCapNear;  // the item's form of tanh so far (see cap_form)
      ScoreConsts sc;
      if constexpr (kMod != 0) {
        if (valid) sees = query_sees(p, p.mods, it.g, it.b, pos);
        sc = score_consts<kMod, false>(p, it.h);
      }
      int jl = 0;
      float off = 0.f;  // how far Delta was off in the walk that made dQ
      bool last;
      for (int2 keys = first_keys<D, kMod>(p, it, last); ok; keys = all_keys(it), last = true) {
        // a sum over part of the row's keys says nothing: such a row sees none here
        if (kMod != 0 && !last && (sees.x < keys.x || sees.y > keys.y)) sees = make_int2(0, 0);
        float eps = 0.f;  // this thread's part of the row sum of P (dP - Delta)
        for_each_kv_tile<kMod>(it, p, keys, [&](int c, int j) {
          if (!ok) return;
          const uint32_t b = g & 1u;
          if (!mbar_wait(&bar_s_full[b], (g >> 1) & 1u, &s_abort) || !mbar_wait(&bar_dp_full, g & 1u, &s_abort)) {
            ok = false;
            return;
          }
          tc_fence_after();
          const int j0 = c * it.g.cbkv + j * kTile;
          int cnt = 0, from = 0;  // the row sees columns [from, cnt)
          if (valid) {
            cnt = imin(kTile, (c + 1) * it.g.cbkv - j0);
            if constexpr (kMod != 0) {
              cnt = imin(cnt, sees.y - j0);
              from = sees.x - j0;
            } else {
              cnt = imin(cnt, it.g.Lkv - j0);
              if (p.causal) cnt = imin(cnt, pos + it.g.koff - j0 + 1);
            }
            cnt = imax(cnt, 0);
          }
          const int ahead = pos + it.g.koff - j0 + 1;  // scored: columns up to the row's own position
          const bool abs_needed = (kMod & kModDist) != 0 && __any_sync(0xffffffffu, cnt > 0 && cnt > ahead);
          const int nch = ceil_div(q_tile_ncols<kMod>(it, p, c, j), 32);
          const uint32_t scol = tmem + lane_base + b * 128u;
          const uint32_t pcol = tmem + lane_base + C::kColDP;
          // dP of this thread's chunks first, so the buffer can take the
          // next tile's dP while dS is computed
          uint32_t dr[kCh][32];
#pragma unroll
          for (int kk = 0; kk < kCh; ++kk)
            if (kCh * part + kk < nch) tmem_ld32(pcol + 32 * (kCh * part + kk), dr[kk]);
#pragma unroll
          for (int kk = 0; kk < kCh; ++kk)
            if (kCh * part + kk < nch) tmem_ld_wait(dr[kk]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_dp_free);
          if constexpr (kMod != 0) {
            // dS = P (dP - Delta) (1 - tanh^2), in place over the scores, and the row
            // sum of P (dP - Delta); on the keys this row may not see P = 2^-inf = 0
            // against dP = 0, and dS is set to 0, whatever stood there
            constexpr bool kCap = (kMod & kModCap) != 0;
            // one chunk a thread, and two results of it: the form is settled before
            // they are made, and they go to TMEM as they are made
            constexpr bool kNow = C::kMass && kCh == 1;
            uint32_t pk[kCh][16], pm[C::kMass ? kCh : 1][16];
            // chunk ch of S, with the cap's masked columns at 0; true if any is masked
            auto load = [&](float(&y)[32], int ch) {
              uint32_t(&sr)[32] = reinterpret_cast<uint32_t(&)[32]>(y);
              tmem_ld32(scol + 32 * ch, sr);
              tmem_ld_wait(sr);
              const bool cut = __any_sync(0xffffffffu, cnt < 32 * ch + 32 || from > 32 * ch);
              if (kCap && cut) score_fill(y, from - 32 * ch, cnt - 32 * ch, 0.f);
              return cut;
            };
            float es[2];
            auto run = [&](auto form) {
              float am = 0.f;
#pragma unroll
              for (int i = 0; i < 2; ++i) es[i] = 0.f;
#pragma unroll
              for (int kk = 0; kk < kCh; ++kk) {
                const int ch = kCh * part + kk;  // this thread's 32-column chunk
                if (ch < nch) {
                  float y[32];
                  const bool cut = load(y, ch);
                  constexpr int kForm = decltype(form)::value;
                  constexpr bool kWide = kCap && kForm == kCapWide;
                  if constexpr (kCap) {
                    am = fmaxf(am, score_abs_max(y));
                    if constexpr (kNow) {
                      const int f = cap_form(am, sc);
                      if (f > kForm) return f;
                    }
                    if constexpr (!kWide) cap_run<kForm, -1, false>(y, sc, 1.f, 0.f, 0.f);
                  }
                  // wide: tanh = -1 there instead of P = 0, and dP - Delta = 0
                  if (cut) {
                    score_fill(y, from - 32 * ch, cnt - 32 * ch, -INFINITY);
                    score_fill(reinterpret_cast<float(&)[32]>(dr[kk]), from - 32 * ch, cnt - 32 * ch,
                               kWide ? dlt : 0.f);
                  }
                  const float a = kCap ? sc.cap_a : sl2;
                  const float top = kWide ? a - lse2 : -lse2;
                  auto write_ds = [&](auto bias) {
#pragma unroll
                    for (int n = 0; n < 32; n += 2) {
                      float x0, x1, t0, t1, w0, w1, b0 = top, b1 = top;
                      if constexpr ((kMod & kModDist) != 0) bias.at(n, b0, b1);
                      if constexpr (kWide) {
                        cap_wide_grad(x0, x1, w0, w1, y[n], y[n + 1], sc.cap_c);
                        ffma2(x0, x1, x0, x1, -a, -a, b0, b1);
                        // a masked key's bias may be far above the row's lse
                        if constexpr ((kMod & kModDist) != 0) x0 = fmin_nan(x0, 127.f), x1 = fmin_nan(x1, 127.f);
                      } else {
                        ffma2(x0, x1, y[n], y[n + 1], a, a, b0, b1);
                      }
                      fadd2(t0, t1, __uint_as_float(dr[kk][n]), __uint_as_float(dr[kk][n + 1]), -dlt, -dlt);
                      x0 = ex2(x0), x1 = ex2(x1);
                      fmul2(t0, t1, x0, x1, t0, t1);
                      fadd2(es[0], es[1], es[0], es[1], t0, t1);
                      if constexpr (kCap) {
                        if constexpr (!kWide) ffma2(w0, w1, -y[n], -y[n + 1], y[n], y[n + 1], 1.f, 1.f);
                        fmul2(y[n], y[n + 1], t0, t1, w0, w1);
                        if constexpr (C::kMass) fmul2(x0, x1, x0, x1, w0, w1);
                      } else {
                        y[n] = t0, y[n + 1] = t1;
                      }
                      if constexpr (C::kMass) pm[kk][n / 2] = pack_bf16x2(x0, x1);
                    }
                  };
                  const float d0 = (float)(ahead - 1 - 32 * ch);
                  if ((kMod & kModDist) != 0 && abs_needed)
                    write_ds(BiasRun<-1, true>(d0, sc.slope, top));
                  else
                    write_ds(BiasRun<-1, false, true>(d0, sc.slope, top));
                  if (cut) {
                    score_fill(y, from - 32 * ch, cnt - 32 * ch, 0.f);
                    if constexpr (C::kMass) score_mask(pm[kk], from - 32 * ch, cnt - 32 * ch);
                  }
#pragma unroll
                  for (int n = 0; n < 16; ++n) pk[kk][n] = pack_bf16x2(y[2 * n], y[2 * n + 1]);
                  // over columns already read
                  if constexpr (kNow)
                    if (C::kMass) tmem_st16(scol + C::ds_col(2 * ch) + C::kMassOff, pm[kk]);
                  if ((!kCap || kNow) && last) tmem_st16(scol + C::ds_col(2 * (kCh * part + kk)), pk[kk]);
                }
              }
              return kCap && !kNow ? cap_form(am, sc) : decltype(form)::value;
            };
            if constexpr (kCap) {
              cap_in_form(cap, run);
#pragma unroll
              for (int kk = 0; kk < kCh; ++kk)
                if (!kNow && last && kCh * part + kk < nch) tmem_st16(scol + C::ds_col(2 * (kCh * part + kk)), pk[kk]);
            } else {
              run(CapForm<kCapNear>{});
            }
            if constexpr (C::kMass && !kNow) {  // over columns that every chunk of this thread has been read from
#pragma unroll
              for (int kk = 0; kk < kCh; ++kk)
                if (kCh * part + kk < nch) tmem_st16(scol + C::ds_col(2 * (kCh * part + kk)) + C::kMassOff, pm[kk]);
            }
            eps += es[0] + es[1];
          } else {
#pragma unroll
            for (int kk = 0; kk < kCh; ++kk) {
              const int ch = kCh * part + kk;  // this thread's 32-column chunk
              if (ch < nch) {
                uint32_t sr[32];
                tmem_ld32(scol + 32 * ch, sr);
                tmem_ld_wait(sr);
                // keys this row may not see get S = -inf: P = 0 and dS = 0
                if (__any_sync(0xffffffffu, cnt < 32 * ch + 32)) {
#pragma unroll
                  for (int n = 0; n < 32; ++n)
                    if (32 * ch + n >= cnt) sr[n] = __float_as_uint(-INFINITY);
                }
                uint32_t pk[16];
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                  float x0, x1, t0, t1, g0, g1;
                  ffma2(x0, x1, __uint_as_float(sr[2 * n]), __uint_as_float(sr[2 * n + 1]), sl2, sl2, -lse2, -lse2);
                  const float p0 = ex2(x0), p1 = ex2(x1);
                  fadd2(t0, t1, __uint_as_float(dr[kk][2 * n]), __uint_as_float(dr[kk][2 * n + 1]), -dlt, -dlt);
                  fmul2(g0, g1, p0, p1, t0, t1);
                  pk[n] = pack_bf16x2(g0, g1);
                }
                tmem_st16(scol + C::ds_col(2 * ch), pk);
              }
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();  // every lane's dS is in TMEM and dP was read: one arrival speaks for the warp
          if (lane == 0) mbar_arrive(&bar_ds_ready[b]);  // dS of tile g is in TMEM
          ++g;
          ++jl;
        });
        if constexpr (kMod != 0) {
          // the row's warpgroups add their parts up, in a fixed order: the last
          // exchange's sum has been read; the parts are there; the sum is there
          if (ok && jl > 0) {
            uint64_t* bar = &bar_eps[warp & 3];
            auto sync = [&]() {
              __syncwarp();
              if (lane == 0) mbar_arrive(bar);
              ok = ok && mbar_wait(bar, n_eps++ & 1u, &s_abort);
            };
            sync();
            if (part > 0) s_eps[part - 1][row] = eps;
            sync();
            if (part == 0) {
#pragma unroll
              for (int i = 1; i < C::kGroups; ++i) eps += s_eps[i - 1][row];
              s_eps[0][row] = eps;
            }
            sync();
            off = s_eps[0][row];
            dlt += off;
          }
        }
        if (last) break;
        if (kMod != 0 && valid) sees = query_sees(p, p.mods, it.g, it.b, pos);
      }
      // (scored: the exchange above leaves each lane its own answer)
      if (kMod != 0 ? !__all_sync(0xffffffffu, ok) : !ok) {
        ok = false;
        break;
      }
      if constexpr (kMod != 0) {
        // the exact Delta, for the dK/dV kernel (every warpgroup has read the old one)
        if (jl > 0 && valid && part == 0) p.delta_out[(int64_t)it.h * p.T_q + grow] = dlt;
      }
      // ---- epilogue: dQ * scale as bf16; zero on rows without a valid query
      if (jl > 0) {
        if (!mbar_wait(&bar_dq_done, n_item & 1u, &s_abort)) break;
        tc_fence_after();
        ++n_item;
      }
#pragma unroll 1
      for (int k = kChO * part; k < kChO * (part + 1) && k < D / 32; ++k) {
        uint32_t o[32];
        if (jl > 0) {
          tmem_ld32(tmem + lane_base + C::kColDQ + 32 * k, o);
          tmem_ld_wait(o);
          if constexpr (C::kMass) {  // dS = P (dP - Delta) w was made with Delta - off
            uint32_t m[32];
            tmem_ld32(tmem + lane_base + C::kColM + 32 * k, m);
            tmem_ld_wait(m);
#pragma unroll
            for (int n = 0; n < 32; ++n)
              o[n] = __float_as_uint(fmaf(-off, __uint_as_float(m[n]), __uint_as_float(o[n])));
          }
        } else {
#pragma unroll
          for (int n = 0; n < 32; ++n) o[n] = 0u;
        }
        if (in_rank)
          store32_bf16(p.dq + (grow * p.Hq + it.h) * D + 32 * k, o, valid ? p.scale : 0.f, dq_v8);
      }
      tc_fence_before();
    }
    // ---- dQ rows past the last sequence (the slack up to dq_rows): zero
    if (ok) {
      const int Tend = p.eff[(p.B + 1) + p.B];
      const int64_t nvec = (p.dq_rows - Tend) * (int64_t)p.Hq * (D / 8);
      const int64_t base = (int64_t)Tend * p.Hq * D;
      for (int64_t i = (int64_t)blockIdx.x * 32 * C::kWarps + tid; i < nvec; i += (int64_t)gridDim.x * 32 * C::kWarps)
        reinterpret_cast<uint4*>(p.dq + base)[i] = make_uint4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (role == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (tid == 0 && s_abort) atomicCAS(p.dev_status, 0, THD_ERR_TIMEOUT);
}

template <int D, bool kGrouped, int kMod>
static cudaError_t launch_dq_t(const DqParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                               cudaStream_t st) {
  using C = DqCfg<D, kMod>;
  cudaError_t ea = cudaFuncSetAttribute(dq_kernel<D, kGrouped, kMod>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (ea != cudaSuccess) return ea;
  prof_before(THD_KERNEL_BWD_DQ, st);
  dq_kernel<D, kGrouped, kMod><<<grid, C::kThreads, C::kSmem, st>>>(p, tk, tv);
  count_launch();
  cudaError_t e = cudaGetLastError();
  prof_after(THD_KERNEL_BWD_DQ, st);
  return e;
}

}  // namespace thd
