// cross_kernel.cuh -- attention of queries to an encoder's states of another
// length, for sm_100a: any Sq and Skv, grouped key heads, and per batch
// element a length on the device behind which states are not seen.
//
// The mathematics and the two-slot pipeline are those of attn_kernel.cuh: per
// slot a 128-row Q tile, S = Q K^T and O (+)= P V on tcgen05 with S, P and O
// in TMEM, the running maximum raised only when it grows by more than 2^8, l
// and m in float32, P rounded to bf16 (the tensor core's operand type).
//
// What differs is the walk.  An encoder's states are short (77 or 512 keys are
// 1 to 4 tiles), so a CTA that served one pair of Q tiles would spend most of
// its life filling and draining its pipeline.  Here one CTA per SM walks units
// (batch element, key head, pair of Q tiles) and every role runs on across
// them: the producer loads the next unit's Q as soon as the last S of this one
// is issued, and the MMA warp issues the next unit's first S behind this one's
// last P V.  The softmax warps, whose exponentials bound the kernel, go
// straight on to the next unit's scores: four warps of their own turn O into
// the output (TMEM, times 1 / l from shared memory, bf16, a swizzled staging
// tile, one tensor store per warp and 64 columns) and then let the next P V
// overwrite O.
//
// A tile's 128 rows are 128 queries of one head, or, when the group is a power
// of two up to 32 heads, 128 / group queries of all its heads (row r is query
// r / group, head r % group: one tensor box with the heads as its second
// axis), which wastes fewer rows when queries are few or odd.  The pair of a
// unit is two consecutive (head of the group, tile) entries: grouped heads
// fill both slots even with one tile each, and both slots read the same K and
// V tiles.
//
// With fewer units than SMs and long states (kSplit), a cluster of CTAs shares
// a unit: each walks a run of its key tiles, leaves its unnormalised O, m and l
// in its own shared memory (the K and V stages are free by then), and each
// joins a share of the rows over the cluster by the LSE rule, in rank order:
// one launch, no workspace, no atomics.
//
// States behind kv_lens may hold anything, NaN included: their scores are
// replaced before use, and their rows of V in a partly valid tile, which
// P = 0 would not cancel, are zeroed in shared memory by warp 2 before P V.
// A batch element without states gives out = 0, LSE = -inf.
//   warp 0   TMA producer         warps 4-7    epilogue of both slots
//   warp 1   TMEM, MMA issuer     warps 8-11   softmax of slot 0
//   warp 2   zeroes V's padding   warps 12-15  softmax of slot 1
//   warp 3   idle
#pragma once

#include <type_traits>

#include "attn_kernel.cuh"
#include "operators_internal.h"
#include "operators_ptx.cuh"

namespace cpattn {

template <int D>
struct CrossSmem {
  static constexpr int kHalves = D / 64;
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kStages = 2;
  static constexpr int kOffQ = 0;                                  // one tile per slot
  static constexpr int kOffK = kOffQ + 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffStage = kOffV + kStages * kTileBytes;   // output staging: 32 rows a warp
  static constexpr int kWarpStage = 32 * D * 2;
  static constexpr int kOffInv = kOffStage + 4 * kWarpStage;       // [2 slots][2 units in turn][128] 1 / l
  static constexpr int kOffBar = kOffInv + 2 * 2 * 128 * 4;
  // q_full[2], q_empty[2], k_full[S], k_empty[S], v_full[S], v_empty[S], v_clean[S], s[2], p_half[2], p[2], o[2],
  // o_read[2], inv[2][2], tail
  static constexpr int kNumBars = 4 + 5 * kStages + 14 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
  // No alignment slack: the window starts 1024-aligned (declared so, and
  // checked at kernel entry).
  static constexpr int kAllocBytes = kBytes;
};
static_assert(CrossSmem<128>::kAllocBytes <= 232448, "cross attention shared memory exceeds the per-CTA limit");

constexpr int kCrossThreads = 512;
// Register split: launched at 128 a thread (512 x 128); the control and the
// epilogue warpgroups give up what the softmax warpgroups need.
constexpr int kCrossRegsControl = 56;
constexpr int kCrossRegsEpilogue = 72;
constexpr int kCrossRegsSoftmax = 192;
static_assert(128 * (kCrossRegsControl + kCrossRegsEpilogue) + 256 * kCrossRegsSoftmax <= kCrossThreads * 128,
              "register split exceeds launch");

// Unit -> batch element, key head, states, and whether slot 1 has a tile.
struct CrossUnit {
  int b, hk, pair;
  int len, n;         // valid keys counted from tile t0, key tiles walked
  int t0;             // first key tile (a split unit's CTAs start at their runs)
  bool two;
};
// Valid states of batch element b: kv_lens[b], held to 0 .. Skv.
__device__ __forceinline__ int cross_len(const CrossParams &p, int b) {
  return p.kv_lens == nullptr ? p.Skv : max(0, min(p.Skv, __ldg(p.kv_lens + b)));
}
template <bool kSplit>
__device__ __forceinline__ CrossUnit cross_unit(const CrossParams &p, int unit) {
  CrossUnit u;
  int rank = 0;
  if (kSplit) {
    const int at = unit;
    unit = at / p.splits;
    rank = at - unit * p.splits;
  }
  const int bh = p.by_pairs.div(unit);
  u.pair = unit - bh * p.pairs;
  u.b = p.by_hk.div(bh);
  u.hk = bh - u.b * p.Hk;
  u.len = cross_len(p, u.b);
  u.n = (u.len + kKVTile - 1) / kKVTile;
  u.t0 = 0;
  if (kSplit) {
    u.t0 = static_cast<int>(static_cast<long long>(u.n) * rank / p.splits);
    const int t1 = static_cast<int>(static_cast<long long>(u.n) * (rank + 1) / p.splits);
    u.len = min(u.len, t1 * kKVTile) - u.t0 * kKVTile;
    u.n = t1 - u.t0;
  }
  u.two = 2 * u.pair + 1 < p.group_tiles;
  return u;
}
// First query head and first query of a slot's tile; its row r is query
// q0 + (r >> pack_log2) of head h + (r & (pack - 1)).
__device__ __forceinline__ void cross_tile(const CrossParams &p, const CrossUnit &u, int slot, int &h, int &q0) {
  const int r = 2 * u.pair + slot;
  const int hg = p.by_q_tiles.div(r);
  h = u.hk * p.group + hg;
  q0 = (r - hg * p.q_tiles) * (kQTile >> p.pack_log2);
}

// Split units: where a CTA keeps 4 columns (piece) of a row of a slot's O, over
// the K and V stages: rows of D floats, the pieces exchanged by the row's
// number so that 32 lanes writing 32 rows spread over the banks.
template <int D>
__device__ __forceinline__ uint32_t cross_part_at(uint32_t sb, int slot, int row, int piece) {
  static_assert(2 * 128 * D * 4 <= CrossSmem<D>::kOffStage - CrossSmem<D>::kOffK, "split partials exceed the stages");
  return sb + CrossSmem<D>::kOffK + ((slot * 128 + row) * (D / 4) + (piece ^ (row & (D / 4 - 1)))) * 16;
}
// Address of another CTA's shared memory, and loads from it.
__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// Limit of the epilogue's waits, which last a unit's whole walk (the other roles
// wait for a tile or two, and their giving up ends this wait too): 10 us more for
// each of its n key tiles, which take 2.
__device__ __forceinline__ uint64_t cross_walk_limit(uint64_t timeout_ns, int n) {
  return timeout_ns + static_cast<uint64_t>(n) * 10000u;
}
// Every thread of every CTA of the cluster arrives and waits.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kCrossThreads, 1) cross_fwd_kernel(const __grid_constant__ CrossParams p) {
  using L = CrossSmem<D>;
  constexpr int NST = L::kStages;
  constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, kKVTile, false);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true);
  extern __shared__ __align__(1024) uint8_t cross_smem[];
  const uint32_t sb = smem_u32(cross_smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_device_status, SITE_LAYOUT);
    return;
  }
  constexpr uint32_t BAR_QF = L::kOffBar;              // [2] Q tile of slot s loaded
  constexpr uint32_t BAR_QE = BAR_QF + 16;             // [2] its last S issued and done
  constexpr uint32_t BAR_KF = BAR_QE + 16;             // [NST]
  constexpr uint32_t BAR_KE = BAR_KF + 8 * NST;        // [NST]
  constexpr uint32_t BAR_VF = BAR_KE + 8 * NST;        // [NST]
  constexpr uint32_t BAR_VE = BAR_VF + 8 * NST;        // [NST]
  constexpr uint32_t BAR_VC = BAR_VE + 8 * NST;        // [NST] padding rows zeroed (every use of the stage)
  constexpr uint32_t BAR_S = BAR_VC + 8 * NST;         // [2] S in TMEM
  constexpr uint32_t BAR_PH = BAR_S + 16;              // [2] first half of P written
  constexpr uint32_t BAR_P = BAR_PH + 16;              // [2] P written
  constexpr uint32_t BAR_O = BAR_P + 16;               // [2] O of the unit complete
  constexpr uint32_t BAR_OR = BAR_O + 16;              // [2] O of the unit read out
  constexpr uint32_t BAR_INV = BAR_OR + 16;            // [2][2] 1 / l of slot s's units r % 2 published
  constexpr uint32_t BAR_TAIL = BAR_INV + 32;
  constexpr uint32_t TMEM_SLOT = L::kOffMisc;
  constexpr uint32_t ABORT = L::kOffMisc + 4;
  static_assert(BAR_TAIL + 8 <= L::kOffMisc, "barrier area");
  static_assert((BAR_VF + 8 * NST - BAR_QF) / 8 <= 32, "the producer's masks");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;
  // the units of this CTA's walk (a split unit's runs are numbered unit * splits + rank: one a CTA)
  const int first = blockIdx.x, step = gridDim.x;
  const int units = kSplit ? static_cast<int>(gridDim.x) : p.units;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(sb + BAR_QF + 8 * i, 1);
      mbar_init(sb + BAR_QE + 8 * i, 1);
      mbar_init(sb + BAR_S + 8 * i, 1);
      mbar_init(sb + BAR_PH + 8 * i, 4);   // one arrival per softmax warp
      mbar_init(sb + BAR_P + 8 * i, 4);
      mbar_init(sb + BAR_O + 8 * i, 1);
      mbar_init(sb + BAR_OR + 8 * i, 4);   // one arrival per epilogue warp
      mbar_init(sb + BAR_INV + 16 * i, 4);  // one arrival per softmax warp
      mbar_init(sb + BAR_INV + 16 * i + 8, 4);
    }
    for (int s = 0; s < NST; ++s) {
      mbar_init(sb + BAR_KF + 8 * s, 1);
      mbar_init(sb + BAR_KE + 8 * s, 1);
      mbar_init(sb + BAR_VF + 8 * s, 1);
      mbar_init(sb + BAR_VE + 8 * s, 1);
      mbar_init(sb + BAR_VC + 8 * s, 1);
    }
    mbar_init(sb + BAR_TAIL, 1);
    st_shared_volatile(sb + ABORT, 0u);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + TMEM_SLOT, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_volatile(sb + TMEM_SLOT);
  const uint32_t abort_flag = sb + ABORT;
  // Without lengths no tile has padding rows inside the tensor (rows past Skv
  // are filled with zeros by the load), and V needs no second barrier.
  const bool cleans = p.kv_lens != nullptr;

  if (warp < 4) {
    setmaxnreg_dec<kCrossRegsControl>();
    if (warp == 0) {
      // =========================================================== producer
      if (lane == 0) {
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
        int it = 0;              // K/V tiles loaded so far
        uint32_t q_used = 0, q_ph = 0;   // slots that loaded a Q tile, and the parity of the next load (a bit each)
        uint32_t loaded = 0, last = 0;   // barriers from BAR_QF on that a load completes on, and its last load's parity
        bool ok = true;
        auto load = [&](uint32_t dst, const CUtensorMap *tm, int h, int row, int b, uint32_t full, uint32_t empty,
                        uint32_t use_parity) -> bool {
          if (!mbar_wait(empty, use_parity ^ 1, abort_flag, tmo, SITE_PRODUCER)) return false;
          mbar_arrive_expect_tx(full, L::kTileBytes);
          for (int hf = 0; hf < L::kHalves; ++hf) tma_load_4d(dst + hf * L::kBoxBytes, tm, hf * 64, h, row, b, full);
          const uint32_t i = (full - sb - BAR_QF) >> 3;
          loaded |= 1u << i;
          last = (last & ~(1u << i)) | (use_parity << i);
          return true;
        };
        for (int unit = first; ok && unit < units; unit += step) {
          const CrossUnit U = cross_unit<kSplit>(p, unit);
          if (U.n == 0) continue;
          for (int s = 0; ok && s < (U.two ? 2 : 1); ++s) {
            int h, q0;
            cross_tile(p, U, s, h, q0);
            ok = load(sb + L::kOffQ + s * L::kTileBytes, &p.tm_q, h, q0, U.b, sb + BAR_QF + 8 * s,
                      sb + BAR_QE + 8 * s, (q_ph >> s) & 1);
            q_used |= 1u << s;
            q_ph ^= 1u << s;
            if (s == 0 && ok) {   // the first K tile between the two Q tiles: slot 0 can start
              const int st = it % NST;
              ok = load(sb + L::kOffK + st * L::kTileBytes, &p.tm_k, U.hk, U.t0 * kKVTile, U.b, sb + BAR_KF + 8 * st,
                        sb + BAR_KE + 8 * st, (it / NST) & 1);
            }
          }
          for (int j = 0; ok && j < U.n; ++j, ++it) {
            const int st = it % NST;
            const uint32_t ph = (it / NST) & 1;
            if (j > 0)
              ok = load(sb + L::kOffK + st * L::kTileBytes, &p.tm_k, U.hk, (U.t0 + j) * kKVTile, U.b, sb + BAR_KF + 8 * st,
                        sb + BAR_KE + 8 * st, ph);
            if (ok)
              ok = load(sb + L::kOffV + st * L::kTileBytes, &p.tm_v, U.hk, (U.t0 + j) * kKVTile, U.b, sb + BAR_VF + 8 * st,
                        sb + BAR_VE + 8 * st, ph);
          }
        }
        // Every last use must be released by the MMAs before the CTA exits.
        if (ok) {
          for (int j = 0; j < NST && j < it; ++j) {
            const int i = it - 1 - j;
            mbar_wait(sb + BAR_KE + 8 * (i % NST), (i / NST) & 1, 0u, tmo, SITE_TAIL);
            mbar_wait(sb + BAR_VE + 8 * (i % NST), (i / NST) & 1, 0u, tmo, SITE_TAIL);
          }
          for (int s = 0; s < 2; ++s)
            if ((q_used >> s) & 1) mbar_wait(sb + BAR_QE + 8 * s, ((q_ph >> s) & 1) ^ 1, 0u, tmo, SITE_TAIL);
        } else {   // a wait gave up: no CTA exits before what it loads has landed
          for (; loaded != 0; loaded &= loaded - 1) {
            const int i = __ffs(loaded) - 1;
            mbar_wait(sb + BAR_QF + 8 * i, (last >> i) & 1, 0u, tmo, SITE_TAIL);
          }
        }
      }
    } else if (warp == 1) {
      // =========================================================== MMA issuer
      {
        // The whole warp runs this role and one elected lane issues.  An MMA
        // takes the tensor core 64 cycles and its operands uniform registers;
        // the code of a lone lane, which computes them in its own registers and
        // shares its scheduler with two softmax warps, took some 105 cycles for
        // each (24 heads, 18432 queries, 2048 states: 415 us, this way 371; 357 since).
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
          return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, tmo, SITE_MMA));
        };
        auto commit = [&](uint32_t bar) {
          if (elect_one()) mma_commit(bar);
          __syncwarp();
        };
        const uint32_t dQ = smem_desc_sw128_lo(sb + L::kOffQ, 16);
        const uint32_t dK = smem_desc_sw128_lo(sb + L::kOffK, 16);
        const uint32_t dV = smem_desc_sw128_lo(sb + L::kOffV, L::kBoxBytes);
        auto issue_qk = [&](int s, int st) {
          const uint32_t a0 = opaque_u32(dQ + ((s * L::kTileBytes) >> 4));
          const uint32_t b0 = opaque_u32(dK + ((st * L::kTileBytes) >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * L::kBoxBytes + (kk & 3) * 32) >> 4;
              mma_ss_lo(tmem + s * 128, a0 + off, b0 + off, IDESC_QK, kk > 0 ? 1u : 0u);
            }
            mma_commit(sb + BAR_S + 8 * s);
          }
          __syncwarp();
        };
        auto issue_pv = [&](int s, int st, bool acc, int half) {
          const uint32_t b0 = opaque_u32(dV + ((st * L::kTileBytes) >> 4));
          if (elect_one()) {
#pragma unroll
            for (int k4 = 0; k4 < kKVTile / 32; ++k4) {
              const int kk = half * (kKVTile / 32) + k4;
              mma_ts_lo(tmem + 256 + s * D, tmem + s * 128 + kk * 8, b0 + ((kk * 2048) >> 4), IDESC_PV,
                        (acc || kk > 0) ? 1u : 0u);
            }
          }
          __syncwarp();
        };
        // The next unit with keys from `unit` on (units without are the
        // epilogue's alone).
        auto next_unit = [&](int unit, int &n, bool &two) -> int {
          for (; unit < units; unit += step) {
            const CrossUnit U = cross_unit<kSplit>(p, unit);
            if (U.n > 0) {
              n = U.n;
              two = U.two;
              return unit;
            }
          }
          n = 0;
          two = false;
          return unit;
        };
        int it = 0;                                   // K/V tile of the walk
        // parities of the slots' next Q tile, P tile and unit of O, a bit each
        // (not arrays: a dynamic index would put them into local memory)
        uint32_t q_ph = 0, p_ph = 0, o_ph = 0;
        int n = 0, n1 = 0;
        bool two = false, two1 = false;
        int unit = next_unit(first, n, two);
        auto pv = [&](int s, int st, bool acc) -> bool {
          const uint32_t ph = (p_ph >> s) & 1;
          p_ph ^= 1u << s;
          if (!acc) {   // a new unit's O: the last one has been read out
            if (!wait(sb + BAR_OR + 8 * s, ((o_ph >> s) & 1) ^ 1)) return false;
            o_ph ^= 1u << s;
          }
          if (!wait(sb + BAR_PH + 8 * s, ph)) return false;
          tc_fence_after();
          issue_pv(s, st, acc, 0);
          if (!wait(sb + BAR_P + 8 * s, ph)) return false;
          tc_fence_after();
          issue_pv(s, st, acc, 1);
          return true;
        };
        bool ok = true;
#pragma unroll 1
        for (int s = 0; ok && n > 0 && s < (two ? 2 : 1); ++s) {   // S of the walk's first tile
          ok = wait(sb + BAR_QF + 8 * s, (q_ph >> s) & 1);
          q_ph ^= 1u << s;
          if (ok) ok = wait(sb + BAR_KF, 0);
          if (!ok) break;
          tc_fence_after();
          issue_qk(s, 0);
          if (n == 1) commit(sb + BAR_QE + 8 * s);
        }
        if (ok && n > 0) commit(sb + BAR_KE);
        while (ok && n > 0) {
          const int after = next_unit(unit + step, n1, two1);
          // One tile: a copy of the code for a unit's last, one for the others.
          auto tile_step = [&](auto is_last, int j) {
            const int st = it % NST, st1 = (it + 1) % NST;
            constexpr bool last = decltype(is_last)::value;
            const bool next_last = last ? n1 == 1 : j + 1 == n - 1;   // the S issued below is its unit's last
            ok = wait(sb + BAR_VF + 8 * st, (it / NST) & 1);
            if (ok && cleans) ok = wait(sb + BAR_VC + 8 * st, (it / NST) & 1);
            // Per slot: this tile's P V, then S of the next tile, or of the
            // next unit's first, behind it -- one copy of the code for both:
            // where the roles' code overflows the instruction cache, every warp
            // of the SM waits (a copy each, and the epilogue unrolled, took
            // 60 us for 18432 queries of 24 heads against 128 states, this 46).
            const int slots = two ? 2 : 1, slots1 = last ? (n1 == 0 ? 0 : two1 ? 2 : 1) : slots;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (!ok) return;
              if (s < slots) {
                ok = pv(s, st, j > 0);
                if (!ok) return;
                if (last) commit(sb + BAR_O + 8 * s);
                if (s == slots - 1) commit(sb + BAR_VE + 8 * st);
              }
              if (s < slots1) {
                if (last) {
                  ok = wait(sb + BAR_QF + 8 * s, (q_ph >> s) & 1);
                  q_ph ^= 1u << s;
                }
                if (ok && s == 0) ok = wait(sb + BAR_KF + 8 * st1, ((it + 1) / NST) & 1);
                if (!ok) return;
                tc_fence_after();
                issue_qk(s, st1);
                if (next_last) commit(sb + BAR_QE + 8 * s);
              }
            }
            if (ok && slots1 > 0) commit(sb + BAR_KE + 8 * st1);
            ++it;
          };
          int j = 0;
          for (; ok && j < n - 1; ++j) tile_step(std::integral_constant<bool, false>{}, j);
          if (ok) tile_step(std::integral_constant<bool, true>{}, j);
          unit = after;
          n = n1;
          two = two1;
        }
        commit(sb + BAR_TAIL);
        if (lane == 0) mbar_wait(sb + BAR_TAIL, 0, 0u, tmo, SITE_TAIL);
        __syncwarp();
      }
    } else if (warp == 2 && cleans) {
      // =========================================================== V padding
      int it = 0;
      bool ok = true;
      for (int unit = first; ok && unit < units; unit += step) {
        const CrossUnit U = cross_unit<kSplit>(p, unit);
        for (int j = 0; j < U.n; ++j, ++it) {
          const int st = it % NST;
          const bool w = mbar_wait(sb + BAR_VF + 8 * st, (it / NST) & 1, abort_flag, tmo, SITE_PRODUCER);
          if (__any_sync(0xffffffffu, !w)) {
            ok = false;
            break;
          }
          const int valid = U.len - j * kKVTile;
          if (valid < kKVTile) {
            // rows valid .. 127 of the tile: 128 bytes each in every column half
            const int chunks = (kKVTile - valid) * 8;
            for (int hf = 0; hf < L::kHalves; ++hf)
              for (int i = lane; i < chunks; i += 32)
                st_shared_v4(sb + L::kOffV + st * L::kTileBytes + hf * L::kBoxBytes + valid * 128 + i * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sb + BAR_VC + 8 * st);
        }
      }
    }
  } else if (warp < 8) {
    setmaxnreg_dec<kCrossRegsEpilogue>();
    // =========================================================== epilogue
    const int part = warp & 3;                         // TMEM lanes [32 part, 32 part + 32)
    const uint32_t lane_base = static_cast<uint32_t>(part * 32) << 16;
    const uint32_t stage = sb + L::kOffStage + part * L::kWarpStage;
    uint32_t rounds = 0;                               // units with keys finished: slot 0's, slot 1's << 16
    bool ok = true;
    if (kSplit) {
      // Unnormalised O of both slots to shared memory, once neither slot's
      // MMAs read the K and V stages any more.
      const CrossUnit U = cross_unit<kSplit>(p, first);
      if (U.n > 0) {
        const uint64_t limit = cross_walk_limit(tmo, U.n);
        bool w = mbar_wait(sb + BAR_O, 0, abort_flag, limit, SITE_EPILOGUE);
        if (U.two) w = w && mbar_wait(sb + BAR_O + 8, 0, abort_flag, limit, SITE_EPILOGUE);
        ok = !__any_sync(0xffffffffu, !w);
        __syncwarp();
        tc_fence_after();
      }
      const int row = part * 32 + lane;
      for (int slot = 0; ok && slot < (U.two ? 2 : 1); ++slot) {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          if (U.n > 0) {
            tmem_ld32_wait(tmem + lane_base + 256 + slot * D + c0, o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(cross_part_at<D>(sb, slot, row, (c0 >> 2) + k), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
    }
    for (int unit = first; !kSplit && ok && unit < units; unit += step) {
      const CrossUnit U = cross_unit<kSplit>(p, unit);
#pragma unroll 1
      for (int slot = 0; slot < (U.two ? 2 : 1); ++slot) {
        float inv = 0.f;
        if (U.n > 0) {
          const uint32_t r = (rounds >> (16 * slot)) & 0xffffu;   // (its low two bits are used)
          rounds = slot == 0 ? (rounds & 0xffff0000u) | ((rounds + 1) & 0xffffu) : rounds + 0x10000u;
          const uint64_t limit = cross_walk_limit(tmo, U.n);
          bool w = mbar_wait(sb + BAR_INV + 16 * slot + 8 * (r & 1), (r >> 1) & 1, abort_flag, limit, SITE_EPILOGUE);
          w = w && mbar_wait(sb + BAR_O + 8 * slot, r & 1, abort_flag, limit, SITE_EPILOGUE);
          if (__any_sync(0xffffffffu, !w)) {
            ok = false;
            break;
          }
          __syncwarp();
          tc_fence_after();
          inv = ld_shared_f32(sb + L::kOffInv + ((slot * 2 + (r & 1)) * 128 + part * 32 + lane) * 4);
        }
        // the staging tile is free once the last stores have read it
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          if (U.n > 0) {
            tmem_ld32_wait(tmem + lane_base + 256 + slot * D + c0, o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          // row `lane` of the staging box of these 64 columns, 128-byte swizzled
          const uint32_t row = stage + (c0 >> 6) * 4096 + lane * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t chunk = ((c0 & 63) >> 3) + k;
            st_shared_v4(row + ((chunk ^ (lane & 7)) << 4),
                         pack_bf16x2(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                         pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                         pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                         pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
          }
        }
        if (U.n > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sb + BAR_OR + 8 * slot);
        }
        fence_proxy_async_shared();
        __syncwarp();
        int h, q;
        cross_tile(p, U, slot, h, q);
        q += (part * 32) >> p.pack_log2;               // queries past Sq are clipped by the store
        if (lane == 0 && q < p.Sq) {
          for (int hf = 0; hf < L::kHalves; ++hf)
            tma_store_4d(&p.tm_out, stage + hf * 4096, hf * 64, h, q, U.b);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else {
    setmaxnreg_inc<kCrossRegsSoftmax>();
    // =========================================================== softmax
    const int slot = (warp - 8) >> 2;
    const int row = ((warp & 3) << 5) + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_base + slot * 128;
    const uint32_t tO = tmem + lane_base + 256 + slot * D;
    const float c = p.scale_log2;
    uint32_t tiles = 0, rounds = 0;   // tiles and units with keys seen by this slot
    for (int unit = first; unit < units; unit += step) {
      const CrossUnit U = cross_unit<kSplit>(p, unit);
      if (slot == 1 && !U.two) continue;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < U.n; ++j, ++tiles) {
        const bool w = mbar_wait(sb + BAR_S + 8 * slot, tiles & 1, abort_flag, tmo, SITE_SOFTMAX);
        if (__any_sync(0xffffffffu, !w)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const int kvalid = U.len - j * kKVTile;
        if (kvalid < kKVTile) {
          // -inf over the scores of states behind the length, in TMEM: loops of
          // a few instructions where selects on 128 registers are 4 KB of code
          int k = kvalid;
#pragma unroll 1
          for (; (k & 15) != 0; ++k) tmem_st1(tS + k, 0xff800000u);
          uint32_t inf[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) inf[x] = 0xff800000u;
#pragma unroll 1
          for (; k < kKVTile; k += 16) tmem_st16(tS + k, inf);
          tmem_st_wait();
        }
        uint32_t s[128];
        tmem_ld128_wait(tS, s);
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 8]));
#pragma unroll
        for (int k = 16; k < 128; k += 16)
#pragma unroll
          for (int q = 0; q < 8; ++q) mx[q] = fmax3(mx[q], __uint_as_float(s[k + q]), __uint_as_float(s[k + 8 + q]));
        const float tmax = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * c;
        if (j == 0) {
          m = tmax;
        } else {
          const bool need = tmax > m + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2_approx(m - tmax) : 1.0f;
            if (need) {
              l *= alpha;
              m = tmax;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16_wait(tO + c0, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st16(tO + c0, o);
            }
          }
        }
        const uint64_t cc = f2_pack(c, c);
        const float mb = m == -INFINITY ? 0.0f : m;
        const uint64_t mm = f2_pack(-mb, -mb);
        uint64_t lsum0 = 0, lsum1 = 0;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[c0 + 2 * k]), __uint_as_float(s[c0 + 2 * k + 1])), cc, mm);
            float x0, x1;
            f2_unpack(x, x0, x1);
            const uint64_t pp = f2_pack(ex2_approx(x0), ex2_approx(x1));
            if (k & 1) lsum1 = f2_add(lsum1, pp); else lsum0 = f2_add(lsum0, pp);
            float p0, p1;
            f2_unpack(pp, p0, p1);
            pk[k] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tS + c0 / 2, pk);
          if (c0 == 32) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sb + BAR_PH + 8 * slot);
          }
        }
        {
          float a0, a1, b0, b1;
          f2_unpack(lsum0, a0, a1);
          f2_unpack(lsum1, b0, b1);
          l += (a0 + a1) + (b0 + b1);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + BAR_P + 8 * slot);
      }
      if (!ok) break;
      if (kSplit) {   // m and l for the join
        st_shared_f32(sb + L::kOffInv + (slot * 128 + row) * 4, m);
        st_shared_f32(sb + L::kOffInv + ((2 + slot) * 128 + row) * 4, l);
        continue;
      }
      // 1 / l for the epilogue, and the row's LSE.  Two buffers with a barrier
      // each in turn: the softmax may be a whole unit ahead of the epilogue,
      // but the scores of the unit after that are issued only when this unit's
      // O has been read, so a barrier never runs two phases ahead of its waiter.
      if (U.n > 0) {
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // l NaN: NaN
        st_shared_f32(sb + L::kOffInv + ((slot * 2 + (rounds & 1)) * 128 + row) * 4, inv);
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + BAR_INV + 16 * slot + 8 * (rounds & 1));
        ++rounds;
      }
      int h, q;
      cross_tile(p, U, slot, h, q);
      q += row >> p.pack_log2;
      h += row & ((1 << p.pack_log2) - 1);
      if (p.lse != nullptr && q < p.Sq)
        p.lse[(static_cast<size_t>(U.b) * p.H + h) * p.Sq + q] =
            l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }

  if (kSplit) {
    // ---- join: CTA `rank` of the cluster takes every splits-th run of rows
    __syncwarp();
    cluster_sync_all();
    const int splits = p.splits, rank = static_cast<int>(blockIdx.x) % splits;
    const CrossUnit U = cross_unit<kSplit>(p, blockIdx.x);
    const int all = (U.two ? 2 : 1) * 128 * (D / 4);
    for (int i = rank * kCrossThreads + threadIdx.x; i < all; i += splits * kCrossThreads) {
      const int piece = i % (D / 4), r = i / (D / 4);      // r: slot * 128 + row
      int h, q;
      cross_tile(p, U, r >> 7, h, q);
      q += (r & 127) >> p.pack_log2;
      h += r & ((1 << p.pack_log2) - 1);
      if (q >= p.Sq) continue;
      const uint32_t am = sb + L::kOffInv + r * 4, ao = cross_part_at<D>(sb, r >> 7, r & 127, piece);
      float M = -INFINITY;
      for (int j = 0; j < splits; ++j) M = fmaxf(M, ld_cluster_f32(map_cluster(am, j)));
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float lt = 0.f;
      for (int j = 0; j < splits; ++j) {
        const float mj = ld_cluster_f32(map_cluster(am, j)), lj = ld_cluster_f32(map_cluster(am + 1024, j));
        const float4 v = ld_cluster_f4(map_cluster(ao, j));
        const float wgt = mj == -INFINITY ? 0.f : ex2_approx(mj - M);
        lt = fmaf(wgt, lj, lt);
        acc.x = fmaf(wgt, v.x, acc.x);
        acc.y = fmaf(wgt, v.y, acc.y);
        acc.z = fmaf(wgt, v.z, acc.z);
        acc.w = fmaf(wgt, v.w, acc.w);
      }
      const float inv = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);   // NaN stays NaN
      uint2 *dst = reinterpret_cast<uint2 *>(p.out + ((static_cast<size_t>(U.b) * p.Sq + q) * p.H + h) * D) + piece;
      *dst = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (piece == 0 && p.lse != nullptr)
        p.lse[(static_cast<size_t>(U.b) * p.H + h) * p.Sq + q] =
            lt == 0.f ? -INFINITY : (M + log2f(lt)) * 0.69314718055994531f;
    }
    cluster_sync_all();   // no CTA leaves while another reads its memory
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace cpattn
