// cross_bwd_kernel.cuh -- gradient of cross attention for sm_100a.
//
// Per (batch element, query head), over the valid states, with P recomputed
// from the forward's LSE and Delta = rowsum(dO * O):
//   dS = P * (dO V^T - Delta),  dQ = dS K * scale,
//   dV = sum over the group's heads of P^T dO,  dK = the same sum of dS^T Q * scale.
// The products, their TMEM layout and the dS tiles are those of
// attn_bwd_kernel.cuh.  What differs:
//   - Delta of elements with few states is summed from P and dP, since the saved
//     output is rounded (cross_delta_kernel).
//   - dK/dV: an encoder's states are few tiles and the queries many, so one CTA
//     a K/V tile would leave most SMs idle or unevenly loaded.  The walks of
//     all valid tiles -- every Q tile of every head of its group -- are laid
//     end to end and cut into equal runs, one CTA an SM: a CTA finishes the
//     tile that its run starts in, takes whole tiles, and starts its last, and
//     its roles run on from tile to tile.  Walks are ordered K tile by K tile,
//     and the CTAs a multiple of the K tiles where that leaves few SMs idle:
//     then the CTAs of a head's K tiles walk the same queries at the same time
//     and share them in L2 (in (head, K tile) order, where they walk apart,
//     the video workload took 743 us, with one part of a walk a CTA 661, so 614).
//     Runs that do not cover their tile leave float32 sums, which warps of the dQ
//     kernel add in a fixed order: no atomics, the same bytes every run.  A
//     group's heads are simply further Q tiles.
//   - dQ: the persistent product over the stored dS with Sq x Skv tiles.  Rows
//     of K behind the length meet dS = 0; they are zeroed in shared memory,
//     since they may hold NaN.
//   - A pair whose dS exceeds the scratch is done in ranges of its walk, one
//     after the other; their dK and dV are added in float32 (cross_range_kernel).
//     32768 queries of 32 / 4 heads of 128 against as many states, 17 GB of dS a
//     pair: 51 ms in ranges of 1 to 8 GB, as whole, and 77 in ranges of 256 MB.
//   - Gradients of states behind the length are zeros: those of a partly valid
//     tile come out of the products so, those of other tiles are written beside
//     the dQ product.
#pragma once

#include "attn_bwd_kernel.cuh"
#include "operators_internal.h"
#include "operators_ptx.cuh"
#include "cross_kernel.cuh"
#include "cross_token_kernel.cuh"

namespace cpattn {

__device__ __forceinline__ int cross_bwd_len(const CrossBwdParams &p, int b) {
  return p.kv_lens == nullptr ? p.Skv : max(0, min(p.Skv, __ldg(p.kv_lens + b)));
}

// Byte offset of the dS tile of pair bh (counted from p.bh0), step w of its walk
// and K tile kt.
__device__ __forceinline__ size_t cross_ds_tile(const CrossBwdParams &p, int bh_local, int w, int kt) {
  return ((static_cast<size_t>(bh_local) * p.walk + w) * p.k_tiles + kt) * kBwdDsTileBytes;
}

// The walks of the valid tiles end to end, in (K tile, pair, Q tile) order, and
// a CTA's run of them as segments: steps [w, w + n) of one tile.
struct CrossRun {
  long long left;               // steps from this segment on
  int w, n;                     // this segment
  int kt, bh_local, b, hk, len;
  // floor(x * inv) for inv = 1 / d: x + 1/2 keeps the quotient at least 1 / (2 d)
  // from an integer, far above a double's error at x < 2^46 (a 64-bit integer
  // division costs some 500 cycles).
  __device__ __forceinline__ static long long over(long long x, double inv) {
    return static_cast<long long>((static_cast<double>(x) + 0.5) * inv);
  }
  // First step of CTA `cta`'s run: floor(total * cta / ctas).
  __device__ __forceinline__ static long long start(const CrossBwdParams &p, long long total, int cta) {
    return over(total * cta, p.inv_ctas);
  }
  __device__ __forceinline__ void set_pair(const CrossBwdParams &p) {
    b = p.by_hk.div(p.bh0 + bh_local);
    hk = p.bh0 + bh_local - b * p.Hk;
  }
  // The first valid tile from element nb of K tile kt on.
  __device__ __forceinline__ void seek(const CrossBwdParams &p, int nb) {
    const int b0 = p.bh0 / p.Hk, b1 = (p.bh0 + p.n_bh - 1) / p.Hk;
    for (;; ++nb) {
      if (nb > b1) {
        nb = b0;
        if (++kt >= p.k_tiles) {   // not while steps are left
          left = 0;
          return;
        }
      }
      len = cross_bwd_len(p, nb);
      if (len > kt * 128) break;
    }
    b = nb;
    bh_local = max(p.bh0, b * p.Hk) - p.bh0;
    hk = p.bh0 + bh_local - b * p.Hk;
  }
  // Valid tile number `tile`; ends (with lengths): see cross_total_steps.
  __device__ __forceinline__ void locate(const CrossBwdParams &p, int tile, const int *ends) {
    if (p.kv_lens == nullptr) {
      kt = tile / p.n_bh;
      bh_local = tile - kt * p.n_bh;
      len = p.Skv;
      set_pair(p);
      return;
    }
    int here = 0;                // pairs with a valid tile kt
    for (int k = 0; k < p.k_tiles; ++k) here += ends[k];
    for (kt = 0; kt < p.k_tiles - 1 && tile >= here; ++kt) {
      tile -= here;
      here -= ends[kt];
    }
    for (seek(p, p.bh0 / p.Hk); left > 0; seek(p, b + 1)) {
      const int pairs = min(p.bh0 + p.n_bh, (b + 1) * p.Hk) - p.bh0 - bh_local;
      if (tile < pairs) break;
      tile -= pairs;
    }
    bh_local += tile;
    hk += tile;
  }
  __device__ __forceinline__ void init(const CrossBwdParams &p, long long total, int cta, const int *ends) {
    const long long x0 = start(p, total, cta);
    left = start(p, total, cta + 1) - x0;
    const int tile = static_cast<int>(over(x0, p.inv_walk));
    w = static_cast<int>(x0 - static_cast<long long>(tile) * p.walk);
    n = static_cast<int>(min(static_cast<long long>(p.walk - w), left));
    if (left > 0) locate(p, tile, ends);
  }
  __device__ __forceinline__ void next(const CrossBwdParams &p) {
    left -= n;
    w = 0;
    n = static_cast<int>(min(static_cast<long long>(p.walk), left));
    if (left <= 0) return;
    ++bh_local;
    if (p.kv_lens == nullptr) {
      if (bh_local == p.n_bh) {
        bh_local = 0;
        ++kt;
      }
      set_pair(p);
    } else if (bh_local < p.n_bh && hk + 1 < p.Hk) {
      ++hk;
    } else {
      seek(p, b + 1);
    }
  }
};
// Steps of all valid tiles' walks.  With lengths the block's threads first
// count, in shared memory, ends[k]: the pairs whose last valid tile is k.
// Every thread of the block takes part.
__device__ __forceinline__ long long cross_total_steps(const CrossBwdParams &p, int *ends) {
  long long tiles = static_cast<long long>(p.n_bh) * p.k_tiles;
  if (p.kv_lens != nullptr) {
    for (int k = threadIdx.x; k < p.k_tiles; k += blockDim.x) ends[k] = 0;
    __syncthreads();
    const int b1 = (p.bh0 + p.n_bh - 1) / p.Hk;
    for (int b = p.bh0 / p.Hk + static_cast<int>(threadIdx.x); b <= b1; b += blockDim.x) {
      const int n_kt = (cross_bwd_len(p, b) + 127) / 128;
      if (n_kt > 0) atomicAdd(ends + n_kt - 1, min(p.bh0 + p.n_bh, (b + 1) * p.Hk) - max(p.bh0, b * p.Hk));
    }
    __syncthreads();
    tiles = 0;
    for (int k = 0; k < p.k_tiles; ++k) tiles += static_cast<long long>(ends[k]) * (k + 1);
  }
  return tiles * p.walk;
}

// ==================================================================== Delta
// rowsum(dO * O) as attn_bwd_delta_kernel, except for elements of at most
// kCrossFewStates states.  The forward's output was rounded to bf16 and made
// with P rounded to bf16, which puts a common error into all of a row's
// dP - Delta; over n states it is some 1 / sqrt(n) of the roundings of P and dS
// themselves.  In dQ and dK, normal data, that error and theirs together are
// 0.0044 of the gradient at 2 states, 0.0038 at 3, 0.0026 at 16 and 0.0025 at
// 32, theirs alone 0.0023.  So few states take Delta by its definition,
// sum_j P_j dP_j, in float32.  Bound by the reads of q and dO, as the other is by out and dO:
// a warp takes 16 rows (queries of all heads of a group) by mma.m16n8k16
// against K and V in shared memory, loaded once a chunk of rows.  A fragment's k
// index may be any order of the head's elements, the same for both operands: a
// lane's are eight consecutive ones of each 32, so that all loads are 16 bytes.
// The whole backward, 32760 queries of 40 heads of 128, takes 519 us with 8
// states and 535 with 32, where rowsum(dO * O) took 524 and 518 (K and V from
// L1 557 and 639; the loads of one piece at a time 560 and 577); heads of 64,
// 8192 queries x 4, 32 / 8 heads, 303 against 277.
//   kMany: elements may also have more states; three CTAs an SM for the row
// sums, whose registers leave room for one piece's loads.
constexpr int kCrossFewStates = 32;
template <int D, bool kMany>
__global__ void __launch_bounds__(256, kMany ? 3 : 2) cross_delta_kernel(const __grid_constant__ CrossDeltaParams p) {
  auto len_of = [&](int b) { return p.kv_lens == nullptr ? p.Skv : max(0, min(p.Skv, __ldg(p.kv_lens + b))); };
  if constexpr (kMany)
    bwd_delta_rows(p.out, p.dout, p.delta, p.B, p.Sq, p.H, D,
                   [&](unsigned b) { return len_of(static_cast<int>(b)) <= kCrossFewStates; },
                   [&](unsigned r0, unsigned r1) {
                     const int b0 = p.by_element.div(static_cast<int>(r0)), b1 = p.by_element.div(static_cast<int>(r1));
                     return b0 == b1 && len_of(b0) <= kCrossFewStates;
                   });
  // K and V of a chunk's states in the order of the operands: [K, V][eight
  // states][32 elements of the head][lane]
  constexpr int kC = D / 32, kN = kCrossFewStates / 8;
  constexpr int kLoads = kMany ? 1 : kC;     // 32-element pieces loaded before any is used
  __shared__ uint4 kv[2][kN][kC][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
  const int group = p.H / p.Hk, rows = group * p.Sq;
  const unsigned chunks = static_cast<unsigned>(p.B) * p.Hk * p.chunks;
  for (unsigned u = blockIdx.x; u < chunks; u += gridDim.x) {
    // the key heads of the same queries next to each other: their rows are in DRAM
    const int bc = p.by_hk.div(static_cast<int>(u)), hk = static_cast<int>(u) - bc * p.Hk;
    const int b = p.by_chunks.div(bc), chunk = bc - b * p.chunks, len = len_of(b);
    if (len > kCrossFewStates) continue;
    __syncthreads();                         // the last chunk's K and V have been read
    for (int i = threadIdx.x; i < 2 * kN * kC * 32; i += 256) {
      const int j = (i / (kC * 32)) % kN * 8 + (i & 31) / 4, e = i / 32 % kC * 32 + (i & 3) * 8;
      const bool is_v = i >= kN * kC * 32;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (j < len)
        x = *reinterpret_cast<const uint4 *>(is_v ? p.v + b * p.vb + hk * p.vh + j * p.vs + e
                                                  : p.k + b * p.kb + hk * p.kh + j * p.ks + e);
      (&kv[0][0][0][0])[i] = x;
    }
    __syncthreads();
    const int end = min(p.blocks, (chunk + 1) * p.chunk_blocks);
    for (int block = chunk * p.chunk_blocks + warp; block < end; block += 8) {
      bool there[2];                         // this lane's rows lane / 4 and lane / 4 + 8 of the block
      size_t at[2];                          // their place in LSE and Delta
      const __nv_bfloat16 *q[2], *g[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = block * 16 + (lane >> 2) + 8 * i;
        there[i] = r < rows;
        const int s = p.by_group.div(there[i] ? r : 0), h = hk * group + (there[i] ? r : 0) - s * group;
        at[i] = (static_cast<size_t>(b) * p.H + h) * p.Sq + s;
        q[i] = p.q + b * p.qb + s * p.qs + h * p.qh + 8 * t;
        g[i] = p.dout + ((static_cast<size_t>(b) * p.Sq + s) * p.H + h) * D + 8 * t;
      }
      float s[kN][4], dp[kN][4];
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = dp[n][e] = 0.f;
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += kLoads) {
        uint4 xs[kLoads][2], ys[kLoads][2];
#pragma unroll
        for (int c = 0; c < kLoads; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            xs[c][i] = ys[c][i] = make_uint4(0u, 0u, 0u, 0u);
            if (there[i]) {
              xs[c][i] = __ldcs(reinterpret_cast<const uint4 *>(q[i] + 32 * (c0 + c)));
              ys[c][i] = __ldcs(reinterpret_cast<const uint4 *>(g[i] + 32 * (c0 + c)));
            }
          }
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          const uint4 (&x)[2] = xs[c], (&y)[2] = ys[c];
          const uint32_t xa[4] = {x[0].x, x[1].x, x[0].y, x[1].y}, xb[4] = {x[0].z, x[1].z, x[0].w, x[1].w};
          const uint32_t ya[4] = {y[0].x, y[1].x, y[0].y, y[1].y}, yb[4] = {y[0].z, y[1].z, y[0].w, y[1].w};
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            if (8 * n >= len) break;           // (the same for the whole warp)
            const uint4 kk = kv[0][n][c0 + c][lane], vv = kv[1][n][c0 + c][lane];
            mma_16n8k16(s[n], xa, kk.x, kk.y);
            mma_16n8k16(s[n], xb, kk.z, kk.w);
            mma_16n8k16(dp[n], ya, vv.x, vv.y);
            mma_16n8k16(dp[n], yb, vv.z, vv.w);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float lse = there[i] ? __ldg(p.lse + at[i]) : INFINITY;
        const float l2 = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;   // -inf: the row saw nothing
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (8 * n + 2 * t + e < len)
              sum = fmaf(ex2_approx(fmaf(s[n][2 * i + e], p.scale_log2, -l2)), dp[n][2 * i + e], sum);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (t == 0 && there[i]) p.delta[at[i]] = sum;
      }
    }
  }
}

// =================================================================== dK, dV
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_bwd_dkv_kernel(const __grid_constant__ CrossBwdParams p) {
  using L = BwdSmem<D, 2, true>;
  constexpr uint32_t IDESC_SS = idesc_bf16_f32(128, 128, false);   // S^T = K Q^T, dP^T = V dO^T
  constexpr uint32_t IDESC_ACC = idesc_bf16_f32(128, D, true);     // dV += P^T dO, dK += dS^T Q
  extern __shared__ __align__(1024) uint8_t bwd_smem[];
  const uint32_t sb = smem_u32(bwd_smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_device_status, SITE_LAYOUT);
    return;
  }
  constexpr int QS = L::kStagesC, OS = L::kStagesE;
  constexpr uint32_t BAR_KV = L::kOffBar;          // K and V loaded
  constexpr uint32_t BAR_QF = BAR_KV + 8;          // [QS]
  constexpr uint32_t BAR_QE = BAR_QF + 8 * QS;     // [QS]
  constexpr uint32_t BAR_OF = BAR_QE + 8 * QS;     // [OS] dO tile full
  constexpr uint32_t BAR_OE = BAR_OF + 8 * OS;     // [OS]
  constexpr uint32_t BAR_S = BAR_OE + 8 * OS;      // S^T(i) in TMEM
  constexpr uint32_t BAR_P = BAR_S + 8;            // P^T(i) written
  constexpr uint32_t BAR_DP = BAR_P + 8;           // dP^T(i) in TMEM
  constexpr uint32_t BAR_DS = BAR_DP + 8;          // dS^T(i) written
  constexpr uint32_t BAR_ACC = BAR_DS + 8;         // dV and dK complete
  constexpr uint32_t BAR_TAIL = BAR_ACC + 8;
  constexpr uint32_t BAR_VEC = BAR_TAIL + 8;       // this Q tile's LSE / Delta in smem
  constexpr uint32_t BAR_KVE = BAR_VEC + 8;        // the segment's last S and dP done: K and V may be replaced
  constexpr uint32_t BAR_ACCE = BAR_KVE + 8;       // dV and dK read out
  constexpr uint32_t TMEM_SLOT = L::kOffMisc;
  constexpr uint32_t ABORT = L::kOffMisc + 4;
  static_assert(BAR_ACCE + 8 <= L::kOffMisc, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;
  const int group = p.H / p.Hk;

  if (threadIdx.x == 0) {
    mbar_init(sb + BAR_KV, 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(sb + BAR_QF + 8 * s, 1);
      mbar_init(sb + BAR_QE + 8 * s, 1);
    }
    for (int s = 0; s < OS; ++s) {
      mbar_init(sb + BAR_OF + 8 * s, 1);
      mbar_init(sb + BAR_OE + 8 * s, 1);
    }
    mbar_init(sb + BAR_S, 1);
    mbar_init(sb + BAR_P, kBwdRowWarps);
    mbar_init(sb + BAR_DP, 1);
    mbar_init(sb + BAR_DS, kBwdRowWarps);
    mbar_init(sb + BAR_ACC, 1);
    mbar_init(sb + BAR_TAIL, 1);
    mbar_init(sb + BAR_VEC, kBwdRowWarps);
    mbar_init(sb + BAR_KVE, 1);
    mbar_init(sb + BAR_ACCE, kBwdRowWarps);
    st_shared_volatile(sb + ABORT, 0u);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + TMEM_SLOT, kBwdTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_volatile(sb + TMEM_SLOT);
  const uint32_t abort_flag = sb + ABORT;
  CrossRun R;
  int *const ends = reinterpret_cast<int *>(bwd_smem + L::kOffStaging);   // before the first dS
  R.init(p, cross_total_steps(p, ends), static_cast<int>(blockIdx.x), ends);
  __syncthreads();
  const int steps = static_cast<int>(R.left);   // (below 2^31: at most B Hk tiles of a walk each over many CTAs)

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
      tma_prefetch_desc(&p.tm_do);
      bool ok = true;
      int i = 0, seg = 0;        // Q tiles and K/V tiles loaded
      int o = 0;                 // dO tiles
      while (ok && R.left > 0) {
        ok = mbar_wait(sb + BAR_KVE, (seg & 1) ^ 1, abort_flag, tmo, SITE_PRODUCER);
        if (!ok) break;
        ++seg;
        mbar_arrive_expect_tx(sb + BAR_KV, 2 * L::kTileBytes);
        for (int hf = 0; hf < L::kHalves; ++hf) {
          tma_load_4d(sb + L::kOffA + hf * L::kBoxBytes, &p.tm_k, hf * 64, R.hk, R.kt * 128, R.b, sb + BAR_KV);
          tma_load_4d(sb + L::kOffB + hf * L::kBoxBytes, &p.tm_v, hf * 64, R.hk, R.kt * 128, R.b, sb + BAR_KV);
        }
        int hg = p.by_q_tiles.div(p.w0 + R.w), qt = p.w0 + R.w - hg * p.q_tiles;
        for (int j = 0; j < R.n; ++j) {
          const int qs = i % QS, os = o % OS;
          const int h = R.hk * group + hg;
          ok = mbar_wait(sb + BAR_QE + 8 * qs, ((i / QS) & 1) ^ 1, abort_flag, tmo, SITE_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + BAR_QF + 8 * qs, L::kTileBytes);
          for (int hf = 0; hf < L::kHalves; ++hf)
            tma_load_4d(sb + L::kOffC + qs * L::kTileBytes + hf * L::kBoxBytes, &p.tm_q, hf * 64, h, qt * 128, R.b,
                        sb + BAR_QF + 8 * qs);
          ++i;
          ok = mbar_wait(sb + BAR_OE + 8 * os, ((o / OS) & 1) ^ 1, abort_flag, tmo, SITE_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(sb + BAR_OF + 8 * os, L::kTileBytes);
          for (int hf = 0; hf < L::kHalves; ++hf)
            tma_load_4d(sb + L::kOffE + os * L::kTileBytes + hf * L::kBoxBytes, &p.tm_do, hf * 64, h, qt * 128, R.b,
                        sb + BAR_OF + 8 * os);
          ++o;
          if (++qt == p.q_tiles) {
            qt = 0;
            ++hg;
          }
        }
        if (ok) R.next(p);
      }
      // every last release must arrive before the CTA exits
      if (ok) {
        for (int j = 0; j < QS && j < i; ++j)
          mbar_wait(sb + BAR_QE + 8 * ((i - 1 - j) % QS), ((i - 1 - j) / QS) & 1, 0u, tmo, SITE_TAIL);
        for (int j = 0; j < OS && j < i; ++j)
          mbar_wait(sb + BAR_OE + 8 * ((i - 1 - j) % OS), ((i - 1 - j) / OS) & 1, 0u, tmo, SITE_TAIL);
        if (seg > 0) mbar_wait(sb + BAR_KVE, (seg - 1) & 1, 0u, tmo, SITE_TAIL);
      } else {   // a wait gave up: no CTA exits before what it loads has landed
        if (seg > 0) mbar_wait(sb + BAR_KV, (seg - 1) & 1, 0u, tmo, SITE_TAIL);
        for (int j = 0; j < QS && j < i; ++j)
          mbar_wait(sb + BAR_QF + 8 * ((i - 1 - j) % QS), ((i - 1 - j) / QS) & 1, 0u, tmo, SITE_TAIL);
        for (int j = 0; j < OS && j < o; ++j)
          mbar_wait(sb + BAR_OF + 8 * ((o - 1 - j) % OS), ((o - 1 - j) / OS) & 1, 0u, tmo, SITE_TAIL);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs this role and one elected lane issues (see
    // cross_fwd_kernel).
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, tmo, SITE_MMA));
    };
    const uint32_t dK = smem_desc_sw128_lo(sb + L::kOffA, 16);
    const uint32_t dV = smem_desc_sw128_lo(sb + L::kOffB, 16);
    const uint32_t dQk = smem_desc_sw128_lo(sb + L::kOffC, 16);               // K-major (S^T)
    const uint32_t dQmn = smem_desc_sw128_lo(sb + L::kOffC, L::kBoxBytes);    // MN-major (dK)
    const uint32_t dOk = smem_desc_sw128_lo(sb + L::kOffE, 16);               // K-major (dP^T)
    const uint32_t dOmn = smem_desc_sw128_lo(sb + L::kOffE, L::kBoxBytes);    // MN-major (dV)
    // d = a b^T, then `done` arrives.
    auto issue_ss = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t done) {
      tc_fence_after();
      const uint32_t a0 = opaque_u32(a), b0 = opaque_u32(b);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * L::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_lo(d, a0 + off, b0 + off, IDESC_SS, kk > 0 ? 1u : 0u);
        }
        mma_commit(done);
      }
      __syncwarp();
    };
    auto issue_acc = [&](uint32_t d, uint32_t a_tmem, uint32_t b, bool acc, uint32_t done) {
      tc_fence_after();
      const uint32_t b0 = opaque_u32(b);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_lo(d, a_tmem + bwd_packed_col(kk), b0 + ((kk * 2048) >> 4), IDESC_ACC, (acc || kk > 0) ? 1u : 0u);
        mma_commit(done);
      }
      __syncwarp();
    };
    auto stage_off = [&](int st) { return static_cast<uint32_t>((st * L::kTileBytes) >> 4); };
    auto commit = [&](uint32_t bar) {
      if (elect_one()) mma_commit(bar);
      __syncwarp();
    };
    // S and dP of walk step i (its segment's first: behind the load of K and V).
    auto first_s = [&](int i, int seg) -> bool {
      if (!wait(sb + BAR_KV, seg & 1) || !wait(sb + BAR_QF + 8 * (i % QS), (i / QS) & 1)) return false;
      issue_ss(tmem, dK, dQk + stage_off(i % QS), sb + BAR_S);
      return true;
    };
    auto dp = [&](int i, bool last) -> bool {
      if (!wait(sb + BAR_OF + 8 * (i % OS), (i / OS) & 1)) return false;
      issue_ss(tmem + 128, dV, dOk + stage_off(i % OS), sb + BAR_DP);
      if (last) commit(sb + BAR_KVE);
      return true;
    };
    int i = 0, seg = 0;
    bool ok = steps == 0 || (first_s(0, 0) && dp(0, R.n == 1));
    for (; ok && R.left > 0; ++seg) {
      const int n = R.n;
      const bool later = R.left > n;              // a further segment
      R.next(p);                                  // (its length is needed below)
      for (int j = 0; j < n; ++j, ++i) {
        const bool last = j == n - 1;
        // dV (+)= P^T dO; dO(i) has no later use, so its stage is released
        // behind it.  A new segment's sums start when the last's are read out.
        ok = wait(sb + BAR_P, i & 1) && (j > 0 || wait(sb + BAR_ACCE, (seg & 1) ^ 1));
        if (!ok) break;
        issue_acc(tmem + 256, tmem, dOmn + stage_off(i % OS), j > 0, sb + BAR_OE + 8 * (i % OS));
        if (!last) {   // P^T(i) is consumed in order before S^T(i+1) overwrites it
          const int qs1 = (i + 1) % QS;
          if (!(ok = wait(sb + BAR_QF + 8 * qs1, ((i + 1) / QS) & 1))) break;
          issue_ss(tmem, dK, dQk + stage_off(qs1), sb + BAR_S);
        }
        // dK (+)= dS^T Q
        if (!(ok = wait(sb + BAR_DS, i & 1))) break;
        issue_acc(tmem + 256 + D, tmem + 128, dQmn + stage_off(i % QS), j > 0, sb + BAR_QE + 8 * (i % QS));
        if (!last) {
          if (!(ok = dp(i + 1, j + 1 == n - 1))) break;
        } else {
          commit(sb + BAR_ACC);
          // the next segment's first products run while dV and dK are read out
          if (later && !(ok = first_s(i + 1, seg + 1) && dp(i + 1, R.n == 1))) break;
        }
      }
    }
    commit(sb + BAR_TAIL);
    if (lane == 0) mbar_wait(sb + BAR_TAIL, 0, 0u, tmo, SITE_TAIL);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ row threads (two per key)
    const int quad = warp & 3;                 // TMEM lane group of this warp
    const int half = (warp - 2) >> 2;          // which 64 queries of the walked tile
    const int col0 = half * 64;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_base + col0;
    const uint32_t tDP = tmem + lane_base + 128 + col0;
    const uint32_t tDV = tmem + lane_base + 256;
    const uint32_t tDK = tmem + lane_base + 256 + D;
    const float c = p.scale_log2;
    bool ok = true;
    // LSE and Delta of the walked Q tile, per query, go through shared memory
    // (two buffers in turn, barrier BAR_VEC): one value per first-half thread,
    // loaded two steps ahead, published one step ahead, at a point where every
    // warp has left the step that used the buffer before.  The loaded values
    // are not touched until then: arithmetic on them would wait for the load
    // in the middle of a step (some 1000 cycles of one).
    CrossRun V = R;                  // the walk as the vectors see it, and the step in its segment
    int vw = R.w;
    float nl = INFINITY, nd = 0.f;
    auto load_vec = [&]() {          // of the next walk step in turn
      const int hg = p.by_q_tiles.div(p.w0 + vw);
      const int q = (p.w0 + vw - hg * p.q_tiles) * 128 + row;
      const size_t at = (static_cast<size_t>(V.b) * p.H + V.hk * group + hg) * p.Sq + q;
      nl = INFINITY;
      nd = 0.f;
      if (q < p.Sq) {
        nl = __ldg(p.lse + at);
        nd = __ldg(p.delta + at);
      }
      if (++vw == V.w + V.n) {
        V.next(p);
        vw = V.w;
      }
    };
    auto publish_vec = [&](int i) {
      if (half == 0) {
        const uint32_t vec = sb + L::kOffVec + (i & 1) * 1024;
        // log2-domain LSE; a query past the sequence, or one whose LSE is -inf
        // (it saw nothing), gets +inf, i.e. P = 0
        st_shared_f32(vec + 4 * row, nl == -INFINITY ? INFINITY : nl * 1.4426950408889634f);
        st_shared_f32(vec + 512 + 4 * row, nd);
        if (i + 1 < steps) load_vec();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sb + BAR_VEC);
    };
    if (steps > 0) {
      if (half == 0) load_vec();
      publish_vec(0);
    }
    const uint32_t ds_part = static_cast<uint32_t>(quad * 8192 + half * 4096);
    const uint32_t ds_stage = sb + L::kOffStaging + ds_part;
    const size_t ds_step = static_cast<size_t>(p.k_tiles) * kBwdDsTileBytes;   // consecutive steps' tiles
    int i = 0, seg = 0;
    for (; ok && R.left > 0; R.next(p), ++seg) {
      const bool seen = row < R.len - R.kt * 128;   // a state behind the length: P and dS exactly 0
      unsigned char *ds_dst = p.ds + cross_ds_tile(p, R.bh_local, R.w, R.kt) + ds_part;
      for (int j = 0; j < R.n; ++j, ++i, ds_dst += ds_step) {
        const uint32_t vec = sb + L::kOffVec + (i & 1) * 1024;
        bool w = mbar_wait(sb + BAR_VEC, i & 1, abort_flag, tmo, SITE_SOFTMAX);
        if (__any_sync(0xffffffffu, !w)) { ok = false; break; }
        w = mbar_wait(sb + BAR_S, i & 1, abort_flag, tmo, SITE_SOFTMAX);
        if (__any_sync(0xffffffffu, !w)) { ok = false; break; }
        __syncwarp();
        tc_fence_after();
        uint32_t s[64];
        tmem_ld64_wait(tS, s);
        const float4 *lse4 = reinterpret_cast<const float4 *>(bwd_smem + (vec - sb)) + (col0 >> 2);
        const float4 *del4 = lse4 + 32;
#pragma unroll
        for (int q4 = 0; q4 < 16; ++q4) {
          const float4 l = lse4[q4];
          const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int q = 4 * q4 + e;
            const float pv = ex2_approx(__uint_as_float(s[q]) * c - lv[e]);
            s[q] = __float_as_uint(seen ? pv : 0.f);
          }
        }
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) pk[k] = pack_bf16x2(__uint_as_float(s[c0 + 2 * k]), __uint_as_float(s[c0 + 2 * k + 1]));
          tmem_st16(tS + c0 / 2, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + BAR_P);
        if (lane == 0) bulk_wait_read_all();     // the staging part is free once its last bulk store has read it
        w = mbar_wait(sb + BAR_DP, i & 1, abort_flag, tmo, SITE_SOFTMAX);
        if (__any_sync(0xffffffffu, !w)) { ok = false; break; }
        __syncwarp();
        tc_fence_after();
        // dP(i) was issued behind dS(i - 1) of every warp: the other vec buffer,
        // last read there, is free
        if (i + 1 < steps) publish_vec(i + 1);
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint32_t dp[32];
          tmem_ld32_wait(tDP + c0, dp);
          uint32_t pk[16];
#pragma unroll
          for (int k4 = 0; k4 < 8; ++k4) {
            const float4 dl = del4[(c0 >> 2) + k4];
            const int q = c0 + 4 * k4;
            auto ds_of = [&](int k, float d) {   // dP of a state behind the length may be NaN: replaced, not multiplied
              return seen ? __uint_as_float(s[q + k]) * (__uint_as_float(dp[4 * k4 + k]) - d) : 0.f;
            };
            pk[2 * k4] = pack_bf16x2(ds_of(0, dl.x), ds_of(1, dl.y));
            pk[2 * k4 + 1] = pack_bf16x2(ds_of(2, dl.z), ds_of(3, dl.w));
          }
          tmem_st16(tDP + c0 / 2, pk);
#pragma unroll
          for (int g = 0; g < 4; ++g)
            st_shared_v4(ds_stage + ((c0 >> 3) + g) * 512 + lane * 16, pk[4 * g], pk[4 * g + 1], pk[4 * g + 2],
                         pk[4 * g + 3]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + BAR_DS);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          bulk_store_hint(ds_dst, ds_stage, 4096, l2_evict_first_policy());
          bulk_commit();
        }
      }
      if (!ok) break;
      // ---- the segment's dV and dK: whole walks to the gradients (or the
      // range's sums), others to this CTA's first (the tile began before the
      // run) or second slot
      {
        const bool w = mbar_wait(sb + BAR_ACC, seg & 1, abort_flag, tmo, SITE_EPILOGUE);
        if (__any_sync(0xffffffffu, !w)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const int k = R.kt * 128 + row;
        const int d0 = half * (D / 2);   // each half of the row writes half of the D columns
        float *part_dst = R.n < p.walk
                              ? p.partial + (static_cast<size_t>(blockIdx.x) * 2 + (R.w > 0 ? 0 : 1)) * (2 * 128 * D)
                          : p.whole != nullptr ? p.whole + static_cast<size_t>(R.kt) * (2 * 128 * D)
                                               : nullptr;
        for (int which = 0; which < 2; ++which) {   // 0: dV, 1: dK (times the softmax scale)
          const float mul = which == 0 ? 1.0f : p.scale;
          const uint32_t tsrc = (which == 0 ? tDV : tDK) + d0;
#pragma unroll
          for (int c0 = 0; c0 < D / 2; c0 += 32) {
            uint32_t o[32];
            tmem_ld32_wait(tsrc + c0, o);
            if (part_dst != nullptr) {
              // [dV, dK][4-column piece][128 rows]: a warp's store is 512 contiguous bytes
              float4 *d4 = reinterpret_cast<float4 *>(part_dst + static_cast<size_t>(which) * 128 * D) + ((d0 + c0) >> 2) * 128 + row;
#pragma unroll
              for (int x = 0; x < 8; ++x)
                d4[x * 128] = make_float4(__uint_as_float(o[4 * x]) * mul, __uint_as_float(o[4 * x + 1]) * mul,
                                          __uint_as_float(o[4 * x + 2]) * mul, __uint_as_float(o[4 * x + 3]) * mul);
            } else if (k < p.Skv) {
              uint4 *d4 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(which == 0 ? p.dv : p.dk) +
                                                    ((static_cast<size_t>(R.b) * p.Skv + k) * p.Hk + R.hk) * D + d0 + c0);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                d4[x] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * x]) * mul, __uint_as_float(o[8 * x + 1]) * mul),
                                   pack_bf16x2(__uint_as_float(o[8 * x + 2]) * mul, __uint_as_float(o[8 * x + 3]) * mul),
                                   pack_bf16x2(__uint_as_float(o[8 * x + 4]) * mul, __uint_as_float(o[8 * x + 5]) * mul),
                                   pack_bf16x2(__uint_as_float(o[8 * x + 6]) * mul, __uint_as_float(o[8 * x + 7]) * mul));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + BAR_ACCE);
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kBwdTmemCols);
  }
}

// The tiles that runs share: dK and dV from the runs' float32 sums, the run
// that starts the tile first.  Tasks 2 c and 2 c + 1 (dV and dK) are the tile
// that the run of CTA c + 1 starts in, if that run is the first to start
// inside it.  A task is done by 128 threads, one a row.
template <int D>
__device__ __forceinline__ void cross_join(const CrossBwdParams &p, int task, long long total, const int *ends, int row) {
  const int which = task & 1, first = task >> 1;
  const long long cut = CrossRun::start(p, total, first + 1);   // where the run of CTA first + 1 starts
  const long long tile = CrossRun::over(cut, p.inv_walk), t0 = tile * p.walk;
  if (cut == t0 || CrossRun::start(p, total, first) > t0 || cut >= total) return;
  int last = first + 1;   // the runs first .. last share the tile
  while (last + 1 < p.ctas && CrossRun::start(p, total, last + 1) < t0 + p.walk) ++last;
  CrossRun R;
  R.left = 1;
  R.locate(p, static_cast<int>(tile), ends);
  const int k = R.kt * 128 + row;
  if (k >= p.Skv) return;
  uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(which == 0 ? p.dv : p.dk) +
                                         ((static_cast<size_t>(R.b) * p.Skv + k) * p.Hk + R.hk) * D);
#pragma unroll 1
  for (int c0 = 0; c0 < D / 4; c0 += 8) {   // 32 columns: eight 16-byte loads of a run in flight
    float4 acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = first; r <= last; ++r) {   // the first run's second slot, the others' first
      if (total < p.ctas && CrossRun::start(p, total, r) == CrossRun::start(p, total, r + 1)) continue;   // an empty run
      const float4 *src = reinterpret_cast<const float4 *>(p.partial) +
                          (((static_cast<size_t>(r) * 2 + (r == first ? 1 : 0)) * 2 + which) * (D / 4) + c0) * 128 + row;
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __ldcs(src + i * 128);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i].x += v[i].x;
        acc[i].y += v[i].y;
        acc[i].z += v[i].z;
        acc[i].w += v[i].w;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = acc[2 * i], y = acc[2 * i + 1];
      dst[c0 / 2 + i] = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    }
  }
}

// A pair in ranges: each tile's sum over the ranges so far, the first range's
// first, and after the last range the gradients.  A CTA a K tile, and dV or dK.
template <int D>
__global__ void __launch_bounds__(128) cross_range_kernel(const __grid_constant__ CrossBwdParams p) {
  const int kt = static_cast<int>(blockIdx.x >> 1), which = static_cast<int>(blockIdx.x & 1), row = static_cast<int>(threadIdx.x);
  const int b = p.by_hk.div(p.bh0), hk = p.bh0 - b * p.Hk;
  const int n_kt = (cross_bwd_len(p, b) + 127) / 128;
  if (kt >= n_kt) return;              // zeros, written beside the dQ product
  const long long total = static_cast<long long>(n_kt) * p.walk, t0 = static_cast<long long>(kt) * p.walk;
  // the runs first .. last share the tile (the quotient is that run or the one before it)
  int first = static_cast<int>(t0 * p.ctas / total);
  while (first + 1 < p.ctas && CrossRun::start(p, total, first + 1) <= t0) ++first;
  int last = first;
  while (last + 1 < p.ctas && CrossRun::start(p, total, last + 1) < t0 + p.walk) ++last;
  const int k = kt * 128 + row;
  for (int c = 0; c < D / 4; ++c) {
    const size_t at = ((static_cast<size_t>(kt) * 2 + which) * (D / 4) + c) * 128 + row;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!p.first_range) a = reinterpret_cast<const float4 *>(p.sums)[at];
    for (int r = first; r <= last; ++r) {
      if (total < p.ctas && CrossRun::start(p, total, r) == CrossRun::start(p, total, r + 1)) continue;   // an empty run
      const float4 v = first == last
                           ? reinterpret_cast<const float4 *>(p.whole)[at]
                           : reinterpret_cast<const float4 *>(p.partial)
                                 [(((static_cast<size_t>(r) * 2 + (r == first ? 1 : 0)) * 2 + which) * (D / 4) + c) * 128 + row];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    if (!p.last_range)
      reinterpret_cast<float4 *>(p.sums)[at] = a;
    else if (k < p.Skv)
      reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(which == 0 ? p.dv : p.dk) +
                                ((static_cast<size_t>(b) * p.Skv + k) * p.Hk + hk) * D)[c] =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

// ============================================================== dQ product
// dQ = dS K * scale, one CTA per SM walking (pair, head, Q tile) units; the
// pipeline of attn_bwd_dq_gemm_kernel, with a third barrier per stage for the
// zeroed rows of K behind the length, and zeros for elements without states.
// Bound by the reads of dS, it has warps to spare for the join of the dK and
// dV tiles that runs share (as a launch of its own 13 to 15 us).
template <int D>
struct CrossGemmSmem {
  static constexpr int kATile = kBwdDsTileBytes;
  static constexpr int kBTile = BwdSmem<D>::kTileBytes;
  static constexpr int kStage = kATile + kBTile;
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kNumBars = 3 * kStages + 5;          // full[S], empty[S], clean[S], acc_full[2], acc_empty[2], tail
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAllocBytes = kBytes;
};
static_assert(CrossGemmSmem<128>::kAllocBytes + 4 * kCrossMaxKTiles <= 232448 &&
                  CrossGemmSmem<64>::kAllocBytes + 4 * kCrossMaxKTiles <= 232448, "shared memory");
constexpr int kCrossGemmThreads = 352;   // producer, MMA, four epilogue warps, one that zeroes K's padding, four that join

template <int D>
__global__ void __launch_bounds__(kCrossGemmThreads, 1) cross_bwd_dq_kernel(const __grid_constant__ CrossBwdParams p) {
  using L = CrossGemmSmem<D>;
  using T = BwdSmem<D>;
  constexpr uint32_t IDESC = idesc_bf16_f32(128, D, true, true);   // dS and K both MN-major
  constexpr uint32_t kAccCols = 2 * D;
  extern __shared__ __align__(1024) uint8_t bwd_smem[];
  const uint32_t sb = smem_u32(bwd_smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_device_status, SITE_LAYOUT);
    return;
  }
  constexpr int ST = L::kStages;
  constexpr uint32_t BAR_FULL = L::kOffBar;                 // [ST] stage loaded
  constexpr uint32_t BAR_EMPTY = BAR_FULL + 8 * ST;         // [ST] stage consumed by the MMAs
  constexpr uint32_t BAR_CLEAN = BAR_EMPTY + 8 * ST;        // [ST] K's padding rows zeroed
  constexpr uint32_t BAR_AF = BAR_CLEAN + 8 * ST;           // [2] accumulator complete
  constexpr uint32_t BAR_AE = BAR_AF + 16;                  // [2] accumulator read out
  constexpr uint32_t BAR_TAIL = BAR_AE + 16;
  constexpr uint32_t TMEM_SLOT = L::kOffMisc;
  constexpr uint32_t ABORT = L::kOffMisc + 4;
  static_assert(BAR_TAIL + 8 <= L::kOffMisc, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;
  const int group = p.H / p.Hk;
  const int units = p.n_bh * p.walk;                        // (head of the group, Q tile) units of the pairs
  const bool cleans = p.kv_lens != nullptr;
  struct Unit {
    int b, hk, h, qt, len, n, bh_local, w;
  };
  auto unit_at = [&](int i) {
    Unit u;
    u.bh_local = p.by_walk.div(i);
    u.w = i - u.bh_local * p.walk;
    const int hg = p.by_q_tiles.div(p.w0 + u.w);
    u.qt = p.w0 + u.w - hg * p.q_tiles;
    const int bh = p.bh0 + u.bh_local;
    u.b = p.by_hk.div(bh);
    u.hk = bh - u.b * p.Hk;
    u.h = u.hk * group + hg;
    u.len = cross_bwd_len(p, u.b);
    u.n = (u.len + 127) / 128;
    return u;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(sb + BAR_FULL + 8 * s, 1);
      mbar_init(sb + BAR_EMPTY + 8 * s, 1);
      mbar_init(sb + BAR_CLEAN + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(sb + BAR_AF + 8 * a, 1);
      mbar_init(sb + BAR_AE + 8 * a, 4);   // one arrival per epilogue warp
    }
    mbar_init(sb + BAR_TAIL, 1);
    st_shared_volatile(sb + ABORT, 0u);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + TMEM_SLOT, kAccCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_volatile(sb + TMEM_SLOT);
  const uint32_t abort_flag = sb + ABORT;
  const int first = blockIdx.x, step = gridDim.x;
  int *const ends = reinterpret_cast<int *>(bwd_smem + L::kBytes);   // [k_tiles] with lengths
  const long long total = cross_total_steps(p, ends);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_k);
      const uint64_t once = l2_evict_first_policy();
      int it = 0;
      bool ok = true;
      for (int i = first; ok && i < units; i += step) {
        const Unit U = unit_at(i);
        const unsigned char *a0 = p.ds + cross_ds_tile(p, U.bh_local, U.w, 0);
        for (int j = 0; j < U.n; ++j, ++it) {
          const int st = it % ST;
          if (!mbar_wait(sb + BAR_EMPTY + 8 * st, ((it / ST) & 1) ^ 1, abort_flag, tmo, SITE_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t full = sb + BAR_FULL + 8 * st;
          const uint32_t dst = sb + st * L::kStage;
          mbar_arrive_expect_tx(full, L::kStage);
          bulk_load_hint(dst, a0 + static_cast<size_t>(j) * kBwdDsTileBytes, L::kATile, full, once);
          for (int hf = 0; hf < T::kHalves; ++hf)
            tma_load_4d(dst + L::kATile + hf * T::kBoxBytes, &p.tm_k, hf * 64, U.hk, j * 128, U.b, full);
        }
      }
      for (int j = 0; j < ST && j < it; ++j) {
        const int i = it - 1 - j;
        mbar_wait(sb + BAR_EMPTY + 8 * (i % ST), (i / ST) & 1, 0u, tmo, SITE_TAIL);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int it = 0, local = 0;
      bool ok = true;
      for (int i = first; ok && i < units; i += step) {
        const Unit U = unit_at(i);
        if (U.n == 0) continue;
        const int a = local & 1;
        const uint32_t use = static_cast<uint32_t>(local >> 1);
        ++local;
        if (!mbar_wait_spin(sb + BAR_AE + 8 * a, (use & 1) ^ 1, abort_flag, tmo, SITE_MMA)) break;
        tc_fence_after();
        const uint32_t d = tmem + a * D;
        for (int j = 0; j < U.n; ++j, ++it) {
          const int st = it % ST;
          ok = mbar_wait_spin(sb + BAR_FULL + 8 * st, (it / ST) & 1, abort_flag, tmo, SITE_MMA);
          if (ok && cleans) ok = mbar_wait_spin(sb + BAR_CLEAN + 8 * st, (it / ST) & 1, abort_flag, tmo, SITE_MMA);
          if (!ok) break;
          tc_fence_after();
          // the operands' layouts as in attn_bwd_dq_gemm_kernel
          const uint64_t da = opaque_u64(smem_desc_plain(sb + st * L::kStage, 128, 512));
          const uint64_t db = opaque_u64(smem_desc_sw128(sb + st * L::kStage + L::kATile, T::kBoxBytes, 1024));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(d, da + ((((kk >> 1) * 8192) + (kk & 1) * 256) >> 4), db + ((kk * 2048) >> 4), IDESC,
                   (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(sb + BAR_EMPTY + 8 * st);
        }
        if (ok) mma_commit(sb + BAR_AF + 8 * a);
      }
      mma_commit(sb + BAR_TAIL);
      mbar_wait(sb + BAR_TAIL, 0, 0u, tmo, SITE_TAIL);
    }
  } else if (warp > 6) {
    // ------------------------------------------------------------ shared dK, dV tiles
    for (int task = first; p.sums == nullptr && task < 2 * (p.ctas - 1); task += step)
      cross_join<D>(p, task, total, ends, static_cast<int>(threadIdx.x) - 224);
  } else if (warp == 6) {
    // ------------------------------------------------------------ K padding
    if (cleans) {
      int it = 0;
      bool ok = true;
      for (int i = first; ok && i < units; i += step) {
        const Unit U = unit_at(i);
        for (int j = 0; j < U.n; ++j, ++it) {
          const int st = it % ST;
          const bool w = mbar_wait(sb + BAR_FULL + 8 * st, (it / ST) & 1, abort_flag, tmo, SITE_PRODUCER);
          if (__any_sync(0xffffffffu, !w)) {
            ok = false;
            break;
          }
          const int valid = U.len - j * 128;
          if (valid < 128) {
            const int chunks = (128 - valid) * 8;
            for (int hf = 0; hf < T::kHalves; ++hf)
              for (int x = lane; x < chunks; x += 32)
                st_shared_v4(sb + st * L::kStage + L::kATile + hf * T::kBoxBytes + valid * 128 + x * 16, 0u, 0u, 0u, 0u);
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sb + BAR_CLEAN + 8 * st);
        }
      }
      // dK and dV of tiles wholly behind the length: zeros
      for (int t = first; t < p.n_bh * p.k_tiles; t += step) {
        const int bh_local = t / p.k_tiles, k0 = (t - bh_local * p.k_tiles) * 128;
        const int bh = p.bh0 + bh_local, b = p.by_hk.div(bh), hk = bh - b * p.Hk;
        if (k0 < cross_bwd_len(p, b)) continue;
        constexpr int kVec = D / 8;                  // 16-byte pieces of a row
        for (int i = lane; i < min(128, p.Skv - k0) * kVec; i += 32) {
          const size_t at = ((static_cast<size_t>(b) * p.Skv + k0 + i / kVec) * p.Hk + hk) * kVec + i % kVec;
          static_cast<uint4 *>(p.dk)[at] = make_uint4(0u, 0u, 0u, 0u);
          static_cast<uint4 *>(p.dv)[at] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;   // accumulator row = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    int local = 0;
    for (int i = first; i < units; i += step) {
      const Unit U = unit_at(i);
      const int a = local & 1;
      if (U.n > 0) {
        const uint32_t use = static_cast<uint32_t>(local >> 1);
        ++local;
        const bool w = mbar_wait(sb + BAR_AF + 8 * a, use & 1, abort_flag, tmo, SITE_EPILOGUE);
        if (__any_sync(0xffffffffu, !w)) break;
        __syncwarp();
        tc_fence_after();
      }
      const int q = U.qt * 128 + r;
      const bool row_ok = q < p.Sq;
      __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.dq) +
                           ((static_cast<size_t>(U.b) * p.Sq + (row_ok ? q : 0)) * p.H + U.h) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        __syncwarp();
        if (U.n > 0) {
          tmem_ld32_wait(tmem + lane_base + a * D + c, v);   // the whole warp, converged
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = 0u;
        }
        if (!row_ok) continue;
        uint4 *d4 = reinterpret_cast<uint4 *>(dst + c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d4[k] = make_uint4(
              pack_bf16x2(__uint_as_float(v[8 * k]) * p.scale, __uint_as_float(v[8 * k + 1]) * p.scale),
              pack_bf16x2(__uint_as_float(v[8 * k + 2]) * p.scale, __uint_as_float(v[8 * k + 3]) * p.scale),
              pack_bf16x2(__uint_as_float(v[8 * k + 4]) * p.scale, __uint_as_float(v[8 * k + 5]) * p.scale),
              pack_bf16x2(__uint_as_float(v[8 * k + 6]) * p.scale, __uint_as_float(v[8 * k + 7]) * p.scale));
      }
      if (U.n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + BAR_AE + 8 * a);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kAccCols);
  }
}

}  // namespace cpattn
