// operators_internal.h -- launch plans of the operators around the attention,
// shared by the host code and the kernels.  Not part of the public ABI.
#pragma once

#include "cpattn_internal.h"

namespace cpattn {

// ------------------------------------------------ norm and rotation of Q and K
struct NormRopeTensor {
  const __nv_bfloat16 *x;      // [B, S, H, D], unit stride in D
  __nv_bfloat16 *y;
  long long xb, xs, xh;        // strides in elements
  long long yb, ys, yh;
  int H;
};
struct NormRopeGrad {
  const __nv_bfloat16 *x;
  long long b, s, h;
};
struct NormRopeParams {
  NormRopeTensor t[2];         // queries, keys (H = 0: absent)
  NormRopeGrad dy[2];          // backward: the upstream gradients
  const void *w[2];            // [D] or null
  const float *cos, *sin;      // [n_pos, rot / 2]
  const int *positions;        // [B, S] or null (token s at position pos0 + s)
  float *partial;              // backward: the CTAs' weight-gradient sums, or null
  int w_f32;
  int B, S;
  int rot, n_pos, pos0;
  int heads_per_warp;
  int chunks[2];               // blocks of heads_per_warp heads of each tensor
  float eps;
};
constexpr int kNormMaxBlocks = 148 * 8;   // CTAs of a backward launch at most: rows of `partial`

// Division of an n in 0 .. 2^31 - 1 by a divisor known at launch, as a
// multiplication and a shift (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (floor(m n / 2^32) + n) >> s.  A
// persistent kernel's roles decode a unit between two tiles, where a division
// instruction sequence of a lone thread costs some 400 cycles.
struct FastDiv {
  unsigned m, s;
  int d;
  void set(int divisor) {
    d = divisor;
    s = 0;
    while ((1ull << s) < static_cast<unsigned long long>(d)) ++s;
    m = static_cast<unsigned>(((1ull << 32) * ((1ull << s) - static_cast<unsigned long long>(d))) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(m, static_cast<unsigned>(n)) + static_cast<unsigned>(n)) >> s);
  }
};

// --------------------------------------------------------- cross attention
// Queries [B, Sq, H, D] against an encoder's states [B, Skv, Hk, D], the first
// kv_lens[b] of them (all: null); query head h uses key head h / (H / Hk).
struct alignas(64) CrossParams {
  // 4-D maps over [B, rows, heads, D] bf16, 128B swizzle; boxes {64, 1, 128, 1},
  // with packed heads {64, group, 128 / group, 1} for q, and a fourth of q's
  // rows for out
  CUtensorMap tm_q, tm_k, tm_v, tm_out;
  __nv_bfloat16 *out;             // [B, Sq, H, D] (split units' joined rows)
  float *lse;                     // [B, H, Sq] or null
  const int *kv_lens;             // [B] device, or null
  int B, Sq, Skv, H, Hk;
  int group;                      // heads of a group, H / Hk
  int pack_log2;                  // log2 of the heads that share a tile's rows (0: one head a tile)
  int q_tiles;                    // tiles of a head's (or the packed heads') queries
  int group_tiles;                // (head or packed heads, tile) entries of a key head
  int pairs;                      // pairs of them
  int units;                      // B * Hk * pairs
  FastDiv by_pairs, by_hk, by_q_tiles;
  int splits;                     // CTAs (a cluster) that share a unit's key tiles
  float scale_log2;
  unsigned long long timeout_ns;
};

// The same with few query rows a key head (all heads of its group together).
struct alignas(64) CrossTokenParams {
  CUtensorMap tm_k, tm_v;         // 4-D maps over [B, Skv, Hk, D] bf16, box {64, 1, 64, 1}, 128B swizzle
  const __nv_bfloat16 *q;
  long long qb, qs, qh;           // strides in elements
  __nv_bfloat16 *out;
  float *lse;
  const int *kv_lens;
  int B, Sq, Skv, H, Hk;
  int splits;                     // CTAs (a cluster) that share a unit's states
  float scale_log2;
  unsigned long long timeout_ns;
};
// Row sums Delta of the gradient.
struct CrossDeltaParams {
  const __nv_bfloat16 *q, *k, *v;        // [B, rows, heads, D] views, strides in elements
  long long qb, qs, qh, kb, ks, kh, vb, vs, vh;
  const __nv_bfloat16 *out, *dout;       // [B, Sq, H, D]
  const float *lse;                      // [B, H, Sq]
  float *delta;
  const int *kv_lens;
  int B, Sq, Skv, H, Hk;
  int blocks;                            // 16-row blocks of a key head's query rows
  int chunk_blocks, chunks;              // of them a CTA at a time, chunks of a key head
  FastDiv by_chunks, by_hk, by_group, by_element;   // (by_element: H * Sq rows)
  float scale_log2;
};
// Its gradient over the (batch element, key head) pairs [bh0, bh0 + n_bh).
struct alignas(64) CrossBwdParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;   // 4-D maps as above
  const float *lse, *delta;              // [B, H, Sq]
  const int *kv_lens;
  void *dq, *dk, *dv;                    // bf16, contiguous
  unsigned char *ds;                     // dS tiles of the pairs (cross_ds_tile), 256-byte aligned
  float *partial;                        // sums of tiles that runs share: [CTA][first, last tile][dV, dK][D / 4][128][4]
  // A pair in ranges of its walk (one pair a launch; else null): the ranges'
  // sums, and this range's of tiles that one run covers, both [K tile][dV, dK][D / 4][128][4]
  float *sums, *whole;
  int w0, first_range, last_range;       // first step of the range
  int B, Sq, Skv, H, Hk;
  int bh0, n_bh;
  int q_tiles, k_tiles;
  int walk;                              // steps of a K/V tile: the Q tiles of its group's heads (or a range of them)
  int ctas;                              // runs that the valid tiles' walks are cut into
  double inv_ctas, inv_walk;
  FastDiv by_walk, by_hk, by_q_tiles;
  float scale, scale_log2;
  unsigned long long timeout_ns;
};
// CTAs of the dK/dV launch at most: their sums are the workspace's (at D = 128,
// 256 KB each).
constexpr int kCrossMaxRuns = 148;
// K tiles at most: the dK/dV kernel counts pairs by their last in its 32 KB dS
// tile.
constexpr int kCrossMaxKTiles = kBwdDsTileBytes / 4;

}  // namespace cpattn
