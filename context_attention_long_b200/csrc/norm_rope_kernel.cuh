// norm_rope_kernel.cuh -- RMS norm of queries and keys for each head, with the
// position rotation in the same pass, and its gradient.
//
// Per (token, head) row x of D elements, in float32:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x * r,  m = n * w  (w absent: 1)
//   y = R m: the first `rot` elements turned pair by pair by the token's
//   angles, y_a = m_a cos - m_b sin, y_b = m_b cos + m_a sin, for the pairs
//   (2i, 2i + 1) or (i, i + rot / 2); the others unchanged.
// Gradient: dm = R^T dy (the opposite turn), g = dm * w,
//   dx = r * (g - n * mean(g * n)),  dw = sum over rows of dm * n.
// The norm's scale is computed again from x, which the gradient reads anyway,
// so the forward keeps nothing for it.
//
// HBM-bound: 4 bytes an element forward, 6 backward.  A row is D / 8 lanes
// with one 16-byte piece each; a warp keeps one (tensor, block of heads) and
// walks tokens, so that the weights stay in registers and a token's angles are
// read once for all heads of the block; the loads of kU passes (with few heads,
// of consecutive tokens) are issued before any is used.  dw: every lane sums its
// 8 columns over the rows of its walk, then lanes, warps and CTAs are added in a
// fixed order (no atomics: the same bytes every run), the CTAs' sums by a second
// small kernel.
#pragma once

#include "operators_internal.h"
#include "operators_ptx.cuh"

namespace cpattn {

// Device status bit: a position outside the rotation table (its row is NaN).
constexpr unsigned int SITE_POSITION = 1u << 7;

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;

enum NormRotation : int { kNoRotation = 0, kPairs = 1, kHalves = 2 };

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// What a warp keeps over its walk: its tensor, its heads and its lane's part
// of a row.
template <int D>
struct NormWalk {
  static constexpr int LPR = D / 8;      // lanes per row
  static constexpr int RPP = 32 / LPR;   // rows per pass of a warp
  int lane, sub, c;                      // row of the pass, 16-byte piece of the row
  int ti, h0, h1;                        // tensor, its heads [h0, h1)
  int ch;                                // the block among its tensor's
  unsigned token, token_stride;

  __device__ __forceinline__ bool init(const NormRopeParams &p) {
    lane = threadIdx.x & 31;
    sub = lane / LPR;
    c = lane - sub * LPR;
    const unsigned gw = blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    const unsigned nch = static_cast<unsigned>(p.chunks[0] + p.chunks[1]);
    const unsigned walks = gridDim.x * kNormWarps / nch;   // whole sets of chunks
    token_stride = walks;
    token = gw / nch;
    ch = static_cast<int>(gw - token * nch);
    if (token >= walks) return false;
    ti = ch >= p.chunks[0] ? 1 : 0;
    if (ti) ch -= p.chunks[0];
    h0 = ch * p.heads_per_warp;
    h1 = min(p.t[ti].H, h0 + p.heads_per_warp);
    return true;
  }
  // Few heads (a block a head): the tensor's warps share its (token, head)
  // rows, kT passes of consecutive ones at a time.  First row and step of the
  // walk, and row r's place.
  template <int kT>
  __device__ __forceinline__ unsigned first_row(int H) const { return (token * H + ch) * (RPP * kT); }
  template <int kT>
  __device__ __forceinline__ unsigned row_step(int H) const { return token_stride * H * (RPP * kT); }
  __device__ __forceinline__ static void place(const NormRopeParams &p, int H, unsigned r, int &b, int &s, int &h) {
    const unsigned t = r / static_cast<unsigned>(H);
    h = static_cast<int>(r - t * H);
    b = static_cast<int>(t / p.S);
    s = static_cast<int>(t - static_cast<unsigned>(b) * p.S);
  }
};

__device__ __forceinline__ void norm_weights(const NormRopeParams &p, int ti, int c, float (&w)[8]) {
  const void *src = p.w[ti];
  if (src == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (p.w_f32) {
    const float4 a = reinterpret_cast<const float4 *>(src)[2 * c], b = reinterpret_cast<const float4 *>(src)[2 * c + 1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else {
    unpack8(reinterpret_cast<const uint4 *>(src)[c], w);
  }
}

// The angles of one token for this lane's piece.  kPairs: cs[i], sn[i] (i < 4)
// turn the pair (2i, 2i + 1).  kHalves: element i pairs with element i of the
// partner lane's piece, out = own * cs + other * sn (sn negated for the first
// half).  Pieces past the rotated part turn by nothing.
template <int ROT>
struct NormAngles {
  static constexpr int kN = ROT == kPairs ? 4 : 8;
  float cs[kN], sn[kN];
  __device__ __forceinline__ void load(const NormRopeParams &p, int b, int s, int c, int half_pieces) {
    int pos = p.positions != nullptr ? p.positions[static_cast<long long>(b) * p.S + s] : p.pos0 + s;
    const bool turned = c < 2 * half_pieces;
    const bool inside = pos >= 0 && pos < p.n_pos;
    if (turned && inside) {
      const int first = ROT == kPairs ? 4 * c : 8 * (c < half_pieces ? c : c - half_pieces);
      const long long at = static_cast<long long>(pos) * (8 * half_pieces) + first;
      const float4 *pc = reinterpret_cast<const float4 *>(p.cos + at), *ps = reinterpret_cast<const float4 *>(p.sin + at);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float4 a = __ldg(pc + i), d = __ldg(ps + i);
        cs[4 * i] = a.x; cs[4 * i + 1] = a.y; cs[4 * i + 2] = a.z; cs[4 * i + 3] = a.w;
        sn[4 * i] = d.x; sn[4 * i + 1] = d.y; sn[4 * i + 2] = d.z; sn[4 * i + 3] = d.w;
      }
      if (ROT == kHalves && c < half_pieces) {
#pragma unroll
        for (int i = 0; i < kN; ++i) sn[i] = -sn[i];
      }
    } else {
      // a piece behind the rotated part, or a position outside the table: NaN
      // over its whole row, the pieces behind the rotated part too
      const float one = inside ? 1.f : __int_as_float(0x7fffffff);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        cs[i] = one;
        sn[i] = turned ? one : 0.f;
      }
      if (turned && c == 0) atomicOr(&g_device_status, SITE_POSITION);
    }
  }
  // v <- R v (kInverse: R^T v).  Every lane of the warp takes part.
  template <bool kInverse>
  __device__ __forceinline__ void turn(float (&v)[8], int partner) const {
    if constexpr (ROT == kPairs) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        const float t = kInverse ? -sn[i] : sn[i];
        v[2 * i] = a * cs[i] - b * t;
        v[2 * i + 1] = b * cs[i] + a * t;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, v[i], partner);
        v[i] = v[i] * cs[i] + o * (kInverse ? -sn[i] : sn[i]);
      }
    }
  }
};
template <>
struct NormAngles<kNoRotation> {
  __device__ __forceinline__ void load(const NormRopeParams &, int, int, int, int) {}
  template <bool kInverse>
  __device__ __forceinline__ void turn(float (&)[8], int) const {}
};

// The lane whose piece pairs with this lane's under kHalves (itself, where
// the piece is not turned).
template <int D>
__device__ __forceinline__ int norm_partner(const NormWalk<D> &W, int half_pieces) {
  const int base = W.sub * NormWalk<D>::LPR;
  if (W.c < half_pieces) return base + W.c + half_pieces;
  if (W.c < 2 * half_pieces) return base + W.c - half_pieces;
  return W.lane;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One row piece: v <- the rotation of v * r * w.
template <int D, int ROT>
__device__ __forceinline__ void norm_row(float (&v)[8], const float (&w)[8], float eps, const NormAngles<ROT> &A,
                                         int partner) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
  const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
  A.template turn<false>(v, partner);
}
// Its gradient: v <- dx from x (v) and dy (g); dw[i] += dm * n where `there`.
template <int D, int ROT>
__device__ __forceinline__ void norm_row_bwd(float (&v)[8], float (&g)[8], const float (&w)[8], float (&dw)[8], bool there,
                                             float eps, const NormAngles<ROT> &A, int partner) {
  A.template turn<true>(g, partner);
  float ss = 0.f, gx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ss = fmaf(v[i], v[i], ss);
    gx = fmaf(g[i] * w[i], v[i], gx);
  }
  const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + eps);
  const float mean_gn = row_sum<D / 8>(gx) * r * (1.f / D);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = v[i] * r;
    v[i] = r * (g[i] * w[i] - n * mean_gn);
    if (there) dw[i] = fmaf(g[i], n, dw[i]);   // a row that is not there adds nothing, NaN angles or not
  }
}

// kT = 1: a token at a time, kU passes of its heads; kT > 1 (few heads): kT
// passes of consecutive (token, head) rows, each lane with its row's angles.
template <int D, int ROT, int kU, int kT>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using Walk = NormWalk<D>;
  Walk W;
  if (!W.init(p)) return;
  const NormRopeTensor &T = p.t[W.ti];
  const int half_pieces = p.rot >> 4;
  const int partner = norm_partner<D>(W, half_pieces);
  float w[8];
  norm_weights(p, W.ti, W.c, w);
  const unsigned tokens = static_cast<unsigned>(p.B) * p.S;
  if constexpr (kT > 1) {
    const unsigned rows = tokens * T.H;
    for (unsigned r0 = W.template first_row<kT>(T.H); r0 < rows; r0 += W.template row_step<kT>(T.H)) {
      NormAngles<ROT> A[kT];
      uint4 raw[kT];
      __nv_bfloat16 *y[kT];
#pragma unroll
      for (int u = 0; u < kT; ++u) {
        const unsigned r = r0 + u * Walk::RPP + W.sub;
        int b, s, h;
        Walk::place(p, T.H, min(r, rows - 1), b, s, h);
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(T.x + b * T.xb + s * T.xs + h * T.xh + 8 * W.c));
        y[u] = r < rows ? T.y + b * T.yb + s * T.ys + h * T.yh + 8 * W.c : nullptr;
        A[u].load(p, b, s, W.c, half_pieces);
      }
#pragma unroll
      for (int u = 0; u < kT; ++u) {
        float v[8];
        unpack8(raw[u], v);
        norm_row<D>(v, w, p.eps, A[u], partner);
        if (y[u] != nullptr) *reinterpret_cast<uint4 *>(y[u]) = pack8(v);
      }
    }
    return;
  }
  for (unsigned t = W.token; t < tokens; t += W.token_stride) {
    const int b = static_cast<int>(t / p.S), s = static_cast<int>(t - static_cast<unsigned>(b) * p.S);
    const __nv_bfloat16 *x = T.x + b * T.xb + s * T.xs + 8 * W.c + (W.h0 + W.sub) * T.xh;
    __nv_bfloat16 *y = T.y + b * T.yb + s * T.ys + 8 * W.c + (W.h0 + W.sub) * T.yh;
    NormAngles<ROT> A;
    A.load(p, b, s, W.c, half_pieces);
    for (int h = W.h0 + W.sub; h < W.h1 + W.sub; h += kU * Walk::RPP, x += kU * Walk::RPP * T.xh, y += kU * Walk::RPP * T.yh) {
      uint4 raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h + u * Walk::RPP < W.h1) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(x + u * Walk::RPP * T.xh));
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float v[8];
        unpack8(raw[u], v);
        norm_row<D>(v, w, p.eps, A, partner);
        if (h + u * Walk::RPP < W.h1) *reinterpret_cast<uint4 *>(y + u * Walk::RPP * T.yh) = pack8(v);
      }
    }
  }
}

// p.t[i].x: the forward's input, p.t[i].y: dx; p.dy[i]: the upstream gradient.
// partial: [gridDim.x][2][D] sums of dm * n for the two tensors.
template <int D, int ROT, int kU, int kT>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  using Walk = NormWalk<D>;
  __shared__ float sums[kNormWarps][D];
  __shared__ int tensor_of[kNormWarps];
  Walk W;
  const bool working = W.init(p);
  float dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  if (working) {
    const NormRopeTensor &T = p.t[W.ti];
    const NormRopeGrad &G = p.dy[W.ti];
    const int half_pieces = p.rot >> 4;
    const int partner = norm_partner<D>(W, half_pieces);
    float w[8];
    norm_weights(p, W.ti, W.c, w);
    const unsigned tokens = static_cast<unsigned>(p.B) * p.S;
    if constexpr (kT > 1) {
      const unsigned rows = tokens * T.H;
      for (unsigned r0 = W.template first_row<kT>(T.H); r0 < rows; r0 += W.template row_step<kT>(T.H)) {
        NormAngles<ROT> A[kT];
        uint4 rx[kT], rg[kT];
        __nv_bfloat16 *dx[kT];
#pragma unroll
        for (int u = 0; u < kT; ++u) {
          const unsigned r = r0 + u * Walk::RPP + W.sub;
          int b, s, h;
          Walk::place(p, T.H, min(r, rows - 1), b, s, h);
          rx[u] = make_uint4(0u, 0u, 0u, 0u);
          rg[u] = rx[u];
          if (r < rows) {
            rx[u] = __ldcs(reinterpret_cast<const uint4 *>(T.x + b * T.xb + s * T.xs + h * T.xh + 8 * W.c));
            rg[u] = __ldcs(reinterpret_cast<const uint4 *>(G.x + b * G.b + s * G.s + h * G.h + 8 * W.c));
          }
          dx[u] = r < rows ? T.y + b * T.yb + s * T.ys + h * T.yh + 8 * W.c : nullptr;
          A[u].load(p, b, s, W.c, half_pieces);
        }
#pragma unroll
        for (int u = 0; u < kT; ++u) {
          float v[8], g[8];
          unpack8(rx[u], v);
          unpack8(rg[u], g);
          norm_row_bwd<D>(v, g, w, dw, dx[u] != nullptr, p.eps, A[u], partner);
          if (dx[u] != nullptr) *reinterpret_cast<uint4 *>(dx[u]) = pack8(v);
        }
      }
    } else {
      for (unsigned t = W.token; t < tokens; t += W.token_stride) {
        const int b = static_cast<int>(t / p.S), s = static_cast<int>(t - static_cast<unsigned>(b) * p.S);
        const __nv_bfloat16 *x = T.x + b * T.xb + s * T.xs + 8 * W.c + (W.h0 + W.sub) * T.xh;
        const __nv_bfloat16 *dy = G.x + b * G.b + s * G.s + 8 * W.c + (W.h0 + W.sub) * G.h;
        __nv_bfloat16 *dx = T.y + b * T.yb + s * T.ys + 8 * W.c + (W.h0 + W.sub) * T.yh;
        NormAngles<ROT> A;
        A.load(p, b, s, W.c, half_pieces);
        for (int h = W.h0 + W.sub; h < W.h1 + W.sub;
             h += kU * Walk::RPP, x += kU * Walk::RPP * T.xh, dy += kU * Walk::RPP * G.h, dx += kU * Walk::RPP * T.yh) {
          uint4 rx[kU], rg[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            rx[u] = make_uint4(0u, 0u, 0u, 0u);
            rg[u] = rx[u];
            if (h + u * Walk::RPP < W.h1) {
              rx[u] = __ldcs(reinterpret_cast<const uint4 *>(x + u * Walk::RPP * T.xh));
              rg[u] = __ldcs(reinterpret_cast<const uint4 *>(dy + u * Walk::RPP * G.h));
            }
          }
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const bool there = h + u * Walk::RPP < W.h1;
            float v[8], g[8];
            unpack8(rx[u], v);
            unpack8(rg[u], g);
            norm_row_bwd<D>(v, g, w, dw, there, p.eps, A, partner);
            if (there) *reinterpret_cast<uint4 *>(dx + u * Walk::RPP * T.yh) = pack8(v);
          }
        }
      }
    }
  }
  if (p.partial == nullptr) return;
  // The rows of a pass hold the same columns: lanes first, then warps.
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = Walk::LPR; off < 32; off <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], off);
  }
  const int warp = threadIdx.x >> 5;
  if (W.lane < Walk::LPR) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][8 * W.lane + i] = dw[i];
  }
  if (W.lane == 0) tensor_of[warp] = working ? W.ti : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) {
    const int ti = i / D, col = i - ti * D;
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < kNormWarps; ++k)
      if (tensor_of[k] == ti) a += sums[k][col];
    p.partial[static_cast<size_t>(blockIdx.x) * 2 * D + i] = a;
  }
}

// dw[tensor][column] = the CTAs' sums in a fixed order: warp k of a CTA adds
// rows k, k + 32, ... of 32 columns, then the 32 warps' sums are added.
constexpr int kNormReduceThreads = 1024;
__global__ void __launch_bounds__(kNormReduceThreads) norm_rope_dw_kernel(const float *__restrict__ partial, int rows,
                                                                          int D, void *dwq, void *dwk, int f32) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;   // column of the [2][D] sums
  float a = 0.f;
  for (int r = warp; r < rows; r += 32) a += partial[static_cast<size_t>(r) * 2 * D + i];
  sums[warp][lane] = a;
  __syncthreads();
  if (warp != 0) return;
  a = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) a += sums[k][lane];
  void *dst = i < D ? dwq : dwk;
  if (dst == nullptr) return;
  const int col = i < D ? i : i - D;
  if (f32)
    static_cast<float *>(dst)[col] = a;
  else
    static_cast<__nv_bfloat16 *>(dst)[col] = __float2bfloat16_rn(a);   // the weight's own type, rounded once
}

}  // namespace cpattn
