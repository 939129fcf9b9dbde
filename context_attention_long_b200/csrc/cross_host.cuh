// cross_host.cuh -- entry points of cross attention: argument checks and
// launches.  Included by cpattn_api.cu, whose helpers it uses.
#pragma once

namespace cpattn {

// 4-D view [B, rows, H, D] of a bf16 tensor, box {64, box_heads, box_rows,
// 1}, 128-byte swizzle; rows past the end of a batch element read as zero.
static bool encode_view_map(CUtensorMap *tm, const void *ptr, int D, int H, int rows, int B, const View4 &v,
                            int box_rows = kQTile, int box_heads = 1) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(B)};
  // an axis of one element is never stepped: any valid stride
  const long long st[3] = {H == 1 ? D : v.h, rows == 1 ? D : v.s, B == 1 ? D : v.b};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) strides[i] = static_cast<cuuint64_t>(st[i]) * 2;
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    std::snprintf(t_encode_detail, sizeof(t_encode_detail),
                  "tensor map encoding (driver result %d; address %p, dims %d x %d x %d x %d, strides %lld, %lld, %lld)",
                  static_cast<int>(r), ptr, D, H, rows, B, st[0], st[1], st[2]);
  return r == CUDA_SUCCESS;
}

// A view that the copy engine reads: no broadcast axes, strides below 2^39
// elements (the map's limit of 2^40 bytes).
static int resolve_map_view(const long long *strides, int B, int S, int H, int D, View4 &v) {
  const int st = resolve_view(strides, B, S, H, D, false, v);
  if (st != CPATTN_OK) return st;
  const int n[3] = {B, S, H};
  const long long s[3] = {v.b, v.s, v.h};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] < D || s[i] >= (1ll << 39))) return CPATTN_ERR_SHAPE;
  return CPATTN_OK;
}

static int check_cross_shape(int B, int H, int Hk, int Sq, int Skv, int D) {
  int st = check_attn_shape(B, H, Sq, D);
  if (st == CPATTN_OK) st = check_attn_shape(B, Hk, Skv, D);
  if (st != CPATTN_OK) return st;
  if (H % Hk != 0) return CPATTN_ERR_INDIVISIBLE;
  // units, rows and (row, head) indices are ints in the kernels
  if (static_cast<long long>(B) * Sq * H >= (1ll << 31) || static_cast<long long>(B) * Skv * Hk >= (1ll << 31))
    return CPATTN_ERR_SHAPE;
  return CPATTN_OK;
}

// Clusters of `splits` CTAs of the split forward kernel that are resident at
// once on the current device, asked once.
constexpr int kCrossMaxSplits = 8;   // portable cluster size
template <int D>
static void cross_split_config(int splits, long long units, cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr,
                                      cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
  cfg.blockDim = dim3(kCrossThreads);
  cfg.dynamicSmemBytes = CrossSmem<D>::kAllocBytes;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

template <int D>
static cudaError_t launch_cross_d(CrossParams &p, cudaStream_t stream) {
  static std::mutex mu;
  static bool configured[kMaxDevices] = {false};
  static int resident[kMaxDevices][kCrossMaxSplits + 1] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  const int sms = std::max(device_sm_count(), 1);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  const int *clusters;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      cudaError_t e = cudaFuncSetAttribute(cross_fwd_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           CrossSmem<D>::kAllocBytes);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(cross_fwd_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               CrossSmem<D>::kAllocBytes);
      if (e != cudaSuccess) return e;
      for (int s = 2; s <= kCrossMaxSplits; ++s) {
        cross_split_config<D>(s, sms, cfg, attr, nullptr);
        if (cudaOccupancyMaxActiveClusters(&resident[dev][s], cross_fwd_kernel<D, true>, &cfg) != cudaSuccess) {
          cudaGetLastError();
          resident[dev][s] = 0;   // this size is not used
        }
      }
      configured[dev] = true;
    }
    clusters = resident[dev];
  }
  // Split when units leave SMs idle and states are long: the size whose waves
  // of clusters end first.  A CTA walks its share of the key tiles (a step of
  // some 2 us each) and pays about two steps for the join.
  const int tiles = (p.Skv + kKVTile - 1) / kKVTile;
  p.splits = 1;
  double least = tiles * std::ceil(static_cast<double>(p.units) / sms);
  for (int s = 2; s <= std::min(kCrossMaxSplits, tiles); ++s) {
    if (clusters[s] < 1) continue;
    const double cost = (std::ceil(static_cast<double>(tiles) / s) + 2.0) * std::ceil(static_cast<double>(p.units) / clusters[s]);
    if (cost < least) {
      least = cost;
      p.splits = s;
    }
  }
  if (p.splits > 1) {
    cross_split_config<D>(p.splits, p.units, cfg, attr, stream);
    return cudaLaunchKernelEx(&cfg, cross_fwd_kernel<D, true>, p);
  }
  const int grid = std::min(p.units, sms);
  cross_fwd_kernel<D, false><<<static_cast<unsigned>(grid), kCrossThreads, CrossSmem<D>::kAllocBytes, stream>>>(p);
  return cudaGetLastError();
}

// Few rows: the kernel of cross_token_kernel.cuh, up to 16 rows (query tokens
// times heads of a group) a key head, where it is faster (8 requests, 32 / 8
// heads, one token, 1500 states: 14.5 us, with tiles 27.7).  At 32 rows of one
// head and short states the tensor-core tiles are (24 heads, 32 queries, 512
// states: 9.3 us, with 32-row fragments 10.3).  Against long states the step to
// tiles costs: 4 x 24 heads, 4096 states, 16 queries take 36.8 us and 17 take
// 60.6; most for groups whose heads do not share a tile (8 x 28 / 4 heads, 4096
// states: 2 queries 13.0 us, 3 queries 58.4).
constexpr int kTokenRows = 16;
constexpr int kTokenSplits = 16;   // above the portable cluster size of 8: needs the kernel's opt-in

// The largest cluster a unit whose clusters are all resident at once, each CTA
// with a stage of states at least (two waves of clusters of 12 took 34 us where
// one wave of clusters of 8 took 23, at 24 units and 8192 states).
template <int D>
static cudaError_t launch_token(CrossTokenParams &p, cudaStream_t stream) {
  static std::mutex mu;
  static bool configured[kMaxDevices] = {false};
  static int resident[kMaxDevices][kTokenSplits + 1] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(kTokenThreads);
  cfg.dynamicSmemBytes = TokenSmem<D>::kAllocBytes;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int *clusters;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      cudaError_t e = cudaFuncSetAttribute(cross_token_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           TokenSmem<D>::kAllocBytes);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(cross_token_kernel<D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      for (int s = 2; s <= kTokenSplits; ++s) {
        cfg.gridDim = dim3(static_cast<unsigned>(s) * 256);
        attr[0].val.clusterDim.x = static_cast<unsigned>(s);
        if (cudaOccupancyMaxActiveClusters(&resident[dev][s], cross_token_kernel<D>, &cfg) != cudaSuccess) {
          cudaGetLastError();
          resident[dev][s] = 0;   // this size is not used
        }
      }
      configured[dev] = true;
    }
    clusters = resident[dev];
  }
  const long long units = static_cast<long long>(p.B) * p.Hk;
  const int stages = (p.Skv + kTokenKeys - 1) / kTokenKeys;
  p.splits = std::min(kTokenSplits, stages);
  while (p.splits > 1 && clusters[p.splits] < units) --p.splits;
  cfg.gridDim = dim3(static_cast<unsigned>(units * p.splits));
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  return cudaLaunchKernelEx(&cfg, cross_token_kernel<D>, p);
}

// ----------------------------------------------------------------- backward
// Workspace: Delta, the parts' sums, then dS tiles of as many (batch element,
// key head) pairs as fit, each part on a 256-byte boundary.
static size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
static size_t cross_delta_bytes(int B, int H, int Sq) { return round256(static_cast<size_t>(B) * H * Sq * sizeof(float)); }
static size_t cross_pair_ds_bytes(int H, int Hk, int Sq, int Skv) {
  return static_cast<size_t>(H / Hk) * ((Sq + 127) / 128) * ((Skv + 127) / 128) * kBwdDsTileBytes;
}
static size_t cross_partial_bytes(int B, int H, int Hk, int Sq, int Skv, int D) {
  const double steps = static_cast<double>(B) * Hk * ((Skv + 127) / 128) * (H / Hk) * ((Sq + 127) / 128);
  const double runs = std::min(static_cast<double>(kCrossMaxRuns), steps);
  return static_cast<size_t>(runs) * 2 * 2 * 128 * D * sizeof(float);
}
// dS of one pair, or where that is more than kCrossLeastDs, of a range of its
// walk: as many steps as fit (a step takes 32 KB for each K tile, so there is
// room for one).
constexpr size_t kCrossLeastDs = size_t{256} << 20;
static_assert(static_cast<size_t>(kCrossMaxKTiles) * kBwdDsTileBytes <= kCrossLeastDs, "a range of one step");
static size_t cross_least_ds_bytes(int H, int Hk, int Sq, int Skv) {
  return std::min(cross_pair_ds_bytes(H, Hk, Sq, Skv), kCrossLeastDs);
}
// The ranges' sums of dK and dV, and one range's of tiles that one run covers.
static size_t cross_sums_bytes(int H, int Hk, int Sq, int Skv, int D) {
  if (cross_pair_ds_bytes(H, Hk, Sq, Skv) <= kCrossLeastDs) return 0;
  return static_cast<size_t>((Skv + 127) / 128) * 2 * 128 * D * sizeof(float);
}

// Delta: the self-attention's row sums where no element can have few states,
// else the kernel that tells the elements apart.
static cudaError_t launch_cross_delta(const CrossBwdParams &p, const void *q, const View4 &vq, const void *k,
                                      const View4 &vk, const void *v, const View4 &vv, const void *out,
                                      const void *dout, float *delta, int D, cudaStream_t stream) {
  if (p.kv_lens == nullptr && p.Skv > kCrossFewStates) return launch_bwd_delta(out, dout, delta, p.B, p.Sq, p.H, D, stream);
  CrossDeltaParams d;
  std::memset(&d, 0, sizeof(d));
  d.q = static_cast<const __nv_bfloat16 *>(q);
  d.k = static_cast<const __nv_bfloat16 *>(k);
  d.v = static_cast<const __nv_bfloat16 *>(v);
  d.qb = vq.b; d.qs = vq.s; d.qh = vq.h;
  d.kb = vk.b; d.ks = vk.s; d.kh = vk.h;
  d.vb = vv.b; d.vs = vv.s; d.vh = vv.h;
  d.out = static_cast<const __nv_bfloat16 *>(out);
  d.dout = static_cast<const __nv_bfloat16 *>(dout);
  d.lse = p.lse;
  d.delta = delta;
  d.kv_lens = p.kv_lens;
  d.B = p.B;
  d.Sq = p.Sq;
  d.Skv = p.Skv;
  d.H = p.H;
  d.Hk = p.Hk;
  const int group = p.H / p.Hk;
  d.blocks = static_cast<int>((static_cast<long long>(group) * p.Sq + 15) / 16);
  const bool many = p.Skv > kCrossFewStates;
  const int ctas = (many ? 3 : 2) * std::max(device_sm_count(), 1);   // resident at once
  // A chunk is at least a block a warp, and at most eight: enough rows for the
  // chunk's K and V to be a small part of what is read.
  const long long blocks = static_cast<long long>(p.B) * p.Hk * d.blocks;
  d.chunk_blocks = 8 * static_cast<int>(std::min(8ll, std::max(1ll, blocks / (8ll * ctas))));
  d.chunks = (d.blocks + d.chunk_blocks - 1) / d.chunk_blocks;
  d.by_chunks.set(d.chunks);
  d.by_hk.set(p.Hk);
  d.by_group.set(group);
  d.by_element.set(p.H * p.Sq);
  d.scale_log2 = p.scale_log2;
  const int grid = static_cast<int>(std::min<long long>(static_cast<long long>(p.B) * p.Hk * d.chunks, ctas));
  if (D == 128)
    (many ? cross_delta_kernel<128, true> : cross_delta_kernel<128, false>)<<<grid, 256, 0, stream>>>(d);
  else
    (many ? cross_delta_kernel<64, true> : cross_delta_kernel<64, false>)<<<grid, 256, 0, stream>>>(d);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_cross_bwd_d(CrossBwdParams &p, cudaStream_t stream) {
  static std::mutex mu;
  static bool configured[kMaxDevices] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      cudaError_t e = cudaFuncSetAttribute(cross_bwd_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           BwdSmem<D, 2, true>::kAllocBytes);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(cross_bwd_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               CrossGemmSmem<D>::kAllocBytes + kCrossMaxKTiles * sizeof(int));
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  const int sms = std::max(device_sm_count(), 1);
  const long long tiles = static_cast<long long>(p.n_bh) * p.k_tiles;
  // One CTA an SM; a multiple of the K tiles where that idles at most a tenth
  // of the SMs, so that the CTAs of a head's K tiles walk in step.
  int ctas = std::min(sms, kCrossMaxRuns);
  if (p.k_tiles <= ctas && ctas % p.k_tiles <= ctas / 10) ctas -= ctas % p.k_tiles;
  p.ctas = static_cast<int>(std::min<long long>(ctas, tiles * p.walk));
  p.inv_ctas = 1.0 / p.ctas;
  p.inv_walk = 1.0 / p.walk;
  cross_bwd_dkv_kernel<D><<<static_cast<unsigned>(p.ctas), kBwdThreads, BwdSmem<D, 2, true>::kAllocBytes, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int units = p.n_bh * p.walk;
  const int grid = std::min(std::max(units, 2 * (p.ctas - 1)), sms);
  cross_bwd_dq_kernel<D><<<static_cast<unsigned>(grid), kCrossGemmThreads,
                           CrossGemmSmem<D>::kAllocBytes + (p.kv_lens ? p.k_tiles * sizeof(int) : 0), stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.sums == nullptr) return e;
  cross_range_kernel<D><<<static_cast<unsigned>(2 * p.k_tiles), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace cpattn

using namespace cpattn;

extern "C" {

int cpattn_cross_attention(const void *q, const long long *q_strides, const void *k, const long long *k_strides,
                           const void *v, const long long *v_strides, void *out, float *lse, const int *kv_lens,
                           int B, int H, int Hk, int Sq, int Skv, int D, cpattn_stream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr) return CPATTN_ERR_NULL;
  int st = check_cross_shape(B, H, Hk, Sq, Skv, D);
  if (st != CPATTN_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4(lse) || !aligned4(kv_lens))
    return CPATTN_ERR_ALIGNMENT;
  View4 vq, vk, vv, vo;
  if ((st = resolve_map_view(q_strides, B, Sq, H, D, vq)) != CPATTN_OK) return st;
  if ((st = resolve_map_view(k_strides, B, Skv, Hk, D, vk)) != CPATTN_OK) return st;
  if ((st = resolve_map_view(v_strides, B, Skv, Hk, D, vv)) != CPATTN_OK) return st;
  if ((st = resolve_map_view(nullptr, B, Sq, H, D, vo)) != CPATTN_OK) return st;
  st = check_device(nullptr);
  if (st != CPATTN_OK) return st;
  const float scale_log2 = static_cast<float>((1.0 / std::sqrt(static_cast<double>(D))) * 1.4426950408889634);
  if (static_cast<long long>(H / Hk) * Sq <= kTokenRows) {
    CrossTokenParams t;
    std::memset(&t, 0, sizeof(t));
    if (!encode_view_map(&t.tm_k, k, D, Hk, Skv, B, vk, kTokenKeys) ||
        !encode_view_map(&t.tm_v, v, D, Hk, Skv, B, vv, kTokenKeys))
      return cuda_fail(cudaErrorInvalidValue, t_encode_detail);
    t.q = static_cast<const __nv_bfloat16 *>(q);
    t.qb = vq.b;
    t.qs = vq.s;
    t.qh = vq.h;
    t.out = static_cast<__nv_bfloat16 *>(out);
    t.lse = lse;
    t.kv_lens = kv_lens;
    t.B = B;
    t.Sq = Sq;
    t.Skv = Skv;
    t.H = H;
    t.Hk = Hk;
    t.scale_log2 = scale_log2;
    t.timeout_ns = wait_timeout_ns();
    return cuda_result(D == 128 ? launch_token<128>(t, stream) : launch_token<64>(t, stream), "cross attention launch");
  }
  CrossParams p;
  std::memset(&p, 0, sizeof(p));
  // All heads of a group share tiles when their number is a power of two up to
  // 32, so that whole queries make up a warp's 32 output rows; that never takes
  // more tiles.  Heads of any other group have a tile each, however few their
  // queries, and every pair of tiles walks the states again (8 x 64 / 1 heads,
  // one query, 8192 states: 218 us, where 16 / 1 heads take 13).
  const int group = H / Hk;
  const bool pack = group <= 32 && (group & (group - 1)) == 0;
  const int heads = pack ? group : 1;
  if (!encode_view_map(&p.tm_q, q, D, H, Sq, B, vq, kQTile / heads, heads) ||
      !encode_view_map(&p.tm_k, k, D, Hk, Skv, B, vk) || !encode_view_map(&p.tm_v, v, D, Hk, Skv, B, vv) ||
      !encode_view_map(&p.tm_out, out, D, H, Sq, B, vo, 32 / heads, heads))
    return cuda_fail(cudaErrorInvalidValue, t_encode_detail);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.kv_lens = kv_lens;
  p.B = B;
  p.Sq = Sq;
  p.Skv = Skv;
  p.H = H;
  p.Hk = Hk;
  p.group = group;
  while ((1 << p.pack_log2) < heads) ++p.pack_log2;
  p.q_tiles = (Sq + kQTile / heads - 1) / (kQTile / heads);
  p.group_tiles = group / heads * p.q_tiles;
  p.pairs = (p.group_tiles + 1) / 2;
  p.units = B * Hk * p.pairs;
  p.by_pairs.set(p.pairs);
  p.by_hk.set(Hk);
  p.by_q_tiles.set(p.q_tiles);
  p.scale_log2 = scale_log2;
  p.timeout_ns = wait_timeout_ns();
  return cuda_result(D == 128 ? launch_cross_d<128>(p, stream) : launch_cross_d<64>(p, stream),
                     "cross attention launch");
}

size_t cpattn_cross_attention_backward_ds_bytes(int H, int Hk, int Sq, int Skv) {
  if (H < 1 || Hk < 1 || H % Hk != 0 || Sq < 1 || Skv < 1) return 0;
  return cross_pair_ds_bytes(H, Hk, Sq, Skv);
}

size_t cpattn_cross_attention_backward_workspace_bytes(int B, int H, int Hk, int Sq, int Skv, int D) {
  if (check_cross_shape(B, H, Hk, Sq, Skv, D) != CPATTN_OK) return 0;
  return 256 + cross_delta_bytes(B, H, Sq) + cross_partial_bytes(B, H, Hk, Sq, Skv, D) +
         2 * cross_sums_bytes(H, Hk, Sq, Skv, D) + cross_least_ds_bytes(H, Hk, Sq, Skv);
}

int cpattn_cross_attention_backward(const void *q, const long long *q_strides, const void *k,
                                    const long long *k_strides, const void *v, const long long *v_strides,
                                    const void *out, const float *lse, const void *dout, const int *kv_lens, void *dq,
                                    void *dk, void *dv, int B, int H, int Hk, int Sq, int Skv, int D, void *workspace,
                                    size_t workspace_bytes, cpattn_stream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || lse == nullptr || dout == nullptr ||
      dq == nullptr || dk == nullptr || dv == nullptr)
    return CPATTN_ERR_NULL;
  int st = check_cross_shape(B, H, Hk, Sq, Skv, D);
  if (st != CPATTN_OK) return st;
  const int q_tiles = (Sq + 127) / 128, k_tiles = (Skv + 127) / 128;
  if (k_tiles > kCrossMaxKTiles) return CPATTN_ERR_SHAPE;
  for (const void *ptr : {q, k, v, out, dout, static_cast<const void *>(dq), static_cast<const void *>(dk),
                          static_cast<const void *>(dv)})
    if (!aligned16(ptr)) return CPATTN_ERR_ALIGNMENT;
  if (!aligned4(lse) || !aligned4(kv_lens)) return CPATTN_ERR_ALIGNMENT;
  View4 vq, vk, vv, vo;
  if ((st = resolve_map_view(q_strides, B, Sq, H, D, vq)) != CPATTN_OK) return st;
  if ((st = resolve_map_view(k_strides, B, Skv, Hk, D, vk)) != CPATTN_OK) return st;
  if ((st = resolve_map_view(v_strides, B, Skv, Hk, D, vv)) != CPATTN_OK) return st;
  if ((st = resolve_map_view(nullptr, B, Sq, H, D, vo)) != CPATTN_OK) return st;
  if (workspace == nullptr ||
      workspace_bytes < cpattn_cross_attention_backward_workspace_bytes(B, H, Hk, Sq, Skv, D))
    return CPATTN_ERR_WORKSPACE;
  st = check_device(nullptr);
  if (st != CPATTN_OK) return st;
  CrossBwdParams p;
  std::memset(&p, 0, sizeof(p));
  if (!encode_view_map(&p.tm_q, q, D, H, Sq, B, vq) || !encode_view_map(&p.tm_k, k, D, Hk, Skv, B, vk) ||
      !encode_view_map(&p.tm_v, v, D, Hk, Skv, B, vv) || !encode_view_map(&p.tm_do, dout, D, H, Sq, B, vo))
    return cuda_fail(cudaErrorInvalidValue, t_encode_detail);
  unsigned char *base = reinterpret_cast<unsigned char *>(round256(reinterpret_cast<uintptr_t>(workspace)));
  unsigned char *const end = static_cast<unsigned char *>(workspace) + workspace_bytes;
  float *delta = reinterpret_cast<float *>(base);
  base += cross_delta_bytes(B, H, Sq);
  p.partial = reinterpret_cast<float *>(base);
  base += cross_partial_bytes(B, H, Hk, Sq, Skv, D);
  float *const sums = reinterpret_cast<float *>(base), *const whole = sums + cross_sums_bytes(H, Hk, Sq, Skv, D) / 4;
  base += 2 * cross_sums_bytes(H, Hk, Sq, Skv, D);
  p.ds = base;
  const size_t pair = cross_pair_ds_bytes(H, Hk, Sq, Skv), space = static_cast<size_t>(end - base);
  const int pairs = B * Hk;
  p.lse = lse;
  p.delta = delta;
  p.kv_lens = kv_lens;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.B = B;
  p.Sq = Sq;
  p.Skv = Skv;
  p.H = H;
  p.Hk = Hk;
  p.q_tiles = q_tiles;
  p.k_tiles = k_tiles;
  const int walk = H / Hk * q_tiles;
  p.by_hk.set(Hk);
  p.by_q_tiles.set(q_tiles);
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  p.scale_log2 = static_cast<float>((1.0 / std::sqrt(static_cast<double>(D))) * 1.4426950408889634);
  p.timeout_ns = wait_timeout_ns();
  if (cudaError_t e = launch_cross_delta(p, q, vq, k, vk, v, vv, out, dout, delta, D, stream); e != cudaSuccess)
    return cuda_fail(e, "cross attention backward launch");
  auto launch = [&](int bh, int n, int w0, int steps) {
    p.bh0 = bh;
    p.n_bh = n;
    p.w0 = w0;
    p.walk = steps;
    p.by_walk.set(steps);
    return D == 128 ? launch_cross_bwd_d<128>(p, stream) : launch_cross_bwd_d<64>(p, stream);
  };
  cudaError_t e = cudaSuccess;
  if (space >= pair) {
    // Pairs whose dS fits together share the launches; the stream orders the
    // next group after the product that read this one's dS.
    const int at_once = static_cast<int>(std::min<size_t>(static_cast<size_t>(pairs), space / pair));
    for (int bh = 0; bh < pairs && e == cudaSuccess; bh += at_once) e = launch(bh, std::min(at_once, pairs - bh), 0, walk);
  } else {
    // Pair by pair in ranges of the walk whose dS fits.
    const int at_once = static_cast<int>(space / (static_cast<size_t>(k_tiles) * kBwdDsTileBytes));
    p.sums = sums;
    p.whole = whole;
    for (int bh = 0; bh < pairs; ++bh)
      for (int w0 = 0; w0 < walk && e == cudaSuccess; w0 += at_once) {
        p.first_range = w0 == 0;
        p.last_range = walk - w0 <= at_once;
        e = launch(bh, 1, w0, std::min(at_once, walk - w0));
      }
  }
  if (e != cudaSuccess) return cuda_fail(e, "cross attention backward launch");
  return CPATTN_OK;
}

}  // extern "C"
