// paged_io.cu -- moving tokens into and out of the paged cache.
//
// append: the decode step writes the new token's K and V into the cache and
// the cache grows by one position per step (BeaconKV abstract; Random
// Attention article, "长推理的显存瓶颈").  The attention backend also hands
// over the step's queries (BeaconKV explainer §7.2), which go to a ring of the
// last W steps for the periodic beacon update.
// gather_dense: a dense copy of one layer, used to check the cache against
// the oracle.
// The 4-bit cache (KVC_INT4) has an append that codes the rows on their way
// into the pool and a gather that returns the values the codes stand for.
// Where the context tracks attention weights, an appended row starts at 0.
//
// All kernels but the 4-bit ones move 16-byte vectors, one per thread, with consecutive
// threads on consecutive bytes of the source (coalesced reads; writes are
// contiguous per row).  Sources may be page-locked host memory, read over
// PCIe through the unified address space.
#include <math_constants.h>

#include "int4.cuh"
#include "kvc_internal.h"

namespace kvc {
namespace {

__global__ void bt_scatter_kernel(const int32_t *__restrict__ pairs, int n,
                                  int32_t *__restrict__ block_table) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) block_table[pairs[2 * i]] = pairs[2 * i + 1];
}

// source [n_req][layers][T][hkv][row] ; one thread per 16-byte vector
__global__ void append_kv_kernel(const uint8_t *__restrict__ k_src, const uint8_t *__restrict__ v_src,
                                 uint8_t *__restrict__ k_pool, uint8_t *__restrict__ v_pool,
                                 int32_t *__restrict__ pos_map, float *__restrict__ weights,
                                 const int32_t *__restrict__ block_table,
                                 const int4 *__restrict__ desc, int layers, int T, int hkv,
                                 int vpr, int64_t total, int64_t num_pages, int bt_stride) {
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= total) return;
  int64_t rest = g;
  const int v = (int)(rest % vpr);
  rest /= vpr;
  const int h = (int)(rest % hkv);
  rest /= hkv;
  const int t = (int)(rest % T);
  rest /= T;
  const int l = (int)(rest % layers);
  const int i = (int)(rest / layers);
  const int4 d = desc[i];  // req, len_before, pos_before
  const int slot = d.y + t;
  const int page = block_table[(int64_t)d.x * bt_stride + (slot >> 4)];
  const int64_t row = (((int64_t)l * num_pages + page) * hkv + h) * kPage + (slot & (kPage - 1));
  const int64_t dst = row * vpr * 16 + (int64_t)v * 16;
  *reinterpret_cast<uint4 *>(k_pool + dst) = *reinterpret_cast<const uint4 *>(k_src + g * 16);
  *reinterpret_cast<uint4 *>(v_pool + dst) = *reinterpret_cast<const uint4 *>(v_src + g * 16);
  if (v == 0) {
    pos_map[row] = d.z + t;
    if (weights) weights[row] = 0.f;
  }
}

// 4-bit append.  D/8 neighbouring lanes take one row, 8 channels (16 bytes of
// bf16) each, so a group of D/4 channels is 4 lanes (D = 128) or 2 (D = 64):
// its smallest and largest value come from one or two shuffles, and the lanes
// of a row write its codes 4 bytes apiece, side by side.
template <int D, bool IS_V>
__device__ __forceinline__ void int4_code_chunk(uint4 x4, uint8_t *row, int v, unsigned lanes) {
  constexpr int kLanes = D / 8 / kInt4Groups;  // lanes of one group
  const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad = fmaf(x[i], 0.f, bad);  // NaN once a value is infinite or NaN
  }
#pragma unroll
  for (int m = 1; m < kLanes; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(lanes, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, m));
    bad += __shfl_xor_sync(lanes, bad, m);
  }
  float s = int4_step(lo, hi) + bad;
  uint32_t codes = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= (uint32_t)__float2int_rn(__fdiv_rn(x[i] - lo, s)) << (4 * i);
  }
  if (v % kLanes == 0) *reinterpret_cast<uint32_t *>(row + (v / kLanes) * 4) = int4_word<IS_V>(s, lo);
  uint8_t *dst = row + kInt4Header;
  if constexpr (IS_V) {
    reinterpret_cast<uint32_t *>(dst)[v] = codes;
  } else if constexpr (D == 128) {
    reinterpret_cast<uint32_t *>(dst)[int4_k_word(v)] = codes;
  } else {
    reinterpret_cast<uint16_t *>(dst)[int4_k_half(2 * v)] = (uint16_t)codes;
    reinterpret_cast<uint16_t *>(dst)[int4_k_half(2 * v + 1)] = (uint16_t)(codes >> 16);
  }
}

template <int D>
__global__ void append_kv4_kernel(const uint4 *__restrict__ k_src, const uint4 *__restrict__ v_src,
                                  uint8_t *__restrict__ k_pool, uint8_t *__restrict__ v_pool,
                                  int32_t *__restrict__ pos_map, float *__restrict__ weights,
                                  const int32_t *__restrict__ block_table, const int4 *__restrict__ desc,
                                  int layers, int T, int hkv, int64_t total, int64_t num_pages, int bt_stride) {
  constexpr int vpr = D / 8;
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  // total is a multiple of vpr, so the lanes of a row leave together
  const unsigned lanes = __ballot_sync(0xffffffffu, g < total);
  if (g >= total) return;
  int64_t rest = g;
  const int v = (int)(rest % vpr);
  rest /= vpr;
  const int h = (int)(rest % hkv);
  rest /= hkv;
  const int t = (int)(rest % T);
  rest /= T;
  const int l = (int)(rest % layers);
  const int i = (int)(rest / layers);
  const int4 d = desc[i];  // req, len_before, pos_before
  const int slot = d.y + t;
  const int page = block_table[(int64_t)d.x * bt_stride + (slot >> 4)];
  const int64_t row = (((int64_t)l * num_pages + page) * hkv + h) * kPage + (slot & (kPage - 1));
  const uint4 kx = k_src[g], vx = v_src[g];
  int4_code_chunk<D, false>(kx, k_pool + row * int4_row_bytes(D), v, lanes);
  int4_code_chunk<D, true>(vx, v_pool + row * int4_row_bytes(D), v, lanes);
  if (v == 0) {
    pos_map[row] = d.z + t;
    if (weights) weights[row] = 0.f;
  }
}

// source [n_req][layers][T][hq][row]; only the last W steps are written
__global__ void append_q_kernel(const uint8_t *__restrict__ q_src, uint8_t *__restrict__ qring,
                                const int4 *__restrict__ desc, int layers, int T, int t0, int W,
                                int hq, int vpr, int64_t total) {
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= total) return;
  int64_t rest = g;
  const int v = (int)(rest % vpr);
  rest /= vpr;
  const int hh = (int)(rest % hq);
  rest /= hq;
  const int tt = (int)(rest % (T - t0));
  rest /= (T - t0);
  const int l = (int)(rest % layers);
  const int i = (int)(rest / layers);
  const int t = t0 + tt;
  const int4 d = desc[i];  // req, ring slot of step 0
  const int ring = (d.y + t) % W;
  const int64_t src = ((((int64_t)i * layers + l) * T + t) * hq + hh) * vpr + v;
  const int64_t dst = ((((int64_t)d.x * layers + l) * W + ring) * hq + hh) * vpr + v;
  reinterpret_cast<uint4 *>(qring)[dst] = reinterpret_cast<const uint4 *>(q_src)[src];
}

__global__ void gather_dense_kernel(const uint8_t *__restrict__ k_pool, const uint8_t *__restrict__ v_pool,
                                    const int32_t *__restrict__ pos_map,
                                    const int32_t *__restrict__ block_table,
                                    const int32_t *__restrict__ lengths, int layer, int req_begin,
                                    int cap, int hkv, int vpr, int64_t total, int64_t num_pages,
                                    int bt_stride, uint8_t *__restrict__ k_out,
                                    uint8_t *__restrict__ v_out, int32_t *__restrict__ pos_out) {
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= total) return;
  int64_t rest = g;
  const int v = (int)(rest % vpr);
  rest /= vpr;
  const int slot = (int)(rest % cap);
  rest /= cap;
  const int h = (int)(rest % hkv);
  const int i = (int)(rest / hkv);
  const int r = req_begin + i;
  uint4 kv = make_uint4(0, 0, 0, 0), vv = make_uint4(0, 0, 0, 0);
  int pos = -1;
  if (slot < lengths[r]) {
    const int page = block_table[(int64_t)r * bt_stride + (slot >> 4)];
    const int64_t row = (((int64_t)layer * num_pages + page) * hkv + h) * kPage + (slot & (kPage - 1));
    kv = *reinterpret_cast<const uint4 *>(k_pool + row * vpr * 16 + (int64_t)v * 16);
    vv = *reinterpret_cast<const uint4 *>(v_pool + row * vpr * 16 + (int64_t)v * 16);
    pos = pos_map[row];
  }
  if (k_out) reinterpret_cast<uint4 *>(k_out)[g] = kv;
  if (v_out) reinterpret_cast<uint4 *>(v_out)[g] = vv;
  if (pos_out && v == 0) pos_out[g / vpr] = pos;
}

// the values of channels 8 v .. 8 v + 7: one lane's share of a row
template <int D, bool IS_V>
__device__ __forceinline__ void int4_values(const uint8_t *row, int v, float4 &a, float4 &b) {
  const uint32_t h = *reinterpret_cast<const uint32_t *>(row + (v * 8 / (D / kInt4Groups)) * 4);
  const uint8_t *src = row + kInt4Header;
  uint32_t c;
  if constexpr (IS_V) {
    c = reinterpret_cast<const uint32_t *>(src)[v];
  } else if constexpr (D == 128) {
    c = reinterpret_cast<const uint32_t *>(src)[int4_k_word(v)];
  } else {
    c = reinterpret_cast<const uint16_t *>(src)[int4_k_half(2 * v)] |
        (uint32_t)reinterpret_cast<const uint16_t *>(src)[int4_k_half(2 * v + 1)] << 16;
  }
  float s, zs, mid, x[8];
  int4_unword(h, s, zs, mid);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((c >> (4 * i)) & 15u), s, -zs) + mid;  // the fma is exact
  a = make_float4(x[0], x[1], x[2], x[3]);
  b = make_float4(x[4], x[5], x[6], x[7]);
}

// dense fp32 copy of one layer of the 4-bit cache
template <int D>
__global__ void gather_dense4_kernel(const uint8_t *__restrict__ k_pool, const uint8_t *__restrict__ v_pool,
                                     const int32_t *__restrict__ pos_map, const int32_t *__restrict__ block_table,
                                     const int32_t *__restrict__ lengths, int layer, int req_begin, int cap,
                                     int hkv, int64_t total, int64_t num_pages, int bt_stride,
                                     float4 *__restrict__ k_out, float4 *__restrict__ v_out,
                                     int32_t *__restrict__ pos_out) {
  constexpr int vpr = D / 8;
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= total) return;
  int64_t rest = g;
  const int v = (int)(rest % vpr);
  rest /= vpr;
  const int slot = (int)(rest % cap);
  rest /= cap;
  const int h = (int)(rest % hkv);
  const int i = (int)(rest / hkv);
  const int r = req_begin + i;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 k0 = zero, k1 = zero, v0 = zero, v1 = zero;
  int pos = -1;
  if (slot < lengths[r]) {
    const int page = block_table[(int64_t)r * bt_stride + (slot >> 4)];
    const int64_t row = (((int64_t)layer * num_pages + page) * hkv + h) * kPage + (slot & (kPage - 1));
    if (k_out) int4_values<D, false>(k_pool + row * int4_row_bytes(D), v, k0, k1);
    if (v_out) int4_values<D, true>(v_pool + row * int4_row_bytes(D), v, v0, v1);
    pos = pos_map[row];
  }
  if (k_out) {
    k_out[2 * g] = k0;
    k_out[2 * g + 1] = k1;
  }
  if (v_out) {
    v_out[2 * g] = v0;
    v_out[2 * g + 1] = v1;
  }
  if (pos_out && v == 0) pos_out[g / vpr] = pos;
}

inline unsigned blocks_for(int64_t total, int nt) { return (unsigned)((total + nt - 1) / nt); }

}  // namespace

cudaError_t launch_bt_scatter(const int32_t *pairs, int n, int32_t *block_table, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  bt_scatter_kernel<<<blocks_for(n, 256), 256, 0, s>>>(pairs, n, block_table);
  return cudaGetLastError();
}

cudaError_t launch_append_kv(const uint8_t *k_src, const uint8_t *v_src, uint8_t *k_pool,
                             uint8_t *v_pool, int32_t *pos_map, float *weights,
                             const int32_t *block_table, const int32_t *desc, int n_req, int layers, int T,
                             int hkv, int row_bytes, int64_t num_pages, int bt_stride, cudaStream_t s) {
  const int vpr = row_bytes / 16;
  const int64_t total = (int64_t)n_req * layers * T * hkv * vpr;
  if (total <= 0) return cudaSuccess;
  append_kv_kernel<<<blocks_for(total, 256), 256, 0, s>>>(
      k_src, v_src, k_pool, v_pool, pos_map, weights, block_table, reinterpret_cast<const int4 *>(desc),
      layers, T, hkv, vpr, total, num_pages, bt_stride);
  return cudaGetLastError();
}

cudaError_t launch_append_kv4(const uint8_t *k_src, const uint8_t *v_src, uint8_t *k_pool, uint8_t *v_pool,
                              int32_t *pos_map, float *weights, const int32_t *block_table, const int32_t *desc,
                              int n_req, int layers, int T, int hkv, int head_dim, int64_t num_pages,
                              int bt_stride, cudaStream_t s) {
  const int64_t total = (int64_t)n_req * layers * T * hkv * (head_dim / 8);
  if (total <= 0) return cudaSuccess;
  auto kernel = head_dim == 128 ? append_kv4_kernel<128> : append_kv4_kernel<64>;
  kernel<<<blocks_for(total, 256), 256, 0, s>>>(
      reinterpret_cast<const uint4 *>(k_src), reinterpret_cast<const uint4 *>(v_src), k_pool, v_pool, pos_map,
      weights, block_table, reinterpret_cast<const int4 *>(desc), layers, T, hkv, total, num_pages, bt_stride);
  return cudaGetLastError();
}

cudaError_t launch_append_q(const uint8_t *q_src, uint8_t *qring, const int32_t *desc, int n_req,
                            int layers, int T, int t0, int W, int hq, int row_bytes,
                            cudaStream_t s) {
  const int vpr = row_bytes / 16;
  const int64_t total = (int64_t)n_req * layers * (T - t0) * hq * vpr;
  if (total <= 0) return cudaSuccess;
  append_q_kernel<<<blocks_for(total, 256), 256, 0, s>>>(
      q_src, qring, reinterpret_cast<const int4 *>(desc), layers, T, t0, W, hq, vpr, total);
  return cudaGetLastError();
}

cudaError_t launch_gather_dense(const uint8_t *k_pool, const uint8_t *v_pool,
                                const int32_t *pos_map, const int32_t *block_table,
                                const int32_t *lengths, int layer, int req_begin, int req_count,
                                int cap, int hkv, int row_bytes, int64_t num_pages, int bt_stride,
                                uint8_t *k_out, uint8_t *v_out, int32_t *pos_out, cudaStream_t s) {
  const int vpr = row_bytes / 16;
  const int64_t total = (int64_t)req_count * hkv * cap * vpr;
  if (total <= 0) return cudaSuccess;
  gather_dense_kernel<<<blocks_for(total, 256), 256, 0, s>>>(
      k_pool, v_pool, pos_map, block_table, lengths, layer, req_begin, cap, hkv, vpr, total,
      num_pages, bt_stride, k_out, v_out, pos_out);
  return cudaGetLastError();
}

cudaError_t launch_gather_dense4(const uint8_t *k_pool, const uint8_t *v_pool, const int32_t *pos_map,
                                 const int32_t *block_table, const int32_t *lengths, int layer, int req_begin,
                                 int req_count, int cap, int hkv, int head_dim, int64_t num_pages, int bt_stride,
                                 float *k_out, float *v_out, int32_t *pos_out, cudaStream_t s) {
  const int64_t total = (int64_t)req_count * hkv * cap * (head_dim / 8);
  if (total <= 0) return cudaSuccess;
  auto kernel = head_dim == 128 ? gather_dense4_kernel<128> : gather_dense4_kernel<64>;
  kernel<<<blocks_for(total, 256), 256, 0, s>>>(
      k_pool, v_pool, pos_map, block_table, lengths, layer, req_begin, cap, hkv, total, num_pages, bt_stride,
      reinterpret_cast<float4 *>(k_out), reinterpret_cast<float4 *>(v_out), pos_out);
  return cudaGetLastError();
}

}  // namespace kvc
