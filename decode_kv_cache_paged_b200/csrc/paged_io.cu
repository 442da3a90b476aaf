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
#include <algorithm>

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

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes one group: D/4 channels as D/8 bf16 pairs.
//
// The append is bound by instructions before memory (at the HBM rate an SM has
// about 300 issue slots for a row's K and V), so a thread takes a whole group:
// smallest and largest value by packed minima and maxima that pass NaN on (an
// infinity makes hi - lo infinite), one step, reciprocal and word for all of it,
// no shuffles.  A code then is six instructions: the difference, the quotient
// in three (int4.cuh), the rounding as a sum with 1.5 * 2^23, whose lowest bits
// are the code, and a multiply-add that puts it in its place (the eight
// constants of a word come off in one).
// 1M rows of K and V, D = 128: 147 us (floor 107); eight channels a thread with
// a division and a conversion per code took 288.
template <int D, bool IS_V>
__device__ __forceinline__ void int4_code_group(const uint32_t (&w)[D / 8], uint8_t *row, int g) {
  uint32_t lo2 = w[0], hi2 = w[0];
#pragma unroll
  for (int i = 1; i < D / 8; ++i) {
    lo2 = min_bf16x2(lo2, w[i]);
    hi2 = max_bf16x2(hi2, w[i]);
  }
  lo2 = min_bf16x2(lo2, __byte_perm(lo2, lo2, 0x1032));
  hi2 = max_bf16x2(hi2, __byte_perm(hi2, hi2, 0x1032));
  const float lo = __uint_as_float(lo2 << 16), s = int4_step(lo, __uint_as_float(hi2 << 16));
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;  // s = 0, or NaN: every code is 0
  const float base = s > 0.f ? lo : 0.f;
  constexpr uint32_t kMagic = 0x4b400000u;  // the bits of 1.5 * 2^23
  uint32_t codes[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = w[4 * j + i / 2];
      const float v = __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
      c += __float_as_uint(quotient(v - base, s, inv) + 12582912.f) * (1u << (4 * i));
    }
    codes[j] = s > 0.f ? c - kMagic * 0x11111111u : 0u;
  }
  *reinterpret_cast<uint32_t *>(row + 4 * g) = int4_word<IS_V>(s, inv, lo);
  uint8_t *dst = row + kInt4Header;
  if constexpr (IS_V && D == 128) {
    *reinterpret_cast<uint4 *>(dst + 16 * g) = make_uint4(codes[0], codes[1], codes[D / 32 - 2], codes[D / 32 - 1]);
  } else if constexpr (IS_V) {
    *reinterpret_cast<uint2 *>(dst + 8 * g) = make_uint2(codes[0], codes[1]);
  } else if constexpr (D == 128) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t *>(dst)[int4_k_word(4 * g + j)] = codes[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<uint16_t *>(dst)[int4_k_half(4 * g + j)] = (uint16_t)(codes[j / 2] >> (16 * (j & 1)));
  }
}

// 4-bit append: a thread takes one group of one row (token, KV head), K and V.
// A segment is one (request, layer): its rows are contiguous in the source.
template <int D>
__global__ void __launch_bounds__(128) append_kv4_kernel(const uint4 *__restrict__ k_src, const uint4 *__restrict__ v_src,
                                                         uint8_t *__restrict__ k_pool, uint8_t *__restrict__ v_pool,
                                                         int32_t *__restrict__ pos_map, float *__restrict__ weights,
                                                         const int32_t *__restrict__ block_table,
                                                         const int4 *__restrict__ desc, int layers, int T, int hkv,
                                                         int n_seg, int64_t num_pages, int bt_stride) {
  const int n_rows = T * hkv;
  const int r = blockIdx.x * 32 + threadIdx.x / kInt4Groups, g = threadIdx.x % kInt4Groups;
  if (r >= n_rows) return;
  const int t = r / hkv, h = r - t * hkv;
  for (int seg = blockIdx.y; seg < n_seg; seg += gridDim.y) {
    const int64_t src = (((int64_t)seg * n_rows + r) * kInt4Groups + g) * (D / 32);
    uint32_t kw[D / 8], vw[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 a = k_src[src + i], b = v_src[src + i];
      kw[4 * i] = a.x, kw[4 * i + 1] = a.y, kw[4 * i + 2] = a.z, kw[4 * i + 3] = a.w;
      vw[4 * i] = b.x, vw[4 * i + 1] = b.y, vw[4 * i + 2] = b.z, vw[4 * i + 3] = b.w;
    }
    const int4 d = desc[seg / layers];  // req, len_before, pos_before
    const int slot = d.y + t;
    const int64_t page = (int64_t)(seg % layers) * num_pages + block_table[(int64_t)d.x * bt_stride + (slot >> 4)];
    const int64_t row = (page * hkv + h) * kPage + (slot & (kPage - 1));
    int4_code_group<D, false>(kw, k_pool + row * int4_row_bytes(D), g);
    int4_code_group<D, true>(vw, v_pool + row * int4_row_bytes(D), g);
    if (g == 0) {
      pos_map[row] = d.z + t;
      if (weights) weights[row] = 0.f;
    }
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

// a group's word and four codes (channels 4 v .. 4 v + 3): one lane's share of a row
struct Int4Piece {
  uint32_t word, codes;
};
template <int D, bool IS_V>
__device__ __forceinline__ Int4Piece int4_piece(const uint8_t *row, int v) {
  constexpr int kLanes = D / 4;
  // 16-bit pieces of the codes: of natural word v / 2 the half v % 2
  const int at = IS_V ? v : D == 128 ? 2 * int4_k_word(v >> 1) + (v & 1) : int4_k_half(v);
  return {*reinterpret_cast<const uint32_t *>(row + v / (kLanes / kInt4Groups) * 4),
          *reinterpret_cast<const uint16_t *>(row + kInt4Header + 2 * at)};
}
__device__ __forceinline__ float4 int4_values(Int4Piece p) {
  float s, zs, mid, x[4];
  int4_unword(p.word, s, zs, mid);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = fmaf(small_float((p.codes >> (4 * i)) & 15u), s, -zs) + mid;  // the fma is exact
  return make_float4(x[0], x[1], x[2], x[3]);
}

// Dense fp32 copy of one layer of the 4-bit cache.  A block takes kGatherSlots
// slots of one (request, KV head), D/4 lanes a row, 16 bytes of each output a
// lane; a thread reads its share of four rows before it writes the first.
constexpr int kGatherSlots = 64;
template <int D>
__global__ void __launch_bounds__(256)
    gather_dense4_kernel(const uint8_t *__restrict__ k_pool, const uint8_t *__restrict__ v_pool,
                         const int32_t *__restrict__ pos_map, const int32_t *__restrict__ block_table,
                         const int32_t *__restrict__ lengths, int layer, int req_begin, int cap, int hkv, int n_seg,
                         int64_t num_pages, int bt_stride, float4 *__restrict__ k_out, float4 *__restrict__ v_out,
                         int32_t *__restrict__ pos_out) {
  constexpr int kLanes = D / 4, kPass = 256 / kLanes, kBatch = 4;
  const int v = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  for (int seg = blockIdx.y; seg < n_seg; seg += gridDim.y) {
    const int i = seg / hkv, h = seg - i * hkv, r = req_begin + i;
    const int len = lengths[r];
    const int32_t *bt = block_table + (int64_t)r * bt_stride;
    for (int x = 0; x < kGatherSlots / kPass; x += kBatch) {
      const int slot0 = blockIdx.x * kGatherSlots + x * kPass + sub;
      Int4Piece kp[kBatch], vp[kBatch];
      int pos[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int slot = slot0 + b * kPass;
        kp[b] = vp[b] = {0u, 0u};  // past the length: zeros
        pos[b] = -1;
        if (slot < min(len, cap)) {
          const int64_t row = (((int64_t)layer * num_pages + bt[slot >> 4]) * hkv + h) * kPage + (slot & (kPage - 1));
          if (k_out) kp[b] = int4_piece<D, false>(k_pool + row * int4_row_bytes(D), v);
          if (v_out) vp[b] = int4_piece<D, true>(v_pool + row * int4_row_bytes(D), v);
          if (v == 0) pos[b] = pos_map[row];
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int slot = slot0 + b * kPass;
        if (slot >= cap) continue;
        const int64_t to = (int64_t)seg * cap + slot;
        if (k_out) k_out[to * kLanes + v] = int4_values(kp[b]);
        if (v_out) v_out[to * kLanes + v] = int4_values(vp[b]);
        if (pos_out && v == 0) pos_out[to] = pos[b];
      }
    }
  }
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
  const int64_t n_seg = (int64_t)n_req * layers;
  if (n_seg * T * hkv <= 0) return cudaSuccess;
  if (n_seg > 0x7fffffff || (int64_t)T * hkv > 0x7fffffff) return cudaErrorInvalidValue;
  auto kernel = head_dim == 128 ? append_kv4_kernel<128> : append_kv4_kernel<64>;
  const dim3 grid(blocks_for((int64_t)T * hkv, 32), (unsigned)std::min<int64_t>(n_seg, 65535));
  kernel<<<grid, 128, 0, s>>>(reinterpret_cast<const uint4 *>(k_src), reinterpret_cast<const uint4 *>(v_src), k_pool, v_pool,
                              pos_map, weights, block_table, reinterpret_cast<const int4 *>(desc), layers, T, hkv,
                              (int)n_seg, num_pages, bt_stride);
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
  const int64_t n_seg = (int64_t)req_count * hkv;
  if (n_seg <= 0 || cap <= 0) return cudaSuccess;
  if (n_seg > 0x7fffffff) return cudaErrorInvalidValue;
  auto kernel = head_dim == 128 ? gather_dense4_kernel<128> : gather_dense4_kernel<64>;
  const dim3 grid(blocks_for(cap, kGatherSlots), (unsigned)std::min<int64_t>(n_seg, 65535));
  kernel<<<grid, 256, 0, s>>>(k_pool, v_pool, pos_map, block_table, lengths, layer, req_begin, cap, hkv, (int)n_seg,
                              num_pages, bt_stride, reinterpret_cast<float4 *>(k_out), reinterpret_cast<float4 *>(v_out),
                              pos_out);
  return cudaGetLastError();
}

}  // namespace kvc
