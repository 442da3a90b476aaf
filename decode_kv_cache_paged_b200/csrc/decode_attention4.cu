// decode_attention4.cu -- decode attention over the 4-bit cache, and decode
// attention that accumulates each cached row's attention weight.
#include <cuda_bf16.h>

#include "int4.cuh"
#include "kvc_internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;

template <int DT>
__device__ __forceinline__ float row_value(const uint8_t *row, int d, int c) {
  if (DT == KVC_F32) return reinterpret_cast<const float *>(row)[c];
  if (DT == KVC_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[c]);
  const uint32_t h = *reinterpret_cast<const uint32_t *>(row + (c / (d / kInt4Groups)) * 4);
  const int code = (row[kInt4Header + c / 2] >> (4 * (c & 1))) & 15;
  return fmaf((float)code, __uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
}

// One CTA per (layer, request, query head); with weights per (layer, request,
// KV head), which then loops over its G query heads.
template <int DT, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(DecodeAttnParams p, int G, int row_bytes) {
  constexpr int W = kThreads / 32, E = D / 32;
  __shared__ float m_s[W], l_s[W], o_s[W][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % p.hkv, r = (blockIdx.x / p.hkv) % p.R, lc = blockIdx.x / (p.hkv * p.R);
  const int len = p.lengths[r];
  const int32_t *bt = p.block_table + (int64_t)r * p.bt_stride;
  const int64_t layer0 = (int64_t)(p.layer_begin + lc) * p.num_pages;
  auto row_of = [&](int j) { return ((layer0 + bt[j / kPage]) * p.hkv + h) * kPage + j % kPage; };
  for (int g = 0; g < G; ++g) {
    const int64_t head = ((int64_t)lc * p.R + r) * p.hq + (int64_t)h * G + g;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = row_value<DT == KVC_F32 ? KVC_F32 : KVC_BF16>(p.q + head * D * (DT == KVC_F32 ? 4 : 2), D, lane + 32 * e);
      o[e] = 0.f;
    }
    auto score = [&](int64_t row) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], row_value<DT>(p.k_pool + row * row_bytes, D, lane + 32 * e), s);
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      return s * p.qscale;
    };
    for (int j = warp; j < len; j += W) {
      const int64_t row = row_of(j);
      const float s = score(row), mn = fmaxf(m, s);
      const float a = exp2f(m - mn), w = exp2f(s - mn);
      m = mn;
      l = l * a + w;
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] = o[e] * a + w * row_value<DT>(p.v_pool + row * row_bytes, D, lane + 32 * e);
    }
    if (lane == 0) {
      m_s[warp] = m;
      l_s[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o_s[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < W; ++w) M = fmaxf(M, m_s[w]);
    for (int w = 0; w < W; ++w)
      if (l_s[w] != 0.f) L += l_s[w] * exp2f(m_s[w] - M);
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float v = 0.f;
      for (int w = 0; w < W; ++w)
        if (l_s[w] != 0.f) v += o_s[w][c] * exp2f(m_s[w] - M);
      p.out[head * D + c] = len > 0 ? v / L : 0.f;
    }
    const float lse2 = M + log2f(L);
    if (p.lse && threadIdx.x == 0) p.lse[head] = len > 0 ? lse2 * kLn2 : -INFINITY;
    if (p.weights) {
      for (int j = warp; j < len; j += W) {
        const int64_t row = row_of(j);
        const float w = exp2f(score(row) - lse2);
        if (lane == 0) p.weights[row] = (g == 0 ? p.decay : 1.f) * p.weights[row] + w;
      }
    }
    __syncthreads();
  }
}

}  // namespace

bool decode_attention4_supported(int dtype, int head_dim, int G) {
  return (dtype == KVC_BF16 || dtype == KVC_F32 || dtype == KVC_INT4) && (head_dim == 64 || head_dim == 128) &&
         (G == 1 || G == 2 || G == 4 || G == 8);
}

cudaError_t launch_decode_attention4(const DecodeAttnParams &p, int head_dim, int dtype, int G, int row_bytes,
                                     cudaStream_t s) {
  const int units = p.layer_count * p.R * p.hkv;
  auto kernel = attend_kernel<KVC_F32, 128>;
  if (dtype == KVC_F32) kernel = head_dim == 128 ? attend_kernel<KVC_F32, 128> : attend_kernel<KVC_F32, 64>;
  if (dtype == KVC_BF16) kernel = head_dim == 128 ? attend_kernel<KVC_BF16, 128> : attend_kernel<KVC_BF16, 64>;
  if (dtype == KVC_INT4) kernel = head_dim == 128 ? attend_kernel<KVC_INT4, 128> : attend_kernel<KVC_INT4, 64>;
  kernel<<<units, kThreads, 0, s>>>(p, G, row_bytes);
  return cudaGetLastError();
}

}  // namespace kvc
