// attn_cluster.cuh -- what the cluster forms of decode attention share: the
// split of a unit's pages over the CTAs of a thread-block cluster, and the
// epilogue that merges the CTAs' softmax states over distributed shared
// memory, writes the outputs and adds the rows' attention weights.
//
// A unit is one (layer, request, KV head).  Its cluster of 1 to 16 CTAs walks
// the request's pages, each CTA a contiguous share, so a unit needs no
// partials in global memory and no second launch, and the whole unit's
// log-sum-exp is known to every CTA while the base-2 scores of its rows still
// sit in its shared memory: the weights exp2(score - lse) then cost one read
// and one write of 4 bytes per row, and no second pass over the keys.  The
// share comes from the request's length on the device, so a captured launch
// follows the cache.
#pragma once
#include "kvc_internal.h"
#include "tc_ptx.cuh"

namespace kvc {
namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// float of another CTA of the cluster, at the address that `p` has here
__device__ __forceinline__ float ld_cluster(const float *p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

struct AttnUnit {
  int rank, cs;              // this CTA in its cluster, and the cluster's size
  int lc, l, r, h;           // layer (in the call, in the cache), request, KV head
  int len, pg0, pg1;         // the request's rows; this CTA's pages [pg0, pg1)
  const int32_t *bt;
};

__device__ __forceinline__ AttnUnit attn_unit(const DecodeAttnParams &p) {
  AttnUnit u;
  u.cs = p.nsplit;
  u.rank = u.cs > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / u.cs;
  u.h = unit % p.hkv;
  u.r = (unit / p.hkv) % p.R;
  u.lc = unit / (p.hkv * p.R);
  u.l = p.layer_begin + u.lc;
  u.len = p.lengths[u.r];
  const int n_pages = (u.len + kPage - 1) / kPage;
  const int per = (n_pages + u.cs - 1) / u.cs;
  u.pg0 = min(n_pages, u.rank * per);
  u.pg1 = min(n_pages, u.pg0 + per);
  u.bt = p.block_table + (int64_t)u.r * p.bt_stride;
  return u;
}

// Shared scratch of the epilogue.
struct AttnMerge {
  float m[8], l[8];                // this CTA's running maximum (base 2) and sum per head
  float all_m[16][8], all_l[16][8];  // every CTA's
  float fac[16][8];                // exp2(m of the CTA - m of the unit) / sum of the unit
  float lse2[8];                   // the unit's log2-sum-exp2
};

// Merges the warps' and then the CTAs' states and writes the outputs.
//   red:  [W][G][D] the warps' sums, m_s, l_s: [W][G] their maxima and sums
//         (a warp without rows has l = 0); the caller has synchronised.
//   scores: [rows of this CTA][G] base-2 scores, or null (no weights).
// Every thread of the CTA calls it.
template <int D, int W, int NT>
__device__ __forceinline__ void attn_finish(const DecodeAttnParams &p, const AttnUnit &u, int G, float *red,
                                            const float *m_s, const float *l_s, AttnMerge &mg, const float *scores) {
  const int tid = threadIdx.x;
  for (int i = tid; i < G * D; i += NT) {
    const int g = i / D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, m_s[w * G + g]);
    float o = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float lw = l_s[w * G + g];
      if (lw == 0.f) continue;
      const float sc = exp2f(m_s[w * G + g] - M);
      o = fmaf(red[w * G * D + i], sc, o);
      l = fmaf(lw, sc, l);
    }
    red[i] = o;
    if (i % D == 0) {
      mg.m[g] = M;
      mg.l[g] = l;
    }
  }
  if (u.cs > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const int64_t head0 = ((int64_t)u.lc * p.R + u.r) * p.hq + (int64_t)u.h * G;
  for (int i = tid; i < u.cs * 8; i += NT) {
    const int c = i >> 3, g = i & 7;
    if (g < G) {
      mg.all_m[c][g] = u.cs > 1 ? ld_cluster(&mg.m[g], c) : mg.m[g];
      mg.all_l[c][g] = u.cs > 1 ? ld_cluster(&mg.l[g], c) : mg.l[g];
    }
  }
  __syncthreads();
  for (int i = tid; i < u.cs * 8; i += NT) {
    const int c = i >> 3, g = i & 7;
    if (g >= G) continue;
    float M = -INFINITY, L = 0.f;
    for (int x = 0; x < u.cs; ++x) M = fmaxf(M, mg.all_m[x][g]);
    for (int x = 0; x < u.cs; ++x)
      if (mg.all_l[x][g] != 0.f) L = fmaf(mg.all_l[x][g], exp2f(mg.all_m[x][g] - M), L);
    mg.fac[c][g] = mg.all_l[c][g] != 0.f ? exp2f(mg.all_m[c][g] - M) / L : 0.f;
    if (c == 0) {
      const float lse2 = M + log2f(L);
      mg.lse2[g] = lse2;
      if (u.rank == 0 && p.lse) p.lse[head0 + g] = u.len > 0 ? lse2 * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncthreads();
  // outputs: each CTA of the cluster writes its share of the G * D values
  const int share = (G * D + u.cs - 1) / u.cs;
  for (int i = u.rank * share + tid; i < min(G * D, (u.rank + 1) * share); i += NT) {
    float o = 0.f;
    if (u.cs > 1) {
#pragma unroll 4
      for (int x = 0; x < u.cs; ++x) {
        const float f = mg.fac[x][i / D], v = ld_cluster(&red[i], x);
        if (f != 0.f) o = fmaf(v, f, o);
      }
    } else {
      o = red[i] * mg.fac[0][i / D];
    }
    p.out[head0 * D + i] = u.len > 0 ? o : 0.f;
  }
  if (scores) {
    float lse2[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) lse2[x] = x < G ? mg.lse2[x] : 0.f;
    const int rows = min(u.len, u.pg1 * kPage) - u.pg0 * kPage;
    for (int j = tid; j < rows; j += NT) {
      float w = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (x < G) w += exp2f(scores[j * G + x] - lse2[x]);
      const int64_t at = (((int64_t)u.l * p.num_pages + u.bt[u.pg0 + j / kPage]) * p.hkv + u.h) * kPage + j % kPage;
      p.weights[at] = fmaf(p.decay, p.weights[at], w);
    }
  }
  if (u.cs > 1) cluster_sync_all();  // the others may still read this CTA's shared memory
}

}  // namespace
}  // namespace kvc
