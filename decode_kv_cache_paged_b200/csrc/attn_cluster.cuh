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
// follows the cache.  With p.part_o the CTAs of a unit are no cluster and leave
// their states for a merge launch (few long requests, decode_attention4.cu).
#pragma once
#include "kvc_internal.h"
#include "tc_ptx.cuh"

namespace kvc {
namespace {

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

__device__ __forceinline__ float attn_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  u.rank = blockIdx.x % u.cs;  // clusters are runs of u.cs blocks
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
template <int W>
struct AttnMerge {
  float m[8], l[8];                    // this CTA's running maximum (base 2) and sum per head
  float part[W][8];                    // the warps' factors
  float all_m[16][8], all_l[16][8];    // every CTA's
  float fac[16][8];                    // exp2(m of the CTA - m of the unit) / sum of the unit
  float lse2[8];                       // the unit's log2-sum-exp2 (+inf: reads as without rows)
};

// Adds the weights of this CTA's rows from their base-2 scores [page][G][16].
// A thread takes four rows of a page at a time (a page's 16 weights are one
// 64-byte run) and starts the reads of kBatch such quads before the first is
// used: one after the other the loop waits for memory once per quad, which
// cost a third of the step at 2048 rows.
template <int NT, int G, bool KEEP_NAN>
__device__ __forceinline__ void attn_add_weights(const DecodeAttnParams &p, const AttnUnit &u,
                                                 const float (&lse2)[8], const float *scores) {
  constexpr int kBatch = 4;
  const int rows = min(u.len, u.pg1 * kPage) - u.pg0 * kPage;
  float *w0 = p.weights + ((int64_t)u.l * p.num_pages * p.hkv + u.h) * kPage;
  const int64_t page_stride = (int64_t)p.hkv * kPage;
  // a head that reads as one without rows has lse2 = +inf: its finite scores give 0, the others NaN, which max drops
  auto weight = [](float s) { return KEEP_NAN ? attn_ex2(s) : fmaxf(attn_ex2(s), 0.f); };
  for (int j0 = threadIdx.x * 4; j0 < rows; j0 += 4 * NT * kBatch) {
    float4 w[kBatch];
    float *at[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int j = j0 + b * 4 * NT;
      if (j < rows) at[b] = w0 + u.bt[u.pg0 + j / kPage] * page_stride + j % kPage;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (j0 + b * 4 * NT < rows) w[b] = *reinterpret_cast<const float4 *>(at[b]);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int j = j0 + b * 4 * NT;
      if (j >= rows) continue;
      const float *sc = scores + (j / kPage) * (kPage * G) + j % kPage;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float4 v = *reinterpret_cast<const float4 *>(sc + g * kPage);
        a.x += weight(v.x - lse2[g]);
        a.y += weight(v.y - lse2[g]);
        a.z += weight(v.z - lse2[g]);
        a.w += weight(v.w - lse2[g]);
      }
      a = make_float4(fmaf(p.decay, w[b].x, a.x), fmaf(p.decay, w[b].y, a.y), fmaf(p.decay, w[b].z, a.z),
                      fmaf(p.decay, w[b].w, a.w));
      if (j + 4 <= rows) {
        *reinterpret_cast<float4 *>(at[b]) = a;
      } else {  // the last rows: what lies past them stays
        at[b][0] = a.x;
        if (j + 1 < rows) at[b][1] = a.y;
        if (j + 2 < rows) at[b][2] = a.z;
      }
    }
  }
}

__device__ __forceinline__ void attn_write_lse(const DecodeAttnParams &p, int64_t head, float lse2) {
  if (p.lse) p.lse[head] = lse2 * 0.6931471805599453f;
  if (p.lse2) p.lse2[head] = lse2;
}

// Merges the warps' and then the CTAs' states and writes the outputs; with
// p.part_o, the CTA's share for a merge launch instead (no cluster).
//   red:  [W][G][D] the warps' sums, m_s, l_s: [W][G] their maxima and sums
//         (a warp without rows has l = 0); the caller has synchronised.
//   scores: [pages of this CTA][G][16] base-2 scores, or null (no weights).
// A head whose sum is 0 or, unless KEEP_NAN (the 4-bit cache), NaN reads as one
// without rows: out = 0, lse = -inf, no weights.
// Every thread of the CTA calls it.
template <int D, int W, int NT, bool KEEP_NAN>
__device__ __forceinline__ void attn_finish(const DecodeAttnParams &p, const AttnUnit &u, int G, float *red,
                                            const float *m_s, const float *l_s, AttnMerge<W> &mg, float *scores) {
  const int tid = threadIdx.x;
  const int64_t head0 = ((int64_t)u.lc * p.R + u.r) * p.hq + (int64_t)u.h * G;
  const bool alone = u.cs == 1 && !p.part_o;
  auto finish_head = [&](int g, float M, float L, bool none, bool write) {
    const float lse2 = M + log2f(L);
    mg.lse2[g] = none ? INFINITY : lse2;
    if (write) attn_write_lse(p, head0 + g, u.len > 0 && !none ? lse2 : -INFINITY);
  };
  // the warps' factors; a CTA that has the unit to itself divides by the sum at once
  for (int i = tid; i < W * 8; i += NT) {
    const int w = i >> 3, g = i & 7;
    if (g >= G) continue;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int x = 0; x < W; ++x) M = fmaxf(M, m_s[x * G + g]);
#pragma unroll
    for (int x = 0; x < W; ++x)
      if (l_s[x * G + g] != 0.f) L = fmaf(l_s[x * G + g], attn_ex2(m_s[x * G + g] - M), L);
    const float f = l_s[w * G + g] != 0.f ? attn_ex2(m_s[w * G + g] - M) : 0.f;
    const bool none = !KEEP_NAN && !(L > 0.f);
    mg.part[w][g] = !alone || f == 0.f ? f : none ? 0.f : f / L;
    if (w == 0) {
      mg.m[g] = M;
      mg.l[g] = L;
      if (p.part_o) {
        const int64_t pu = (head0 + g) * u.cs + u.rank;
        p.part_ml[pu * 2] = M;
        p.part_ml[pu * 2 + 1] = L;
      }
      if (alone) finish_head(g, M, L, none, true);
    }
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += NT) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = mg.part[w][i / D];
      if (f != 0.f) o = fmaf(red[w * G * D + i], f, o);
    }
    if (p.part_o)
      p.part_o[((head0 + i / D) * u.cs + u.rank) * D + i % D] = o;
    else if (u.cs > 1)
      red[i] = o;
    else
      p.out[head0 * D + i] = o;
  }
  if (p.part_o) return;
  if (u.cs > 1) {
    cluster_sync_all();
    for (int i = tid; i < u.cs * 8; i += NT) {
      const int c = i >> 3, g = i & 7;
      if (g < G) {
        mg.all_m[c][g] = ld_cluster(&mg.m[g], c);
        mg.all_l[c][g] = ld_cluster(&mg.l[g], c);
      }
    }
    __syncthreads();
    for (int i = tid; i < u.cs * 8; i += NT) {
      const int c = i >> 3, g = i & 7;
      if (g >= G) continue;
      float M = -INFINITY, L = 0.f;
      for (int x = 0; x < u.cs; ++x) M = fmaxf(M, mg.all_m[x][g]);
      for (int x = 0; x < u.cs; ++x)
        if (mg.all_l[x][g] != 0.f) L = fmaf(mg.all_l[x][g], attn_ex2(mg.all_m[x][g] - M), L);
      const bool none = !KEEP_NAN && !(L > 0.f);
      mg.fac[c][g] = mg.all_l[c][g] != 0.f && !none ? attn_ex2(mg.all_m[c][g] - M) / L : 0.f;
      if (c == 0) finish_head(g, M, L, none, u.rank == 0);
    }
    __syncthreads();
    // outputs: each CTA of the cluster writes its share of the G * D values
    const int share = (G * D + u.cs - 1) / u.cs;
    for (int i = u.rank * share + tid; i < min(G * D, (u.rank + 1) * share); i += NT) {
      float o = 0.f;
#pragma unroll 4
      for (int x = 0; x < u.cs; ++x) {
        const float f = mg.fac[x][i / D], v = ld_cluster(&red[i], x);
        if (f != 0.f) o = fmaf(v, f, o);
      }
      p.out[head0 * D + i] = o;
    }
  }
  if (scores) {
    float lse2[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) lse2[x] = x < G ? mg.lse2[x] : 0.f;
    switch (G) {
      case 1: attn_add_weights<NT, 1, KEEP_NAN>(p, u, lse2, scores); break;
      case 2: attn_add_weights<NT, 2, KEEP_NAN>(p, u, lse2, scores); break;
      case 4: attn_add_weights<NT, 4, KEEP_NAN>(p, u, lse2, scores); break;
      default: attn_add_weights<NT, 8, KEEP_NAN>(p, u, lse2, scores);
    }
  }
  if (u.cs > 1) cluster_sync_all();  // the others may still read this CTA's shared memory
}

}  // namespace
}  // namespace kvc
