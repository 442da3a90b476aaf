// decode_attention4.cu -- one decode step of grouped-query attention over the
// 4-bit cache (KVC_INT4), with or without accumulating the rows' attention
// weights.
//
// What it computes: as decode_attention.cu, with k_j and v_j the values that
// the codes of int4.cuh stand for.
//
// Design (B200).  A cached row is 80 bytes (D = 128) against 256 in bf16, so
// at the HBM rate an SM meets a page of 16 rows (2.5 KB of K and V) every 100
// clocks: 400 issue slots in which 4096 codes become operands of 2 * 4096 * G
// products.  The CUDA cores alone need more than that for the products, and
// feeding tcgen05 would cost a write and a read of the decoded page through
// shared memory (8 KB each way, 160 clocks of its port).  So the codes are
// decoded in registers, straight into the fragments of warp-level mma with the
// rows on M and the query heads on N:
//   S^T[16 rows x 8] = K . Q^T per group       m16n8k16, fp16
//   O^T[D x 8]      += V^T . P^T               m16n8k16, bf16
// Which channel sits at which k of the first product, and which at which row
// of the second, is free as long as both operands agree, so a lane reads its
// codes where they lie and no transposing load is needed.  The logic pipe (one
// and-or, shift or byte permute every two clocks per scheduler) is what the
// decoding fills, so each form is chosen for the fewest of those:
//   * K: the low and the high nibble of a byte, masked in place, are the fp16
//     subnormals code * 2^-24 and code * 2^-20: a word of eight codes takes one
//     shift and four ands, and nothing else.  The query is the other operand,
//     scaled per head to |q| < 2048 and split into an integer and the rest, both
//     fp16: the integers' products and sums are exact (the tensor cores
//     truncate each product to the place of the largest, which costs 5e-6 of a
//     score otherwise); the rest's have columns of their own, or join the sum (8
//     heads) with a truncation the size of an fp32 rounding.  A group is a sum of its own,
//     which s multiplies in fp32, where lo * the group's sum of q joins it.
//     (8-bit floats would take fewer ands, but their products expand to fp16
//     ones with a conversion per two codes: measured 24 instructions of the
//     logic pipe more per page.)
//   * V: the low and the high nibble of a byte, masked in place, are the bf16
//     numbers code * 2^-133 and code * 2^-129 (linear from the subnormals
//     through the first binade), so one byte permute and two ands make four operands, and
//     one fma by (s * 2^69 or s * 2^65, -z s / 2^64) gives s (code - z) / 2^64
//     exactly.  mid is one more product, with a row of ones beside it that
//     gives the softmax's sum.
//   * P enters as three bf16 terms, all of its 24 bits: two would leave 2^-17 of
//     a weight, 1.2e-6 of an output where fp32 sums leave 3e-7.
//   * With at most 4 query heads per KV head the two parts of a head's query, and
//     the first two terms of its P, are neighbouring columns of one product, which
//     one lane holds: no lane repeats another's softmax, and a head's sums are one.
//     P's third term takes another product; with 8 heads each part and term takes
//     one.
//   * The running maximum is lazy: two pages' scores are compared with it and
//     the sums are rescaled only when one exceeds it by more than 2^8, so a
//     page needs no reduction across lanes.
// Each warp walks its own pairs of pages through its own ring of slots, one
// bulk copy each for the K and the V rows of a page.  The split over a cluster
// and the merge are attn_cluster.cuh's.
// Every mbarrier wait is bounded (tc_ptx.cuh).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attn_cluster.cuh"
#include "int4.cuh"

namespace kvc {
namespace {

constexpr size_t kMaxSmem = 227 * 1024 - 4608;  // the most for one, less the static shared memory
constexpr int kPair = 2;    // pages per slot: K, V of the first, K, V of the second
constexpr int kStages = 2;  // slots per warp

template <int D>
struct Shape4 {
  static constexpr int kRow = int4_row_bytes(D);
  static constexpr int kPageBytes = kPage * kRow;       // K (or V) of one page
  static constexpr int kWords = D / 32;  // 32-bit words of codes per lane and K row
  static constexpr int kTiles = D / 16;  // products per page on the V side
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = A . B without a sum to add to; bf16
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// fp16: d = A . B, and d += A . B
__device__ __forceinline__ void mma16816h_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816h(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (lo, hi) rounded to a bf16 pair, lo in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// s * 2^69, s * 2^65 and -z s / 2^64 of a pair of V rows, from their words' high halves
__device__ __forceinline__ void unpack_steps(uint32_t r, uint32_t &s_lo, uint32_t &s_hi, uint32_t &off) {
  const uint32_t s2 = r & 0xfff0fff0u;
  s_lo = s2 + 0x22802280u;
  s_hi = s2 + 0x20802080u;
  off = mul_bf16x2(r & 0x000f000fu, s2 + 0xa280a280u);  // z * 2^-133 by -s * 2^69
}
constexpr uint32_t kOnes = 0x3f803f80u;
constexpr float kLazy = 8.f;  // a score may exceed the running maximum by this much (base 2)

// What a launch does: the step; the step with the weights added from scores
// kept in shared memory; the weights alone, from the keys and the step's
// log-sum-exp (p.lse2), for rows too many to keep the scores of.
enum Mode4 { kStep, kStepWeights, kWeights };

// GP: query heads that a product's 8 columns hold, 4 (G <= 4: two columns each) or 8.  W: warps of a CTA.
template <int GP, Mode4 MODE, int W>
constexpr int kFit4 = (GP == 8 && MODE != kWeights ? 12 : 16) / W;  // CTAs whose registers fit an SM

template <int D, int GP, Mode4 MODE, int W>
__global__ void __launch_bounds__(32 * W, kFit4<GP, MODE, W>) decode_attention4_kernel(DecodeAttnParams p, int G) {
  using S = Shape4<D>;
  constexpr int kWarps = W, kThreads = 32 * W;
  constexpr bool kValues = MODE != kWeights;
  constexpr int kYStride = (kValues ? 2 : 1) * S::kPageBytes;  // from a page of a slot to the next
  constexpr int kSlot = kPair * kYStride;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_align<128>(smem_raw);
  float *scores = reinterpret_cast<float *>(smem + W * kStages * kSlot);  // [pages of this CTA][G][16] (kStepWeights)
  __shared__ float m_s[kWarps * 8], l_s[kWarps * 8];
  __shared__ AttnMerge<W> mg;
  __shared__ __align__(8) uint64_t full[kWarps][kStages];
  __shared__ int abort_flag_s;
  volatile int *abort_flag = &abort_flag_s;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, t = lane & 3;  // a fragment's row and column index of this lane
  const AttnUnit u = attn_unit(p);
  // this warp's pairs of pages: u.pg0 + 2 (warp + k * kWarps), the last one maybe half
  const int n_pages = u.pg1 - u.pg0, first = u.pg0 + kPair * warp;
  const int n_my = n_pages > kPair * warp ? (n_pages - kPair * warp + kPair * kWarps - 1) / (kPair * kWarps) : 0;
  const int rows_end = min(u.len, u.pg1 * kPage);
  uint8_t *ring = smem + warp * kStages * kSlot;

  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&full[w][i], 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  // page ids of this warp's pages, 32 at a time, one per lane; the next 32
  // are on their way before they are needed
  auto load_ids = [&](int k0) {
    const int pg = first + (k0 + lane / kPair) * kPair * kWarps + lane % kPair;
    return pg < u.pg1 ? u.bt[pg] : -1;
  };
  int ids = load_ids(0), ids_next = load_ids(32 / kPair);
  int ids_base = 0;
  const uint32_t ring_u = smem_u32(ring);
  const int page_stride = p.hkv * S::kPageBytes;  // bytes from a page id to the next in a pool
  const uint8_t *pool = (kValues && (lane & 1) ? p.v_pool : p.k_pool) +
                        ((int64_t)u.l * p.num_pages * p.hkv + u.h) * S::kPageBytes;  // page 0 of this unit
  auto issue_pair = [&](int k) {
    if (k >= ids_base + 32 / kPair) {
      ids = ids_next;
      ids_base += 32 / kPair;
      ids_next = load_ids(ids_base + 32 / kPair);
    }
    const int slot = k % kStages;
    // lanes 0..3 copy K, V of the first page, K, V of the second; without values lanes 0 and 1 the pages' K
    constexpr int kParts = kValues ? 2 : 1;
    const int id = __shfl_sync(0xffffffffu, ids, kPair * (k - ids_base) + (lane / kParts) % kPair);
    const bool both = __shfl_sync(0xffffffffu, ids, kPair * (k - ids_base) + kPair - 1) >= 0;
    if (lane == 0) mbar_expect_tx(&full[warp][slot], (uint32_t)(both ? kSlot : kSlot / 2));
    __syncwarp();
    if (lane < (both ? kParts * kPair : kParts))
      bulk_load(ring_u + slot * kSlot + lane * S::kPageBytes, pool + (int64_t)id * page_stride,
                (uint32_t)S::kPageBytes, &full[warp][slot]);
  };
  for (int k = 0; k < min(n_my, kStages); ++k) issue_pair(k);

  // query fragments.  Column n: GP = 4: head n / 2, its integers in even columns
  // and the rest in odd ones, so that a lane's two columns are one head; GP = 8:
  // head n, the two parts in two tiles.  A smaller group repeats.  Products 2 gr
  // and 2 gr + 1 are group gr's, with this lane's unit t of it: low nibbles
  // first, then high ones (times 2^-4: their codes are 2^4 larger).
  constexpr int kQt = GP == 4 ? 1 : 2;
  constexpr int C = GP == 4 ? 1 : 2;  // heads of this lane: head t, or 2 t and 2 t + 1
  const int head_of_lane = C * t;
  uint32_t qb[kQt][2 * kInt4Groups][2];
  float qsum[kInt4Groups][C];  // sums of q beside lo
  float lam[C];                // from a head's sum to base-2 scores
  {
    const int g = (GP == 4 ? n >> 1 : n) % G;
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p.q) +
                        ((((int64_t)u.lc * p.R + u.r) * p.hq + (int64_t)u.h * G + g) * D + t * (D / 16));
    float x[kInt4Groups][D / 16], top = 0.f, bad = 0.f, sum[kInt4Groups];
    if (reinterpret_cast<uintptr_t>(p.q) % 16 == 0) {  // the unit in one read
#pragma unroll
      for (int gr = 0; gr < kInt4Groups; ++gr) {
        uint32_t v[D / 32];
        if constexpr (D == 128) {
          const uint4 r = *reinterpret_cast<const uint4 *>(q + gr * (D / 4));
          v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
        } else {
          const uint2 r = *reinterpret_cast<const uint2 *>(q + gr * (D / 4));
          v[0] = r.x, v[1] = r.y;
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x[gr][2 * i] = bf16_lo(v[i]), x[gr][2 * i + 1] = bf16_hi(v[i]);
      }
    } else {
#pragma unroll
      for (int gr = 0; gr < kInt4Groups; ++gr)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) x[gr][i] = bf16_lo(q[gr * (D / 4) + i]);
    }
#pragma unroll
    for (int gr = 0; gr < kInt4Groups; ++gr)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        top = fmaxf(top, fabsf(x[gr][i]));
        bad = fmaf(x[gr][i], 0.f, bad);  // NaN once a query value is infinite or NaN
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    bad += __shfl_xor_sync(0xffffffffu, bad, 1);
    bad += __shfl_xor_sync(0xffffffffu, bad, 2);
    // sigma: the power of two that brings the head's largest |q| into [1024, 2048)
    const int ex = max(-120, min(100, 137 - (int)(__float_as_uint(top) >> 23)));
    const float sigma = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
    for (int gr = 0; gr < kInt4Groups; ++gr) {
      sum[gr] = bad;
      float part[2][D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float v = x[gr][i] * sigma;
        sum[gr] += v;
        part[0][i] = rintf(v);
        part[1][i] = v - part[0][i];
      }
#pragma unroll
      for (int z = 0; z < kQt; ++z) {
        float c[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) c[i] = (GP == 4 ? n & 1 : z) ? part[1][i] : part[0][i];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if constexpr (D == 128) {  // codes i and i + 4 of a word share a register
            qb[z][2 * gr + y][0] = pack_f16(c[2 * y], c[2 * y + 4]);
            qb[z][2 * gr + y][1] = pack_f16(c[2 * y + 1] * 0.0625f, c[2 * y + 5] * 0.0625f);
          } else {  // codes i of two groups share one: the other group's place is 0
            const float a = c[2 * y], b = c[2 * y + 1] * 0.0625f;
            qb[z][2 * gr + y][0] = (gr & 1) ? pack_f16(0.f, a) : pack_f16(a, 0.f);
            qb[z][2 * gr + y][1] = (gr & 1) ? pack_f16(0.f, b) : pack_f16(b, 0.f);
          }
        }
      }
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
      sum[gr] *= 0x1p-24f;  // the codes' unit
    }
    // column c's values sit with lanes n = c
    const float lam_n = p.qscale * 0x1p24f * __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < kInt4Groups; ++i) qsum[i][c] = __shfl_sync(0xffffffffu, sum[i], (2 * t + c) * 4);
      lam[c] = __shfl_sync(0xffffffffu, lam_n, (2 * t + c) * 4);
    }
  }

  constexpr int kPt = GP == 4 ? 2 : 3;  // products for the terms of P
  // rows of a page: fragment rows n and n + 8 are page rows ra and ra + 1, an
  // order in which no two lanes of a shared-memory phase meet in a bank
  const int ra = (n & 1) ? ((n + 3) & 7) + 8 : n;
  [[maybe_unused]] float w_lse[C];
  if constexpr (MODE == kWeights) {
    const float *src = p.lse2 + ((int64_t)u.lc * p.R + u.r) * p.hq + (int64_t)u.h * G;
#pragma unroll
    for (int c = 0; c < C; ++c)
      w_lse[c] = head_of_lane + c < G ? src[head_of_lane + c] : INFINITY;  // a repeated head adds exp2(-inf)
  }
  const int v0 = 2 * t, v1 = ((2 * t + 4) & 7) + 8;  // P's rows 2t and 2t + 1; v0 + 1 and v1 + 1 are 2t + 8 and 2t + 9

  [[maybe_unused]] float *const w_base = p.weights + ((int64_t)u.l * p.num_pages * p.hkv + u.h) * kPage + ra + (t & 1);
  [[maybe_unused]] const int w_stride = p.hkv * kPage;

  float m[C];  // running maxima (base 2)
  float o[S::kTiles][2 * C], e[2 * C];  // [x C + c]: fragment rows n + 8 x; e: the mid term (x = 0), the sum of P
#pragma unroll
  for (int c = 0; c < C; ++c) m[c] = -INFINITY;
#pragma unroll
  for (int i = 0; i < S::kTiles; ++i)
#pragma unroll
    for (int x = 0; x < 2 * C; ++x) o[i][x] = 0.f;
#pragma unroll
  for (int x = 0; x < 2 * C; ++x) e[x] = 0.f;
  // adds a product to a sum; GP = 4: the columns of P's first and second terms together
  auto add_tile = [](float (&sum)[2 * C], const float (&d)[4]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if constexpr (C == 1) {
        sum[x] += d[2 * x] + d[2 * x + 1];
      } else {
        sum[x * C] += d[2 * x];
        sum[x * C + C - 1] += d[2 * x + 1];
      }
    }
  };

  int k = 0;
  for (; k < n_my; ++k) {
    const int slot = k % kStages;
    [[maybe_unused]] float w_old = 0.f;
    [[maybe_unused]] float *w_at = nullptr;
    if constexpr (MODE == kWeights) {  // this lane's row (page t / 2, row ra + t % 2): its weight, read ahead of the wait
      const int pg = first + k * kPair * kWarps + (t >> 1);
      if (pg < u.pg1 && pg * kPage + ra + (t & 1) < u.len) {
        w_at = w_base + (int64_t)u.bt[pg] * w_stride;
        w_old = *w_at;
      }
    }
    const uint32_t parity = (uint32_t)((k / kStages) & 1);
    if (__any_sync(0xffffffffu, !mbar_try(&full[warp][slot], parity)) &&
        __any_sync(0xffffffffu, !mbar_wait(&full[warp][slot], parity, abort_flag, p.status)))
      break;
    const uint8_t *base = ring + slot * kSlot;
    const int valid = rows_end - (first + k * kPair * kWarps) * kPage;  // rows here; what lies past them is anything

    // 1. base-2 scores s[y][x C + c] of page row ra + x
    float s[kPair][2 * C];
#pragma unroll
    for (int y = 0; y < kPair; ++y) {
      const uint8_t *row0 = base + y * kYStride + ra * S::kRow, *row1 = row0 + S::kRow;
      const uint4 h0 = *reinterpret_cast<const uint4 *>(row0), h1 = *reinterpret_cast<const uint4 *>(row1);
      const uint32_t ga[4] = {h0.x, h0.y, h0.z, h0.w}, gb[4] = {h1.x, h1.y, h1.z, h1.w};
      uint32_t wa[S::kWords], wb[S::kWords];
      if constexpr (S::kWords == 4) {
        const uint4 a = *reinterpret_cast<const uint4 *>(row0 + kInt4Header + t * 16);
        const uint4 b = *reinterpret_cast<const uint4 *>(row1 + kInt4Header + t * 16);
        wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
        wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
      } else {
        const uint2 a = *reinterpret_cast<const uint2 *>(row0 + kInt4Header + t * 8);
        const uint2 b = *reinterpret_cast<const uint2 *>(row1 + kInt4Header + t * 8);
        wa[0] = a.x, wa[1] = a.y;
        wb[0] = b.x, wb[1] = b.y;
      }
      float acc[2 * C];
      // lo by the sums of q
#pragma unroll
      for (int c = 0; c < C; ++c) {
        acc[c] = acc[C + c] = 0.f;
#pragma unroll
        for (int i = 0; i < kInt4Groups; ++i) {
          acc[c] = fmaf(bf16_lo(ga[i]), qsum[i][c], acc[c]);
          acc[C + c] = fmaf(bf16_lo(gb[i]), qsum[i][c], acc[C + c]);
        }
      }
#pragma unroll
      for (int gr = 0; gr < kInt4Groups; ++gr) {
        const uint32_t a = wa[D == 128 ? gr : gr / 2], b = wb[D == 128 ? gr : gr / 2];
        const uint32_t a0 = a & 0x000f000fu, a1 = a & 0x00f000f0u, a2 = a >> 8 & 0x000f000fu, a3 = a >> 8 & 0x00f000f0u;
        const uint32_t b0 = b & 0x000f000fu, b1 = b & 0x00f000f0u, b2 = b >> 8 & 0x000f000fu, b3 = b >> 8 & 0x00f000f0u;
        const float sa = __uint_as_float(ga[gr] & 0xfff00000u), sb = __uint_as_float(gb[gr] & 0xfff00000u);
        float d[4];
        mma16816h_zero(d, a0, b0, a1, b1, qb[0][2 * gr][0], qb[0][2 * gr][1]);
        mma16816h(d, a2, b2, a3, b3, qb[0][2 * gr + 1][0], qb[0][2 * gr + 1][1]);
        if constexpr (kQt == 2) {
          mma16816h(d, a0, b0, a1, b1, qb[kQt - 1][2 * gr][0], qb[kQt - 1][2 * gr][1]);
          mma16816h(d, a2, b2, a3, b3, qb[kQt - 1][2 * gr + 1][0], qb[kQt - 1][2 * gr + 1][1]);
        }
        if constexpr (C == 1) {  // the columns of the head's two parts
          acc[0] = fmaf(sa, d[1], fmaf(sa, d[0], acc[0]));
          acc[1] = fmaf(sb, d[3], fmaf(sb, d[2], acc[1]));
        } else {
          acc[0] = fmaf(sa, d[0], acc[0]);
          acc[C - 1] = fmaf(sa, d[1], acc[C - 1]);
          acc[C] = fmaf(sb, d[2], acc[C]);
          acc[2 * C - 1] = fmaf(sb, d[3], acc[2 * C - 1]);
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        s[y][c] = acc[c] * lam[c];
        s[y][C + c] = acc[C + c] * lam[c];
      }
    }
    if (MODE != kWeights && valid < kPair * kPage) {
#pragma unroll
      for (int y = 0; y < kPair; ++y) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (y * kPage + ra >= valid) s[y][c] = -INFINITY;
          if (y * kPage + ra + 1 >= valid) s[y][C + c] = -INFINITY;
        }
      }
    }
    if constexpr (MODE == kWeights) {
      static_assert(kPair == 2);
      // sums over this lane's heads, then over the four lanes of a row, each left with one row
      float a[kPair], b[kPair];
#pragma unroll
      for (int y = 0; y < kPair; ++y) {
        a[y] = attn_ex2(s[y][0] - w_lse[0]);
        b[y] = attn_ex2(s[y][C] - w_lse[0]);
        if constexpr (C == 2) {
          a[y] += attn_ex2(s[y][C - 1] - w_lse[C - 1]);
          b[y] += attn_ex2(s[y][2 * C - 1] - w_lse[C - 1]);
        }
      }
      const bool hi = t & 2, odd = t & 1;
      float x = (hi ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, hi ? a[0] : a[1], 2);
      float z = (hi ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, hi ? b[0] : b[1], 2);
      x = (odd ? z : x) + __shfl_xor_sync(0xffffffffu, odd ? x : z, 1);
      if (w_at) *w_at = fmaf(p.decay, w_old, x);
      __syncwarp();  // every lane has read the slot
      if (k + kStages < n_my) issue_pair(k + kStages);
      continue;
    }
    if constexpr (MODE == kStepWeights) {
#pragma unroll
      for (int y = 0; y < kPair; ++y) {
        // the buffer holds whole pages: the second page of the last pair may lie past it
        if (y * kPage >= valid) continue;
        float *dst = scores + ((kPair * (warp + k * kWarps) + y) * G + head_of_lane) * kPage + ra;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (head_of_lane + c < G) *reinterpret_cast<float2 *>(dst + c * kPage) = make_float2(s[y][c], s[y][C + c]);
      }
    }

    // 2. lazy running maximum
    float top[C];
    bool above = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      top[c] = fmaxf(fmaxf(s[0][c], s[0][C + c]), fmaxf(s[1][c], s[1][C + c]));
      above |= top[c] > m[c] + kLazy;
    }
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float now = fmaxf(top[c], m[c]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, x));
        const float f = attn_ex2(m[c] - now);  // now > -inf: a slot has a row
        m[c] = now;
#pragma unroll
        for (int i = 0; i < S::kTiles; ++i) {
          o[i][c] *= f;
          o[i][C + c] *= f;
        }
        e[c] *= f;
        e[C + c] *= f;
      }
    }
    // 3. P as three bf16 terms, transposed into the second product's fragments.
    // The pairs that are rounded together are the two rows (C = 1) or the two heads.
    uint32_t bp[kPair][kPt][2];
#pragma unroll
    for (int y = 0; y < kPair; ++y) {
      uint32_t h[C], l[C], r[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int at = C == 1 ? 0 : C * i;  // of s: the pair is at and at + 1
        const float p0 = attn_ex2(s[y][at] - m[0]), p1 = attn_ex2(s[y][at + 1] - m[C - 1]);
        h[i] = pack_bf16(p0, p1);
        const float r0 = p0 - bf16_lo(h[i]), r1 = p1 - bf16_hi(h[i]);
        l[i] = pack_bf16(r0, r1);
        // what is left has eight bits
        r[i] = __byte_perm(__float_as_uint(r0 - bf16_lo(l[i])), __float_as_uint(r1 - bf16_hi(l[i])), 0x7632);
      }
      if constexpr (C == 1) {  // columns 2t and 2t + 1: the first two terms; the third and nothing
        bp[y][0][0] = transpose8x8(__byte_perm(h[0], l[0], 0x5410));
        bp[y][0][1] = transpose8x8(__byte_perm(h[0], l[0], 0x7632));
        bp[y][1][0] = transpose8x8(r[0] & 0xffffu);
        bp[y][1][1] = transpose8x8(r[0] >> 16);
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          bp[y][0][x] = transpose8x8(h[x % C]);
          bp[y][1][x] = transpose8x8(l[x % C]);
          bp[y][kPt - 1][x] = transpose8x8(r[x % C]);
        }
      }
    }
    // 4. O^T += V^T . P^T.  Each tile's products of the slot are a chain of their
    // own, added to the running sum in fp32: the tensor cores truncate what they
    // add to, which over a long chain would leave 1e-6 of the result.
    const int vr[4] = {v0, v1, v0 + 1, v1 + 1};
    uint32_t la[kPair], lb[kPair], ha[kPair], hb[kPair], oa[kPair], ob[kPair];  // of rows (v0, v1), (v0 + 1, v1 + 1)
    {
      float te[4];
#pragma unroll
      for (int y = 0; y < kPair; ++y) {
        const uint8_t *vp = base + (2 * y + 1) * S::kPageBytes;
        uint32_t hd[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) hd[x] = *reinterpret_cast<const uint32_t *>(vp + vr[x] * S::kRow + (n >> 1) * 4);
        if (valid < kPair * kPage) {  // rows past the end: 0 * code + 0, whatever the bytes are
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (y * kPage + vr[x] >= valid) hd[x] = 0;
        }
        unpack_steps(__byte_perm(hd[0], hd[1], 0x7632), la[y], ha[y], oa[y]);
        unpack_steps(__byte_perm(hd[2], hd[3], 0x7632), lb[y], hb[y], ob[y]);
        const uint32_t ma = __byte_perm(hd[0], hd[1], 0x5410), mb = __byte_perm(hd[2], hd[3], 0x5410);
#pragma unroll
        for (int x = 0; x < kPt; ++x) {
          if (x + y == 0)
            mma16816_zero(te, ma, kOnes, mb, kOnes, bp[y][x][0], bp[y][x][1]);
          else
            mma16816(te, ma, kOnes, mb, kOnes, bp[y][x][0], bp[y][x][1]);
        }
      }
      add_tile(e, te);
    }
    // codes: D = 128: lane n's channels 16n + i (word 0: rows n of tile i) and 16n + 8 + i (word 1: rows n + 8);
    // D = 64: channels 8n + i and 8n + 4 + i, the halves of one word
    uint32_t w[kPair][4][D / 64];
#pragma unroll
    for (int y = 0; y < kPair; ++y)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint8_t *src = base + (2 * y + 1) * S::kPageBytes + vr[x] * S::kRow + kInt4Header;
        if constexpr (D == 128) {
          const uint2 v = *reinterpret_cast<const uint2 *>(src + n * 8);
          w[y][x][0] = v.x;
          w[y][x][D / 64 - 1] = v.y;
        } else {
          w[y][x][0] = *reinterpret_cast<const uint32_t *>(src + n * 4);
        }
      }
#pragma unroll
    for (int j = 0; j < S::kTiles / 2; ++j) {  // byte j of a word: tiles 2j and 2j + 1
      float t0[4], t1[4];
#pragma unroll
      for (int y = 0; y < kPair; ++y) {
        // byte a of word x of two rows, in the halves of a register
        const uint32_t by0 = 0x4400u + 0x1111u * j, by1 = D == 128 ? by0 : by0 + 0x2222u;
        constexpr int z = D / 64 - 1;
        const uint32_t xa = __byte_perm(w[y][0][0], w[y][1][0], by0), xb = __byte_perm(w[y][2][0], w[y][3][0], by0);
        const uint32_t za = __byte_perm(w[y][0][z], w[y][1][z], by1), zb = __byte_perm(w[y][2][z], w[y][3][z], by1);
        const uint32_t a0 = fma_bf16x2(xa & 0x000f000fu, la[y], oa[y]), a1 = fma_bf16x2(za & 0x000f000fu, la[y], oa[y]);
        const uint32_t a2 = fma_bf16x2(xb & 0x000f000fu, lb[y], ob[y]), a3 = fma_bf16x2(zb & 0x000f000fu, lb[y], ob[y]);
        const uint32_t b0 = fma_bf16x2(xa & 0x00f000f0u, ha[y], oa[y]), b1 = fma_bf16x2(za & 0x00f000f0u, ha[y], oa[y]);
        const uint32_t b2 = fma_bf16x2(xb & 0x00f000f0u, hb[y], ob[y]), b3 = fma_bf16x2(zb & 0x00f000f0u, hb[y], ob[y]);
#pragma unroll
        for (int x = 0; x < kPt; ++x) {
          if (x + y == 0) {
            mma16816_zero(t0, a0, a1, a2, a3, bp[y][x][0], bp[y][x][1]);
            mma16816_zero(t1, b0, b1, b2, b3, bp[y][x][0], bp[y][x][1]);
          } else {
            mma16816(t0, a0, a1, a2, a3, bp[y][x][0], bp[y][x][1]);
            mma16816(t1, b0, b1, b2, b3, bp[y][x][0], bp[y][x][1]);
          }
        }
      }
      add_tile(o[2 * j], t0);
      add_tile(o[2 * j + 1], t1);
    }
    __syncwarp();  // every lane has read the slot
    if (k + kStages < n_my) issue_pair(k + kStages);
  }
  if (k < n_my) {  // a wait ran out: let this warp's copies land (bounded), then leave through the epilogue
    *abort_flag = 1;
    if (lane == 0)
      for (int j = k; j < min(n_my, k + kStages); ++j)
        mbar_wait(&full[warp][j % kStages], (uint32_t)((j / kStages) & 1), abort_flag, p.status, false);
  }

  if constexpr (MODE == kWeights) {
    __syncthreads();  // a warp whose wait ran out has set the flag for the others by now
    return;
  }

  __syncthreads();  // every warp is past its loop: the page slots are free
  float *red = reinterpret_cast<float *>(smem);  // [kWarps][G][D]
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int g = head_of_lane + c;
    if (g >= G) continue;
    float *dst = red + (warp * G + g) * D + n * (D / 8);
#pragma unroll
    for (int i = 0; i < S::kTiles; ++i) {
      dst[i] = fmaf(o[i][c], 0x1p64f, e[c]);
      dst[S::kTiles + i] = fmaf(o[i][C + c], 0x1p64f, e[c]);
    }
    if (n == 0) {
      m_s[warp * G + g] = m[c];
      l_s[warp * G + g] = e[C + c];
    }
  }
  __syncthreads();
  attn_finish<D, kWarps, kThreads, true>(p, u, G, red, m_s, l_s, mg, MODE == kStepWeights ? scores : nullptr);
}

// Cluster size: CTAs that share a unit, a power of two up to 16, so that every
// warp keeps more than a page and a CTA at most 256 (requests of different
// lengths then end together).  Of those the one with the least estimated time:
//   waves * (pages of a CTA + kFixed) * a / rate(a),
// a the CTAs that share an SM (at most what its shared memory, page_smem bytes
// a page with weights, and `fit` allow) and rate(a) = 1 - 2^(-warps / 4) how near
// their warps bring it to its full rate; a last wave that is not full counts
// for three quarters of a full one more.  kFixed is a CTA's start and end in
// pages.
// Measured for 4 warps a CTA (us at 1, 2, 4, 8, 16 CTAs): 4 bits with weights, 4
// heads, 64 units of 8192 rows 97, 54, *39, 48; 256 units of 4096 rows *67, 74, 77,
// 78; 4096 units of 2048 rows *380, 456, 514; 8 heads, 160 units of 3000 rows 85,
// 61, *49, 62; without weights, 4 heads, 64 units of 8192 rows 91, 52, *36, 33; 512
// units of 2048 rows *54, 62, 66; bf16 with weights, 32 units of 16384 rows -, 154,
// 82, *58, 83 (* the rule's).
// A captured launch (np.now below np.most) runs over any length up to np.most, with
// shared memory for that: of the sizes that fit, the one with the least product of
// the estimated times over today's rows and over the longest (so neither is much
// above its best).  Us of a step over 2048 rows in a context of 32768 planned for
// the longest rows alone, so, and called: 4 bits, 512 units 67, 48, 51; 8 heads, 512
// units of up to 2048 rows 84, 51, 47; with weights, 2048 units 369, 224, 189; bf16
// with weights, 1024 units 681, 458, 187, 64 units 44, 29, 21.  The price, over 30000
// rows: 4 bits, 512 units 515, 586, 517; bf16 with weights, 64 units 242, 279, 242.
struct ClusterRule {
  int64_t units;
  int sms, warps, fit;
  size_t base_smem, page_smem;

  size_t smem(int cs, int pages) const { return base_smem + page_smem * ((pages + cs - 1) / cs); }
  // estimated time over `pages` pages a unit with shared memory for `most`
  double cost(int cs, int pages, int most) const {
    constexpr double kFixed = 48;
    constexpr size_t kSm = 228 * 1024, kCta = 1024 + 2304;  // shared memory of an SM; a CTA's beside the dynamic
    const int share = (pages + cs - 1) / cs;
    const int slots = std::max(1, std::min(fit, (int)(kSm / (smem(cs, most) + kCta))));
    const double ctas = (double)units * cs, waves = ctas / ((double)sms * slots);
    const int a = std::min<int64_t>(slots, (units * cs + sms - 1) / sms);
    return (waves <= 1 ? 1 : 0.25 * waves + 0.75 * std::ceil(waves)) * (share + kFixed) * a /
           (1 - std::exp2(-a * warps / 4.0));
  }
  // the size for launches over `pages` pages a unit
  int best(int pages) const {
    int at = 16;
    double least = 1e300;
    for (int cs = 1; cs <= 16 && !too_many(cs, pages); cs *= 2) {
      if (smem(cs, pages) > kMaxSmem || ((pages + cs - 1) / cs > 256 && cs < 16)) continue;
      if (const double c = cost(cs, pages, pages); c < least) least = c, at = cs;
    }
    return at;
  }
  bool too_many(int cs, int pages) const { return cs > 1 && (pages + cs / 2 - 1) / (cs / 2) <= 2 * warps; }
  int operator()(AttnPages np) const {
    const int most = best(np.most);
    if (np.now >= np.most) return most;
    int at = most;
    double least = 1e300;
    for (int cs = 1; cs <= 16 && !too_many(cs, np.most); cs *= 2) {
      if (smem(cs, np.most) > kMaxSmem) continue;
      const double c = cost(cs, np.now, np.most) * cost(cs, np.most, np.most);
      if (c < least) least = c, at = cs;
    }
    return at;
  }
};

// shared memory of the page slots
template <int D, Mode4 MODE, int W>
constexpr size_t kRing4 = 128 + (size_t)W * kStages * kPair * (MODE == kWeights ? 1 : 2) * Shape4<D>::kPageBytes;

template <int D, int GP, Mode4 MODE, int W>
cudaError_t launch4_w(DecodeAttnParams p, int G, AttnPages np, int sms, cudaStream_t s) {
  auto kernel = decode_attention4_kernel<D, GP, MODE, W>;
  p.part_o = p.part_ml = nullptr;
  return launch_attn_cluster(reinterpret_cast<const void *>(kernel), p, G, np, sms, kFit4<GP, MODE, W>,
                             kRing4<D, MODE, W>, MODE == kStepWeights ? (size_t)kPage * G * 4 : 0, 32 * W,
                             MODE != kWeights, s);
}

// A unit split over `splits` CTAs that are no cluster, and a launch that merges them.
template <int D, int GP, int W>
cudaError_t launch4_split(DecodeAttnParams p, int G, int splits, cudaStream_t s) {
  auto kernel = decode_attention4_kernel<D, GP, kStep, W>;
  const int64_t units = (int64_t)p.layer_count * p.R * p.hkv;
  const size_t smem = kRing4<D, kStep, W>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e != cudaSuccess) return e;
  p.nsplit = splits;
  p.part_ml = p.part_o + (size_t)p.layer_count * p.R * p.hq * splits * D;
  kernel<<<(unsigned)(units * splits), 32 * W, smem, s>>>(p, G);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_decode_attention_merge(p, D, true, s);
}

// The step without weights.
//   * With 24 units an SM (one and a half for each of its 16 warp slots, two for
//     each of 12 with 8 query heads), a unit is one warp's: no merge, and the
//     start and end of a unit cost a quarter of what four warps pay (2048 rows,
//     4096 units: 272 us against 290; 1024 units: 109 against 83).  A captured
//     launch keeps the form over longer rows (4096 units of 8192 rows 1038 us,
//     clusters 1069).
//   * A few long requests are split without a cluster: the SMs take at most
//     seven clusters of 16 with a CTA each, so that clusters share SMs while
//     others idle (8 units of 32768 rows: 23 us against 35).
//   * So are units whose CTAs do not all fit at once: a cluster waits until
//     places for all its CTAs are free together, and gives none back before its
//     last CTA is done (512 units of 4096 to 32768 rows, 8 heads: 454 us against
//     539, 4 heads: 338 against 373).  The merge launch costs more than that where
//     they do fit (64 units of 8192 rows: 36 against 33) or are only pairs (512
//     units of 8192 rows: 160 against 155).
//   The partials of a split must fit the workspace (p.max_splits), and no fewer
//   than half the CTAs that the rule asks for will do.
template <int D, int GP>
cudaError_t launch4_step(const DecodeAttnParams &p, int G, AttnPages np, int sms, cudaStream_t s) {
  const int64_t units = (int64_t)p.layer_count * p.R * p.hkv;
  if (units * 2 >= 16LL * sms * 3 && np.now <= 512)
    return launch4_w<D, GP, kStep, 1>(p, G, AttnPages{np.now, np.now}, sms, s);
  const int splits = std::min({p.max_splits, (np.most + 15) / 16, (int)(2LL * sms / units)});
  if (splits > 8 && np.most >= 16 * splits) return launch4_split<D, GP, 8>(p, G, splits, s);
  const int cs = ClusterRule{units, sms, 4, kFit4<GP, kStep, 4>, kRing4<D, kStep, 4>, 0}(np);
  const int parts = std::min(cs, p.max_splits);
  if (parts >= 4 && 2 * parts > cs && units * parts > (int64_t)kFit4<GP, kStep, 4> * sms)
    return launch4_split<D, GP, 4>(p, G, parts, s);
  return launch4_w<D, GP, kStep, 4>(p, G, np, sms, s);
}

// With weights the scores stay in shared memory unless a CTA of the largest
// cluster would have to keep more than 36 KB of them, 20 KB from 128 units on or
// 11 KB from 384 units on (at 8 heads 18432, 10240 and 5632 rows): then too few
// warps fit an SM, and the weights take a launch of their own that reads the
// keys again.  Us in one launch and in two: 512 units, 8 heads, of 4096 to 32768
// rows 979, 645, of 12288 rows 510, 430, of 8192 rows 324, 303; 4 heads, of 24576
// rows 770, 636, of 12288 rows 376, 335, of 8192 rows 216, 231; 2 heads, of 4096 to
// 32768 rows 504, 497.  128 units, 4 heads, of 24576 rows 216, 181, of 16384 rows
// 130, 138.  32 units of 32768 rows, 8 heads 124, 96, 4 heads 68, 74; 8 units 43,
// 44 and 38, 40.
template <int D, int GP>
cudaError_t launch4(const DecodeAttnParams &p, int G, AttnPages np, int sms, cudaStream_t s) {
  if (!p.weights) return launch4_step<D, GP>(p, G, np, sms, s);
  const size_t keep = (size_t)kPage * G * 4 * ((np.most + 15) / 16);
  const int64_t units = (int64_t)p.layer_count * p.R * p.hkv;
  const size_t most = (units >= 384 ? 11 : units >= 128 ? 20 : 36) * 1024;
  if (!p.lse2 || keep <= most) return launch4_w<D, GP, kStepWeights, 4>(p, G, np, sms, s);
  DecodeAttnParams step = p;
  step.weights = nullptr;
  if (cudaError_t e = launch4_step<D, GP>(step, G, np, sms, s)) return e;
  return launch4_w<D, GP, kWeights, 4>(p, G, np, sms, s);
}

// Loads every form that launch4 may choose.
template <int D, int GP>
cudaError_t load4() {
  cudaFuncAttributes a;
  for (const void *kernel : {reinterpret_cast<const void *>(decode_attention4_kernel<D, GP, kStep, 1>),
                             reinterpret_cast<const void *>(decode_attention4_kernel<D, GP, kStep, 4>),
                             reinterpret_cast<const void *>(decode_attention4_kernel<D, GP, kStep, 8>),
                             reinterpret_cast<const void *>(decode_attention4_kernel<D, GP, kStepWeights, 4>),
                             reinterpret_cast<const void *>(decode_attention4_kernel<D, GP, kWeights, 4>)})
    if (cudaError_t e = cudaFuncGetAttributes(&a, kernel)) return e;
  return cudaSuccess;
}

}  // namespace

cudaError_t load_decode_attention4(int head_dim, int G) {
  if (head_dim == 128) return G <= 4 ? load4<128, 4>() : load4<128, 8>();
  return G <= 4 ? load4<64, 4>() : load4<64, 8>();
}

cudaError_t launch_attn_cluster(const void *kernel, DecodeAttnParams &p, int G, AttnPages np, int sms, int fit,
                                size_t base_smem, size_t page_smem, int threads, bool cluster, cudaStream_t s) {
  const int64_t units = (int64_t)p.layer_count * p.R * p.hkv;
  if (units <= 0) return cudaSuccess;
  const ClusterRule rule{units, sms, threads / 32, fit, base_smem, page_smem};
  const int cs = rule(np);
  const size_t smem = rule.smem(cs, np.most);
  if (smem > kMaxSmem) return cudaErrorInvalidConfiguration;
  cudaError_t e;
  // the same limit for every launch: two threads' calls may interleave
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e == cudaSuccess && cs > 8 && cluster)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  p.nsplit = cs;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cs > 1 && cluster ? 1 : 0;
  void *args[] = {&p, &G};
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_decode_attention4(const DecodeAttnParams &p, int head_dim, int G, AttnPages np, int sms,
                                     cudaStream_t s) {
  if (head_dim == 128) return G <= 4 ? launch4<128, 4>(p, G, np, sms, s) : launch4<128, 8>(p, G, np, sms, s);
  return G <= 4 ? launch4<64, 4>(p, G, np, sms, s) : launch4<64, 8>(p, G, np, sms, s);
}

}  // namespace kvc
