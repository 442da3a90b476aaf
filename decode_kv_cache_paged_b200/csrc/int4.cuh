// int4.cuh -- the 4-bit cache row (KVC_INT4): its layout, how a row is coded
// and the value a code stands for.
//
// A row of D channels (64 or 128) is four groups of D/4 channels.  For each
// group, with lo and hi its smallest and largest value,
//     s     = (hi - lo) / 15 rounded up to four significant bits
//             (0 where (hi - lo) / 15 < 2^-56),
//     code  = rint((x - lo) / s) in [0, 15]   (ties to even; 0 where s = 0),
//     value = lo + s * code,
// so a value is off by at most s / 2.  A group that holds an infinity or a
// NaN, or whose (hi - lo) / 15 reaches 2^56, stands for NaN throughout.
// Differences and quotients are rounded to fp32.
//
// Bytes of a row: for each group, group 0 first, a 4-byte word, then D/2
// bytes of codes: 80 bytes at D = 128, 48 at D = 64.  The row is one
// contiguous block, so the rounds move it like any other row.
//   * A group's word holds s in its high half and mid in its low half, as
//     bf16.  The four lowest bits of s, which s does not use, hold z:
//     value = mid + s * (code - z).  In a K row z = 0 and mid = lo.  In a V
//     row z = min(15, rint(-lo / s)) where 0 < -lo / 2^e < 32 (2^e the power
//     of two at or below s), else 0, and mid = lo + z * s.  A broken group
//     has s = z = 0 and a NaN for mid.
//   * The codes of a V row follow in channel order, two to a byte with the
//     lower channel in the low half.  Those of a K row come in units of D/16
//     channels: unit t of group g (the channels from g * D/4 + t * D/16 on,
//     packed as above) is unit 4 t + g of the row.
//
// Why so: s is rounded up (never down) so that 15 steps reach hi without
// clipping, and to four significant bits so that s * (code - z) has at most
// eight and is exact in bf16: what the tensor cores read of V carries no
// rounding.  The wider step costs 4.6 % of the quantisation error on average.
// z centres the codes of V: sums of s * (code - z) over rows are of the size
// of the result, where sums of s * code are up to a hundred times larger and
// cancel against those of lo (measured at 32768 rows: an output error of 6e-5
// without, below 1e-6 with it).  mid is exact: where z > 0 it is a multiple of
// lo's last place (which is at most s's) and no larger than max(|lo|, s / 2).
// A K row's sums over channels are short, and its codes enter the products
// without s, as fp16 numbers, so there z would only cost; their order puts
// what one lane of those products reads side by side.  The limits of s keep
// s * 2^64 and s / 2^64 within bf16's normal numbers (decode_attention4.cu).
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace kvc {

constexpr int kInt4Groups = 4;
constexpr int kInt4Header = 16;  // bytes of the groups' words before the codes
__host__ __device__ constexpr int int4_row_bytes(int d) { return d / 2 + kInt4Header; }

// a / b from b's correctly rounded reciprocal: a product and one correction by
// the remainder (Markstein, IBM J. Res. Dev. 34(1), 1990).  That is the correctly
// rounded quotient where the product is within one unit in the last place, which
// not every pair's is, but for the divisors here, of at most four significant
// bits (a step, or 15), it is so for every a: all 8 * 2^23 pairs of mantissas
// agree with the division.  Overflow and underflow are harmless: a quotient that
// overflows is refused or NaN, one that underflows rounds to code 0 like the
// exact one.
__device__ __forceinline__ float quotient(float a, float b, float inv) {
  const float q = a * inv;
  return fmaf(fmaf(-q, b, a), inv, q);
}

// step of a group from its smallest and largest value
__device__ __forceinline__ float int4_step(float lo, float hi) {
  const float r = quotient(hi - lo, 15.f, 1.f / 15.f);
  if (!(r < 0x1p56f)) return __int_as_float(0x7fffffff);  // NaN: infinities, NaN, a range too wide
  if (r < 0x1p-56f) return 0.f;
  return __uint_as_float((__float_as_uint(r) + 0xFFFFFu) & ~0xFFFFFu);
}

// a group's word from its step, the step's reciprocal and its lowest value (the
// step NaN for a broken group)
template <bool IS_V>
__device__ __forceinline__ uint32_t int4_word(float s, float inv, float lo) {
  if (isnan(s)) return 0x7fffu;
  float z = 0.f;
  if (IS_V && s > 0.f) {
    const uint32_t e = __float_as_uint(s) & 0x7f800000u;      // 2^e
    const float x = -lo * __uint_as_float(0x7f000000u - e);  // -lo / 2^e
    if (x > 0.f && x < 32.f) z = fminf(rintf(quotient(-lo, s, inv)), 15.f);
  }
  const float mid = fmaf(z, s, lo);
  return (__float_as_uint(s) & 0xfff00000u) | (uint32_t)z << 16 | __float_as_uint(mid) >> 16;
}

// a small integer as a float: 2^23 + n has n in its lowest bits
__device__ __forceinline__ float small_float(uint32_t n) { return __uint_as_float(0x4b000000u | n) - 0x1p23f; }

// what a group's word says: s, z * s (exact) and mid
__device__ __forceinline__ void int4_unword(uint32_t h, float &s, float &zs, float &mid) {
  s = __uint_as_float(h & 0xfff00000u);
  zs = small_float(h >> 16 & 15u) * s;
  mid = __uint_as_float(h << 16);
}

// 32-bit word of a K row's codes that holds the natural word v (8 channels
// from 8 v on) at D = 128; at D = 64 the two halves of word v are units 2 v
// and 2 v + 1, 16 bits each
__device__ __forceinline__ int int4_k_word(int v) { return (v & 3) * 4 + (v >> 2); }
__device__ __forceinline__ int int4_k_half(int h) { return (h & 3) * 4 + (h >> 2); }

}  // namespace kvc
