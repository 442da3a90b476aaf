// int4.cuh -- the 4-bit cache row (KVC_INT4): its layout, how a row is coded
// and the value a code stands for.
//
// A row of D channels (64 or 128) is four groups of D/4 channels.  For each
// group, with lo and hi its smallest and largest value,
//     s     = (hi - lo) / 15 rounded up to four significant bits
//             (0 where (hi - lo) / 15 < 2^-100),
//     code  = rint((x - lo) / s) in [0, 15]   (ties to even; 0 where s = 0),
//     value = lo + s * code,
// so a value is off by at most s / 2.  A group that holds an infinity or a
// NaN, or whose (hi - lo) / 15 reaches 2^100, stands for NaN throughout.
//
// Bytes of a row: 16 bytes of (s, lo) bf16 pairs, group 0 first, then D/2
// bytes of codes, two to a byte with the lower channel in the low half: 80
// bytes at D = 128, 48 at D = 64.  The row is one contiguous block, so the
// rounds move it like any other row.
//
// lo is one of the row's bf16 values, so it is stored exactly.  s is rounded
// up (never down) so that 15 steps reach hi without clipping, and to four
// significant bits so that s * code has at most eight and is exact in bf16:
// the tensor-core operands of the attention over the cache carry no rounding.
// The wider step costs 4.6 % of the quantisation error on average.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace kvc {

constexpr int kInt4Groups = 4;
constexpr int kInt4Header = 16;  // bytes of (s, lo) pairs before the codes
__host__ __device__ constexpr int int4_row_bytes(int d) { return d / 2 + kInt4Header; }

// step of a group from its smallest and largest value
__device__ __forceinline__ float int4_step(float lo, float hi) {
  const float r = __fdiv_rn(hi - lo, 15.f);
  if (!(r < 0x1p100f)) return __int_as_float(0x7fffffff);  // NaN: infinities, NaN, a range too wide
  if (r < 0x1p-100f) return 0.f;
  return __uint_as_float((__float_as_uint(r) + 0xFFFFFu) & ~0xFFFFFu);
}

}  // namespace kvc
