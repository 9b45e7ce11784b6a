// The quantised paged KV cache: where the bytes of one (page, head) lie, and
// the arithmetic of a row's parameters.
//
// A token row x[0..D) of a head is held as whole numbers n_d of `bits` bits
// and two bf16 parameters, and stands for s n_d + z:
//   z = min x rounded down to bf16,  s = bf16(float32((max x - z) / (2^bits - 1)))
//   n_d = (x_d - z) / s rounded to the nearest, ties to even (float64 quotient)
// One scale per token and head (not per page and channel) lets a row be
// written the moment it exists: no other row of the page changes. z is
// rounded down so that no n_d is negative; n_d above 2^bits - 1 (s rounded
// down) is clamped, which moves it by at most 2^-8 of the row's range.
//
// One (page, head) is one contiguous run of bytes, so that one bulk copy
// fetches it:
//   K numbers  [D*bits/128][P][16 B]  channel pieces of 16 bytes, token by token
//   K (s, z)   [P][2] bf16
//   V numbers  [P*bits/8/u][D][u B]   u = min(16, P*bits/8): token pieces, channel by channel
//   V (s, z)   [P][2] bf16
// The keys lie token-major and the values channel-major: attention's two
// contractions run over channels (q k) and over tokens (p v), and each of its
// threads unpacks one row of its operand from 16-byte pieces that neighbouring
// threads read from neighbouring addresses.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "s3r.h"

namespace s3r {

constexpr float kKvqTiny = 7.888609052210118e-31f;   // 2^-100: rows of a smaller step are held flat (s = 1, n = 0)

struct KvqLayout {
  int half;      // bytes of one side's numbers, P * D * bits / 8
  int unit;      // bytes of one V piece
  int ut;        // tokens of one V piece
  int off_kp, off_v, off_vp, page_bytes;
};
__host__ __device__ constexpr KvqLayout kvq_layout(int D, int P, int bits) {
  KvqLayout l{};
  l.half = P * D * bits / 8;
  l.unit = P * bits / 8 < 16 ? P * bits / 8 : 16;
  l.ut = l.unit * 8 / bits;
  l.off_kp = l.half;
  l.off_v = l.half + 4 * P;
  l.off_vp = 2 * l.half + 4 * P;
  l.page_bytes = 2 * l.half + 8 * P;
  return l;
}

struct KvqRow {
  float z, s;   // parameters (bf16 values)
  float inv;    // 1 / s; 0: every n is 0
  bool wide;    // z is so much smaller than the largest value that x - z may lose its low bits in float32
};

// Two values by one instruction: a b + c.
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// min and max that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Parameters of a row with minimum mn and maximum mx (either NaN if the row
// holds one). The float32 quotient is off by at most 2^-23 of itself, so it
// decides the bf16 rounding unless it lies within a few steps of a midpoint;
// there, and where max - z overflows, the float64 quotient is taken.
template <int BITS>
__device__ __forceinline__ KvqRow kvq_row(float mn, float mx) {
  constexpr int kTop = (1 << BITS) - 1;
  KvqRow r;
  r.s = 1.f;
  r.inv = 0.f;
  r.wide = false;
  if (!(mn > -INFINITY && mx < INFINITY)) {            // NaN or infinity in the row
    r.z = __int_as_float(0x7fc00000);
    return r;
  }
  r.z = __bfloat162float(__float2bfloat16_rd(mn));
  const float range = mx - r.z;
  float q = __fdiv_rn(range, (float)kTop);
  const uint32_t low = __float_as_uint(q) & 0xffffu;
  if (!(range < INFINITY) || (low > 0x7ff8u && low < 0x8008u)) q = (float)(((double)mx - (double)r.z) / kTop);
  const float s = __bfloat162float(__float2bfloat16_rn(q));
  if (s < kKvqTiny) return r;
  r.s = s;
  r.inv = __frcp_rn(s);
  r.wide = fabsf(r.z) < 0x1p-15f * mx && r.z != 0.f;
  return r;
}

// n of x, from float64: (x - z) / s rounded to the nearest, ties to even.
template <int BITS>
__device__ __forceinline__ uint32_t kvq_number_exact(float x, float z, float s) {
  constexpr int kTop = (1 << BITS) - 1;
  const int n = __double2int_rn(((double)x - (double)z) / (double)s);
  return (uint32_t)(n < kTop ? n : kTop);
}

}  // namespace s3r
