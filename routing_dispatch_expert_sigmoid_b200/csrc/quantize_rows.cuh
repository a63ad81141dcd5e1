// The int8 form of a row of activations, shared by the kernels that write it:
//   scale = max|v| / 127 (fp32 division; 1 when that is 0)
//   code  = v / scale (fp32 division) rounded to the nearest integer, ties to
//           even, within -127 .. 127
// A row holding an infinity or a NaN gets the scale NaN and codes 0, so that
// everything computed from it is NaN.
#pragma once

#include <math.h>

#include "tcgen05_common.cuh"

namespace moe {
namespace i8 {

struct RowScale {
  float scale;    // what is stored
  float divisor;  // what the values are divided by (1 for a non-finite row)
  bool fine;
};

// From the row's largest magnitude (INFINITY when any value is not finite).
__device__ __forceinline__ RowScale row_scale(float top) {
  RowScale r;
  r.fine = top < INFINITY;
  const float q = __fdiv_rn(top, 127.0f);
  r.scale = r.fine ? (q == 0.0f ? 1.0f : q) : __int_as_float(0x7fc00000);
  r.divisor = r.fine ? r.scale : 1.0f;
  return r;
}

__device__ __forceinline__ int code(float v, const RowScale &r) {
  const float q = rintf(__fdiv_rn(v, r.divisor));
  // the clamp matters for subnormal scales, whose few bits let |q| pass 127
  return r.fine ? (int)fminf(fmaxf(q, -127.0f), 127.0f) : 0;
}

// N (4 or 8) consecutive codes with one store.
template <int N>
__device__ __forceinline__ void store_codes(int8_t *to, const float (&f)[N], const RowScale &r) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) w[i] |= (uint32_t)(code(f[4 * i + q], r) & 0xff) << (8 * q);
  }
  if (N == 8)
    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[N / 4 - 1]);
  else
    *reinterpret_cast<uint32_t *>(to) = w[0];
}

}  // namespace i8
}  // namespace moe
