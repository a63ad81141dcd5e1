// The int8 form of a row of activations, shared by the kernels that write it:
//   scale = max|v| / 127 (fp32 division; 1 when that is 0)
//   code  = v / scale (fp32 division) rounded to the nearest integer, ties to
//           even, within -127 .. 127
// A row holding an infinity or a NaN gets the scale NaN and codes 0, so that
// everything computed from it is NaN.  Also the 16-byte vectors of activations
// that these kernels read.
#pragma once

#include <math.h>

#include "tcgen05_common.cuh"

namespace moe {

// 16 bytes of T as fp32 values and back.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4 &u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

namespace i8 {

struct RowScale {
  float scale;    // what is stored
  float divisor;  // what the values are divided by
  float inv;      // 1 / divisor, or 0: divide every value
  bool fine;
};

// |v|, a NaN as infinity.
__device__ __forceinline__ float magnitude(float v) {
  const float m = fabsf(v);
  return m < INFINITY ? m : INFINITY;
}

// From the row's largest magnitude (INFINITY when any value is not finite).
__device__ __forceinline__ RowScale row_scale(float top) {
  RowScale r;
  r.fine = top < INFINITY;
  const float q = __fdiv_rn(top, 127.0f);
  r.divisor = (r.fine && q != 0.0f) ? q : 1.0f;
  r.scale = r.fine ? r.divisor : __int_as_float(0x7fc00000);
  r.inv = (r.fine && r.divisor > 1e-30f) ? __fdiv_rn(1.0f, r.divisor) : 0.0f;
  return r;
}

__device__ __forceinline__ int code(float v, const RowScale &r) {
  const float q = rintf(__fdiv_rn(v, r.divisor));
  // the clamp matters for subnormal scales, whose few bits let |q| pass 127
  return r.fine ? (int)fminf(fmaxf(q, -127.0f), 127.0f) : 0;
}

// The codes of N (4 or 8) values, four to a word.  A value's quotient is
// within 2e-5 of v * inv (two roundings of at most 2^-24 of 127, and that of
// the quotient itself), so where v * inv is further than 1e-4 from the middle
// between two integers its nearest integer is the quotient's, and only the few
// values in between are divided.  Adding 1.5 * 2^23 rounds to the nearest
// integer and leaves it in the low bits of the sum, two's complement.
template <int N>
__device__ __forceinline__ void codes(const float (&f)[N], const RowScale &r,
                                      uint32_t (&c)[N / 4]) {
  constexpr float kMagic = 12582912.0f;
  uint32_t b[N];
  float worst = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = fmaf(f[i], r.inv, kMagic);
    worst = fmaxf(worst, fabsf(fmaf(f[i], r.inv, kMagic - t)));
    b[i] = __float_as_uint(t);
  }
  if (r.inv == 0.0f || worst > 0.4999f) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = (uint32_t)code(f[i], r);
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    c[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                       __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
}

template <int N>
__device__ __forceinline__ void store(int8_t *to, const uint32_t (&c)[N / 4]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint2 *>(to) = make_uint2(c[0], c[1]);
  else
    *reinterpret_cast<uint32_t *>(to) = c[0];
}

}  // namespace i8
}  // namespace moe
