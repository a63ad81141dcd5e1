// The int8 form of a row of activations, shared by the kernels that write it:
//   scale = max|v| / 127 (fp32 division; 1 when that is 0)
//   code  = v / scale (fp32 division) rounded to the nearest integer, ties to
//           even, within -127 .. 127
// A row holding an infinity or a NaN gets the scale NaN and codes 0, so that
// everything computed from it is NaN.  Also the 16-byte vectors of activations
// that the row kernels read and their copies into shared memory.
#pragma once

#include <math.h>

#include "tcgen05_common.cuh"

namespace moe {

// 16 bytes of T as fp32 values and back.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4, P = 2;  // values and pairs of values
  // Largest magnitude so far, as bits: a NaN's are above infinity's.
  static __device__ __forceinline__ uint32_t peak(const uint4 &u, uint32_t top) {
    const uint32_t m = 0x7fffffffu;
    return max(max(max(u.x & m, u.y & m), max(u.z & m, u.w & m)), top);
  }
  static __device__ __forceinline__ float peak_value(uint32_t top) { return __uint_as_float(top); }
  static __device__ __forceinline__ float2 pair(const uint4 &u, int p) {
    return p ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w))
             : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
  static __device__ __forceinline__ void set(uint4 &u, int p, float2 f) {
    (p ? u.z : u.x) = __float_as_uint(f.x);
    (p ? u.w : u.y) = __float_as_uint(f.y);
  }
  static __device__ __forceinline__ void get(const uint4 &u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8, P = 4;
  // The same for two values at a time, one in each half.
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162 *>(&w);
  }
  static __device__ __forceinline__ uint32_t peak(const uint4 &u, uint32_t top) {
    const __nv_bfloat162 m =
        __hmax2_nan(__hmax2_nan(__hmax2_nan(__habs2(two(u.x)), __habs2(two(u.y))),
                                __hmax2_nan(__habs2(two(u.z)), __habs2(two(u.w)))),
                    two(top));
    return *reinterpret_cast<const uint32_t *>(&m);
  }
  static __device__ __forceinline__ float peak_value(uint32_t top) {
    return __uint_as_float(max(top << 16, top & 0xffff0000u));
  }
  static __device__ __forceinline__ float2 pair(const uint4 &u, int p) {
    const uint32_t w = p == 0 ? u.x : (p == 1 ? u.y : (p == 2 ? u.z : u.w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void set(uint4 &u, int p, float2 f) {
    const __nv_bfloat162 b = __float22bfloat162_rn(f);
    (p == 0 ? u.x : (p == 1 ? u.y : (p == 2 ? u.z : u.w))) =
        *reinterpret_cast<const uint32_t *>(&b);
  }
  static __device__ __forceinline__ void get(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// cp.async: 16 bytes from global into shared memory, in groups.
__device__ __forceinline__ void copy16(uint32_t smem, const void *gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Wait until at most n (0, 1 or 2) of this thread's copy groups are still in
// flight.
__device__ __forceinline__ void copy_wait(int n) {
  switch (n) {
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
  }
}
namespace i8 {

struct RowScale {
  float scale;    // what is stored
  float divisor;  // what the values are divided by
  float inv;      // 1 / divisor, or 0: divide every value
  bool fine;
};

// From the row's largest magnitude (infinity or NaN when any value is not finite).
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

// The integer nearest to fl(v / s) for a quotient next to the middle h between
// two integers, without the division.  v - h s is exact in one fused multiply-
// add (a multiple of half the last bit of s, under 2^12 of them); fl(v / s) is
// h itself when |v / s - h| is at most half a unit in h's last place, 2^(e-24)
// for h in [2^e, 2^(e+1)) (h's last bit is 0, so the bound belongs to h).
__device__ __forceinline__ float beside_middle(float v, float s, float h) {
  const float r = fmaf(-h, s, v);
  const float unit = __uint_as_float(__float_as_uint(h) & 0x7f800000u);  // 2^e
  if (fabsf(r) <= s * (unit * 0x1p-24f)) return rintf(h);  // to even
  return r > 0.0f ? h + 0.5f : h - 0.5f;
}

// The codes of N (4 or 8) values, four to a word.  384 + v * inv lies in [256,
// 512), so its bits count steps of 2^-15: doubled, with 128 and a half and kNear
// added, they hold the rounded integer in byte 2 and, in the low half, how far
// above the middle between two integers the quotient lies.  v * inv + 384 is within
// 4e-5 of the quotient (three roundings), kNear is 8 * 2^-16 = 1.2e-4, so a low
// half above 2 kNear says that the integer is the quotient's; the others are
// decided by beside_middle.  (Of bf16 values one in some hundreds is half the
// row's largest, 63.5 steps: with them about a third of a warp's vectors have a
// value to decide.  Out of line that cost more than it saved, 172 us against 145
// for 131072 x 2048, and so did rows in registers, whose unrolled code leaves the
// instruction cache, 170.)
template <int N>
__device__ __forceinline__ void codes(const float (&f)[N], const RowScale &r,
                                      uint32_t (&c)[N / 4]) {
  constexpr uint32_t kNear = 8;
  constexpr float kBase = 384.0f;
  uint32_t b[N], low = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 w = __ffma2_rn(make_float2(f[i], f[i + 1]), make_float2(r.inv, r.inv),
                                make_float2(kBase, kBase));
    b[i] = 2u * __float_as_uint(w.x) + (0x808000u + kNear);
    b[i + 1] = 2u * __float_as_uint(w.y) + (0x808000u + kNear);
  }
#pragma unroll
  for (int i = 0; i < N; i += 2) low = __vminu2(low, __byte_perm(b[i], b[i + 1], 0x5410));
  if (min(low & 0xffffu, low >> 16) <= 2 * kNear) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if ((b[i] & 0xffffu) <= 2 * kNear) {
        // the middle that the quotient is next to: the integer behind it less a half
        const float h = (float)(int8_t)(b[i] >> 16) - 0.5f;
        b[i] = (uint32_t)(int)beside_middle(f[i], r.divisor, h) << 16;
      }
    }
  }
  if (r.inv == 0.0f) {  // a row without a usable reciprocal: divide
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = (uint32_t)code(f[i], r) << 16;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    c[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0062),
                       __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0062), 0x5410);
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
