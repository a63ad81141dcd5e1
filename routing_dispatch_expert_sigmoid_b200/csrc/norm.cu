// The norms around a block (moe_norm, moe_norm_backward).
//
// Forward, per token, with rms(v) = v / sqrt(mean(v^2) + eps):
//   z = residual_scale * x + gate * (w_post * rms(y))    (z = x without y)
//   h = w_pre * rms(z)          of z as it is stored, in the storage type
//   codes and one scale of h    of h as it is stored (moe_quantize_rows_int8)
// Backward, from dz (what arrives at z) and dh (what arrives at h), with
// v = z * rstd_pre, u = y * rstd_post, c = gate * w_post:
//   g  = dz + rstd_pre * (dh w_pre - v * mean(dh w_pre v))      dw_pre += dh v
//   dx = residual_scale * g        dgate += g u w_post          dw_post += g gate u
//   dy = rstd_post * (g c - u * mean(g c u))
// The second mean expands into sums that need no g:
//   sum(g c u) = sum(c u (dz + rstd_pre dh w_pre)) - rstd_pre m sum(c u v),
//   m = mean(dh w_pre v),
// so a row takes one block reduction of three sums instead of two in turn.
//
// Bound: HBM.  Forward reads x and y and writes z and h once; backward reads
// dz, dh, z, y and writes dx, dy once.  A CTA walks a contiguous range of rows.
// Every thread owns the same 16-byte vectors of each row, so a ring of the next
// rows in shared memory needs no barrier: a thread copies its vectors there
// with cp.async and is the only one to read them.  That keeps several rows per
// CTA in flight while the row at hand waits in its reductions, and the weight
// vectors and the gradients' sums stay in registers over the whole range.
//
// Sums over tokens (dw_post, dw_pre, dgate) are fp32, taken per CTA in row
// order, written as partial sums and added in CTA order by a second kernel:
// the result does not depend on timing.  A gate row whose tokens lie in one
// CTA's range is written directly; one that crosses ranges leaves a partial sum
// in each (slot 0 for the range's first rows, slot 1 for its last).
//
// bf16, gate and both norms: forward 8192 x 7168 82 us (5.7 TB/s), backward
// 16381 x 4096 147 us (5.5 TB/s); a copy reaches 6.45.  16 x 4096 takes 3 us.
// With codes (hq), a third block reduction and the instructions of the codes:
// 8192 x 7168 95 us for 87 in the same run (the row quantiser alone takes 36),
// 16384 x 4096 123 for 92 (41), 131072 x 2048 497 for 356 (142): short rows gain
// little over two launches.
#include <algorithm>

#include "quantize_rows.cuh"

namespace moe {
namespace {

constexpr int kMaxStages = 3;
constexpr size_t kRingLimit = 220u << 10;  // shared memory for weights and rings of one SM
constexpr int kNormSms = 148;
// threads of a row, at most: two CTAs of 448 leave 72 registers a thread
constexpr int row_threads(int vpt) { return vpt == 2 ? 448 : 512; }

__device__ __forceinline__ uint4 lds16(uint32_t smem) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem)
               : "memory");
  return v;
}

// Sums over the block, in a fixed order and the same in every thread.  `red`:
// one of two buffers that consecutive calls take in turn (a thread that writes
// a buffer again has passed the barrier of the call between, which every
// thread reaches only after reading it); entries of warps that there are not
// stay 0.
constexpr int kMaxWarps = 16;
struct Red {
  float v[3][kMaxWarps];
};
__device__ __forceinline__ float warp_sum16(float v) {  // over each half of the warp
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float block_sum(float v, Red &red) {
  const int lane = threadIdx.x % 32;
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  v = warp_sum16(v);
  if (lane == 0) red.v[0][threadIdx.x / 32] = v;
  __syncthreads();
  return warp_sum16(red.v[0][lane % kMaxWarps]);
}
// Three sums.  Inside the warp each exchange step halves the values a lane
// carries, so that three sums cost six shuffles instead of fifteen: lanes 0-7
// end with the first, 8-15 with the second, 16-23 with the third.
__device__ __forceinline__ void block_sum3(float &v0, float &v1, float &v2, Red &red) {
  const int lane = threadIdx.x % 32;
  const bool hi = lane & 16, mid = lane & 8;
  const float a = (hi ? v2 : v0) + __shfl_xor_sync(0xffffffffu, hi ? v0 : v2, 16);
  const float b = (hi ? 0.f : v1) + __shfl_xor_sync(0xffffffffu, hi ? v1 : 0.f, 16);
  float c = (mid ? b : a) + __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
  if (lane % 8 == 0 && lane < 24) red.v[lane / 8][threadIdx.x / 32] = c;
  __syncthreads();
  const float r01 = warp_sum16(red.v[lane / 16][lane % kMaxWarps]);
  v2 = warp_sum16(red.v[2][lane % kMaxWarps]);
  v0 = __shfl_sync(0xffffffffu, r01, 0);
  v1 = __shfl_sync(0xffffffffu, r01, 16);
}
// Largest of values >= 0 (or NaN, which is above them: the order of the bits).
__device__ __forceinline__ float block_max(float v, Red &red) {
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v));
  if (threadIdx.x % 32 == 0) red.v[0][threadIdx.x / 32] = __uint_as_float(m);
  __syncthreads();
  return __uint_as_float(
      __reduce_max_sync(0xffffffffu, __float_as_uint(red.v[0][threadIdx.x % kMaxWarps])));
}
__device__ __forceinline__ void clear(Red (&red)[2]) {
  for (int i = threadIdx.x; i < 2 * 3 * kMaxWarps; i += blockDim.x)
    (&red[0].v[0][0])[i] = 0.f;
  __syncthreads();
}

// Two fp32 values at a time: one instruction for both.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ void sts16(uint32_t smem, const uint4 &v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(smem), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
// A weight row: this thread's vectors of it, or ones, wait in its places in
// shared memory.  There they cost a load per use instead of registers, which
// the rows in hand and the sums need (spilled to local memory, they were the
// longest stall of the first versions).  Rows of more than 14 KB (gradient: 16
// KB; VPT 4) leave no room for them and read the weights through L1 instead.
template <typename T, int VPT>
struct Weights {
  static constexpr bool kKept = VPT < 4;
  const uint4 *w;
  uint32_t smem, step;
  __device__ __forceinline__ uint4 global(int i) const {
    uint4 u;
#pragma unroll
    for (int p = 0; p < Vec<T>::P; ++p) Vec<T>::set(u, p, both(1.f));
    return w ? __ldg(w + i * blockDim.x + threadIdx.x) : u;
  }
  __device__ __forceinline__ void keep(uint32_t at, const void *row, uint32_t st, int live) {
    w = static_cast<const uint4 *>(row);
    smem = at;
    step = st;
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i * (int)blockDim.x < live) sts16(smem + i * step, global(i));
    }
  }
  __device__ __forceinline__ uint4 get(int i) const {
    if constexpr (kKept) return lds16(smem + i * step);
    return global(i);
  }
};

// A gate of few tokens a row travels with the rows in the ring; else its row is
// kept like a weight row and loaded anew where the next one begins.  In the ring
// it costs a quarter of the copies and of the room: gradient, 16381 x 4096, rows
// of 2048 tokens 162 us against 147; forward, 8192 x 7168, rows of 10 tokens 103
// against 87, of 6 103 against 91, but 14333 x 4096 97.5 against 103.  Weights
// that are not kept are read through L1, rows of 20 tokens 109 us in the ring and
// not (4775 x 12288), of 2048 109 and 100, gradient 282 and 294, 198 and 203.
__host__ __device__ __forceinline__ bool gate_in_ring(const void *gate, int span, int rows,
                                                      bool kept) {
  return gate && span < rows && span < (kept ? 8 : 64);
}

__device__ __forceinline__ const void *gate_row(const void *gate, int g, int nvec) {
  return gate ? static_cast<const uint4 *>(gate) + (size_t)g * nvec : nullptr;
}

// First row of CTA b of n over T rows.
__host__ __device__ __forceinline__ int first_row(int b, int n, int T) {
  return (int)((long long)b * T / n);
}

struct NormArgs {
  const void *x, *y, *w_post, *gate, *w_pre;
  void *z, *h;
  int8_t *hq;
  float *h_scale, *rstd_post, *rstd_pre;
  int T, d, span, stages, post_norm;
  float alpha, eps_post, eps_pre;
};

// The rows of a CTA's range as its ring sees them: where a thread's next copies
// come from and go to, and the slot that is read next.  Everything advances by
// additions.
struct Ring {
  uint32_t base, end, put, get;  // shared memory, this thread's first vector
  uint32_t stage;                // bytes of a slot
  __device__ __forceinline__ void start(uint32_t smem, int stages, uint32_t stage_bytes) {
    base = put = get = smem;
    stage = stage_bytes;
    end = smem + stages * stage_bytes;
  }
  __device__ __forceinline__ uint32_t next(uint32_t at) const {
    at += stage;
    return at == end ? base : at;
  }
};

template <typename T, int VPT, bool POST, bool PRE>
__global__ void __launch_bounds__(row_threads(VPT), VPT == 4 ? 1 : 2) k_norm(const NormArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using V = Vec<T>;
  constexpr int N = V::N, PN = V::P;
  extern __shared__ uint4 s_ring[];  // weights, then [stages][tensors][VPT * blockDim.x]
  __shared__ Red s_red[2];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = a.d / N;
  const bool gate_rows = POST && gate_in_ring(a.gate, a.span, a.T, Weights<T, VPT>::kKept);
  const int tensors = 1 + POST + gate_rows;
  const uint32_t step = nt * 16, tensor = VPT * step;  // bytes
  const int live = nvec - tid;  // vector i of this thread exists when i * nt < live
  clear(s_red);

  const uint32_t mine = tc::smem_addr(s_ring) + tid * 16;
  Weights<T, VPT> wpost, gate, wpre;
  if constexpr (POST) {
    wpost.keep(mine, a.w_post, step, live);
  }
  if constexpr (PRE) wpre.keep(mine + (POST ? 2 * tensor : 0), a.w_pre, step, live);
  const uint32_t kept = Weights<T, VPT>::kKept ? (2 * POST + PRE) * tensor : 0;
  const int r0 = first_row(blockIdx.x, gridDim.x, a.T);
  const int r1 = first_row(blockIdx.x + 1, gridDim.x, a.T);
  const float inv_d = 1.0f / (float)a.d;
  int red = 0;

  Ring ring;
  ring.start(mine + kept, a.stages, tensors * tensor);
  size_t in = (size_t)r0 * nvec + tid, out = in;  // vectors: next row to copy, to write
  const uint4 *pg = nullptr;
  int to_copy = r1 - r0, gate_left = 0;
  if (gate_rows) {
    pg = static_cast<const uint4 *>(a.gate) + (size_t)(r0 / a.span) * nvec + tid;
    gate_left = a.span - r0 % a.span;
  }
  auto issue = [&]() {  // this thread's vectors of the next row into the ring
    if (to_copy > 0) {
      --to_copy;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          copy16(ring.put + i * step, static_cast<const uint4 *>(a.x) + in + i * nt);
          if constexpr (POST) {
            copy16(ring.put + tensor + i * step, static_cast<const uint4 *>(a.y) + in + i * nt);
            if (gate_rows) copy16(ring.put + 2 * tensor + i * step, pg + i * nt);
          }
        }
      }
      in += nvec;
      if constexpr (POST) {
        if (gate_rows && --gate_left == 0) {
          pg += nvec;
          gate_left = a.span;
        }
      }
      ring.put = ring.next(ring.put);
    }
    copy_commit();
  };
  for (int s = 0; s < a.stages - 1; ++s) issue();

  int next_gate = r0;  // the row from which the kept gate is another one
  for (int r = r0; r < r1; ++r) {
    issue();
    if (POST && !gate_rows && r == next_gate) {
      const int g = a.gate ? r / a.span : 0;
      gate.keep(mine + tensor, gate_row(a.gate, g, nvec), step, live);
      next_gate = a.gate ? r + min(a.T - r, a.span - (r - g * a.span)) : a.T;
    }
    copy_wait(a.stages - 1);
    const uint32_t st = ring.get;
    ring.get = ring.next(st);
    uint4 z[VPT];
    float2 sq = both(0.f);
    if constexpr (POST) {
      float rs = 1.f;
      if (a.post_norm) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          if (i * nt < live) {
            const uint4 y = lds16(st + tensor + i * step);
#pragma unroll
            for (int q = 0; q < PN; ++q) {
              const float2 f = V::pair(y, q);
              sq = fma2(f, f, sq);
            }
          }
        }
        rs = rsqrtf(fmaf(block_sum(sq.x + sq.y, s_red[red ^= 1]), inv_d, a.eps_post));
        if (tid == 0 && a.rstd_post) a.rstd_post[r] = rs;
      }
      sq = both(0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          const uint4 x = lds16(st + i * step), y = lds16(st + tensor + i * step);
          const uint4 w = wpost.get(i);
          const uint4 gt = gate_rows ? lds16(st + 2 * tensor + i * step) : gate.get(i);
#pragma unroll
          for (int q = 0; q < PN; ++q) {
            float2 f = mul2(mul2(V::pair(y, q), both(rs)), V::pair(w, q));
            f = mul2(f, V::pair(gt, q));
            V::set(z[i], q, fma2(both(a.alpha), V::pair(x, q), f));
            if constexpr (PRE) {
              f = V::pair(z[i], q);  // z as stored
              sq = fma2(f, f, sq);
            }
          }
          static_cast<uint4 *>(a.z)[out + i * nt] = z[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          z[i] = lds16(st + i * step);
#pragma unroll
          for (int q = 0; q < PN; ++q) {
            const float2 f = V::pair(z[i], q);
            sq = fma2(f, f, sq);
          }
        }
      }
    }
    if constexpr (PRE) {
      const float rs = rsqrtf(fmaf(block_sum(sq.x + sq.y, s_red[red ^= 1]), inv_d, a.eps_pre));
      if (tid == 0 && a.rstd_pre) a.rstd_pre[r] = rs;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          const uint4 w = wpre.get(i);
#pragma unroll
          for (int q = 0; q < PN; ++q)  // z holds h from here on
            V::set(z[i], q, mul2(mul2(V::pair(z[i], q), both(rs)), V::pair(w, q)));
          if (a.h) static_cast<uint4 *>(a.h)[out + i * nt] = z[i];
        }
      }
      if (a.hq) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (i * nt < live) top = V::peak(z[i], top);
        const i8::RowScale q8 = i8::row_scale(block_max(V::peak_value(top), s_red[red ^= 1]));
        if (tid == 0) a.h_scale[r] = q8.scale;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          if (i * nt < live) {
            float f[N];
            V::get(z[i], f);
            uint32_t c[N / 4];
            i8::codes<N>(f, q8, c);
            i8::store<N>(a.hq + (out + i * nt) * N, c);
          }
        }
      }
    }
    out += nvec;
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
struct NormGradArgs {
  const void *dz, *dh, *z, *y, *w_post, *gate, *w_pre;
  const float *rstd_post, *rstd_pre;
  void *dx, *dy;
  float *dgate;        // complete gate rows are written here by the row kernel
  float *part_post;    // [CTAs][d] partial sums, or nullptr: not wanted
  float *part_pre;
  float *part_gate;    // [CTAs][2][d]
  int T, d, span, stages, post_norm;
  float alpha;
};

template <int PN>
__device__ __forceinline__ void store_sums(float *to, const float2 (&f)[PN]) {
#pragma unroll
  for (int q = 0; q < PN; q += 2)
    *reinterpret_cast<float4 *>(to + 2 * q) = make_float4(f[q].x, f[q].y, f[q + 1].x, f[q + 1].y);
}

template <typename T, int VPT, int THREADS, bool POST, bool PRE>
__global__ void __launch_bounds__(THREADS, VPT == 1 ? 2 : 1) k_norm_grad(const NormGradArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using V = Vec<T>;
  constexpr int N = V::N, PN = V::P;
  extern __shared__ uint4 s_ring[];  // weights, then [stages][tensors][VPT * blockDim.x]
  __shared__ Red s_red[2];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = a.d / N;
  const bool gate_rows = POST && gate_in_ring(a.gate, a.span, a.T, Weights<T, VPT>::kKept);
  // ring tensors, in order: dh, z, y (those that there are), dz, gate
  const bool has_dz = a.dz != nullptr;
  const uint32_t step = nt * 16, tensor = VPT * step;  // bytes
  const uint32_t at_z = tensor, at_y = PRE ? 2 * tensor : 0;
  const uint32_t at_dz = at_y + (POST ? tensor : 0), at_g = at_dz + (has_dz ? tensor : 0);
  const int live = nvec - tid;  // vector i of this thread exists when i * nt < live
  clear(s_red);

  // w_post and the gate are constant over the tokens of one gate row, so both
  // their gradients come from one sum over those tokens, acc_gu = sum(g u):
  // dgate = w_post acc_gu, and dw_post grows by gate acc_gu
  float2 acc_post[POST ? VPT : 1][PN] = {}, acc_gu[POST ? VPT : 1][PN] = {};
  float2 acc_pre[PRE ? VPT : 1][PN] = {};
  const uint32_t mine = tc::smem_addr(s_ring) + tid * 16;
  Weights<T, VPT> wpost, gate, wpre;
  if constexpr (POST) {
    wpost.keep(mine, a.w_post, step, live);
  }
  if constexpr (PRE) wpre.keep(mine + (POST ? 2 * tensor : 0), a.w_pre, step, live);
  const uint32_t kept = Weights<T, VPT>::kKept ? (2 * POST + PRE) * tensor : 0;
  const int r0 = first_row(blockIdx.x, gridDim.x, a.T);
  const int r1 = first_row(blockIdx.x + 1, gridDim.x, a.T);
  const float inv_d = 1.0f / (float)a.d;
  int red = 0;

  Ring ring;
  ring.start(mine + kept, a.stages, at_g + (gate_rows ? tensor : 0));
  uint32_t st = 0;  // the slot of the row at hand
  size_t in = (size_t)r0 * nvec + tid, out = in;  // vectors: next row to copy, to write
  const uint4 *pg = nullptr;
  int to_copy = r1 - r0, gate_left = 0;
  if (gate_rows) {
    pg = static_cast<const uint4 *>(a.gate) + (size_t)(r0 / a.span) * nvec + tid;
    gate_left = a.span - r0 % a.span;
  }
  auto issue = [&]() {
    if (to_copy > 0) {
      --to_copy;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          const uint32_t to = ring.put + i * step;
          if constexpr (PRE) {
            copy16(to, static_cast<const uint4 *>(a.dh) + in + i * nt);
            copy16(to + at_z, static_cast<const uint4 *>(a.z) + in + i * nt);
          }
          if constexpr (POST) copy16(to + at_y, static_cast<const uint4 *>(a.y) + in + i * nt);
          if (has_dz) copy16(to + at_dz, static_cast<const uint4 *>(a.dz) + in + i * nt);
          if (gate_rows) copy16(to + at_g, pg + i * nt);
        }
      }
      in += nvec;
      if (gate_rows && --gate_left == 0) {
        pg += nvec;
        gate_left = a.span;
      }
      ring.put = ring.next(ring.put);
    }
    copy_commit();
  };
  for (int s = 0; s < a.stages - 1; ++s) issue();
  float next_pre = 0.f, next_post = 0.f;
  if (r0 < r1) {
    if (PRE) next_pre = a.rstd_pre[r0];
    if (POST) next_post = a.post_norm ? a.rstd_post[r0] : 1.f;
  }
  // the rows of one gate row at a time
  int seg1 = r1;
  for (int seg0 = r0; seg0 < r1; seg0 = seg1) {
    int g = 0;
    if (POST && a.gate) {
      g = seg0 / a.span;
      seg1 = seg0 + min(r1 - seg0, a.span - (seg0 - g * a.span));
    }
    if (POST && !gate_rows)
      gate.keep(mine + tensor, gate_row(a.gate, g, nvec), step, live);
    for (int r = seg0; r < seg1; ++r) {
      issue();
      const float rs_pre = next_pre, rs_post = next_post;
      if (r + 1 < r1) {
        if (PRE) next_pre = a.rstd_pre[r + 1];
        if (POST && a.post_norm) next_post = a.rstd_post[r + 1];
      }
      copy_wait(a.stages - 1);
      st = ring.get;
      ring.get = ring.next(st);
      float2 s0 = both(0.f), s1 = both(0.f), s2 = both(0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          const uint32_t at = st + i * step;
          uint4 qdz = make_uint4(0, 0, 0, 0), qdh, qz, qy, qg, qw, qp;
          if (has_dz) qdz = lds16(at + at_dz);
          if constexpr (PRE) {
            qdh = lds16(at);
            qz = lds16(at + at_z);
            qp = wpre.get(i);
          }
          if constexpr (POST) {
            qy = lds16(at + at_y);
            qg = gate_rows ? lds16(at + at_g) : gate.get(i);
            qw = wpost.get(i);
          }
#pragma unroll
          for (int q = 0; q < PN; ++q) {
            float2 dv, z;
            if constexpr (PRE) {
              dv = mul2(V::pair(qdh, q), V::pair(qp, q));
              z = V::pair(qz, q);
              s0 = fma2(dv, z, s0);
            }
            if constexpr (POST) {
              const float2 c = mul2(mul2(V::pair(qy, q), V::pair(qw, q)), V::pair(qg, q));
              float2 t = V::pair(qdz, q);
              if constexpr (PRE) {
                t = fma2(both(rs_pre), dv, t);
                s2 = fma2(c, z, s2);
              }
              s1 = fma2(c, t, s1);
            }
          }
        }
      }
      // of z and y as stored; their factors rstd follow here
      float t0 = s0.x + s0.y, t1 = s1.x + s1.y, t2 = s2.x + s2.y;
      if constexpr (PRE && POST) {
        block_sum3(t0, t1, t2, s_red[red ^= 1]);
      } else if constexpr (PRE) {
        t0 = block_sum(t0, s_red[red ^= 1]);
      } else {
        t1 = block_sum(t1, s_red[red ^= 1]);
      }
      const float m_pre = t0 * rs_pre * inv_d;  // mean(dh w_pre v)
      float m_post = rs_post * (t1 - rs_pre * rs_pre * m_pre * t2) * inv_d;
      if (!a.post_norm) m_post = 0.f;  // no mean to take out
      // g = dz + rs_pre dh w_pre + k_pre z;  dy = rs_post g c + k_post y
      const float k_pre = -rs_pre * rs_pre * m_pre, k_post = -rs_post * rs_post * m_post;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          const uint32_t at = st + i * step;
          uint4 qdz = make_uint4(0, 0, 0, 0), qdh, qz, qy, qg, qw, qp, o, oy;
          if (has_dz) qdz = lds16(at + at_dz);
          if constexpr (PRE) {
            qdh = lds16(at);
            qz = lds16(at + at_z);
            qp = wpre.get(i);
          }
          if constexpr (POST) {
            qy = lds16(at + at_y);
            qg = gate_rows ? lds16(at + at_g) : gate.get(i);
            qw = wpost.get(i);
          }
#pragma unroll
          for (int q = 0; q < PN; ++q) {
            float2 gr = V::pair(qdz, q);
            if constexpr (PRE) {
              const float2 z = V::pair(qz, q);
              const float2 dh = mul2(V::pair(qdh, q), both(rs_pre));
              acc_pre[i][q] = fma2(dh, z, acc_pre[i][q]);
              gr = fma2(both(k_pre), z, fma2(dh, V::pair(qp, q), gr));
            }
            V::set(o, q, POST ? mul2(both(a.alpha), gr) : gr);
            if constexpr (POST) {
              const float2 y = V::pair(qy, q), gt = V::pair(qg, q), w = V::pair(qw, q);
              gr = mul2(gr, both(rs_post));
              acc_gu[i][q] = fma2(gr, y, acc_gu[i][q]);
              V::set(oy, q, fma2(both(k_post), y, mul2(mul2(gr, gt), w)));
            }
          }
          static_cast<uint4 *>(a.dx)[out + i * nt] = o;
          if constexpr (POST) static_cast<uint4 *>(a.dy)[out + i * nt] = oy;
        }
      }
      out += nvec;
    }
    if constexpr (POST) {
      // whole gate rows are done; parts of one wait for the others
      const int first = g * a.span;
      const bool whole = seg0 == first && seg1 - first == min(a.T - first, a.span);
      float *to = whole ? a.dgate + (size_t)g * a.d
                        : a.part_gate + ((size_t)blockIdx.x * 2 + (seg0 != r0)) * a.d;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * nt < live) {
          const uint4 qg = gate_rows ? lds16(st + i * step + at_g) : gate.get(i);
          const uint4 qw = wpost.get(i);
          float2 dg[PN];
#pragma unroll
          for (int q = 0; q < PN; ++q) {
            acc_post[i][q] = fma2(acc_gu[i][q], V::pair(qg, q), acc_post[i][q]);
            dg[q] = mul2(acc_gu[i][q], V::pair(qw, q));
            acc_gu[i][q] = both(0.f);
          }
          if (a.dgate) store_sums<PN>(to + (size_t)(i * nt + tid) * N, dg);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (i * nt < live) {
      const size_t at = (size_t)blockIdx.x * a.d + (size_t)(i * nt + tid) * N;
      if constexpr (POST)
        if (a.part_post) store_sums<PN>(a.part_post + at, acc_post[i]);
      if constexpr (PRE)
        if (a.part_pre) store_sums<PN>(a.part_pre + at, acc_pre[i]);
    }
  }
}

// The partial sums of `ctas` CTAs into dw_post (blockIdx.y 0), dw_pre (1) and
// the gate rows that cross CTA ranges (2 ..).  A block takes 128 columns, four a
// lane; its warps add every kReduceWarps-th CTA and the warps' sums are added in
// order.
constexpr int kReduceWarps = 16;
struct NormReduceArgs {
  const float *part_post, *part_pre, *part_gate;
  float *dw_post, *dw_pre, *dgate;
  int ctas, T, d, span, by_group;
};
__global__ void __launch_bounds__(kReduceWarps * 32) k_norm_reduce(const NormReduceArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  __shared__ float4 s_sum[kReduceWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int col = (blockIdx.x * 32 + lane) * 4;  // d is a multiple of 4
  const float *part;
  float *out;
  int b0 = 0, b1 = a.ctas - 1;
  size_t step = a.d, first_off = 0;  // later CTAs of a gate row have it in slot 0
  if (blockIdx.y < 2) {
    part = blockIdx.y ? a.part_pre : a.part_post;
    out = blockIdx.y ? a.dw_pre : a.dw_post;
    if (!out) return;
  } else {
    // the gate row: number y - 2, or the one that holds CTA y - 2's last row
    const int y = blockIdx.y - 2;
    const int g = a.by_group ? y : (first_row(y + 1, a.ctas, a.T) - 1) / a.span;
    const int lo = g * a.span, hi = lo + min(a.T - lo, a.span) - 1;
    // the CTA of a row: first_row(b) <= row < first_row(b + 1)
    b0 = (int)((long long)lo * a.ctas / a.T);
    while (b0 + 1 < a.ctas && first_row(b0 + 1, a.ctas, a.T) <= lo) ++b0;
    b1 = (int)((long long)hi * a.ctas / a.T);
    while (b1 + 1 < a.ctas && first_row(b1 + 1, a.ctas, a.T) <= hi) ++b1;
    if (b0 == b1) return;                      // written by its one CTA
    if (!a.by_group && b0 != y) return;        // another block's
    part = a.part_gate;
    out = a.dgate + (size_t)g * a.d;
    step = 2 * (size_t)a.d;
    first_off = first_row(b0, a.ctas, a.T) == lo ? 0 : a.d;
  }
  auto add = [](float4 x, float4 y) {
    return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  };
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < a.d) {
#pragma unroll 8
    for (int b = b0 + warp; b <= b1; b += kReduceWarps)
      s = add(s, *reinterpret_cast<const float4 *>(part + (size_t)b * step +
                                                   (b == b0 ? first_off : 0) + col));
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < a.d) {
    s = s_sum[0][lane];
#pragma unroll
    for (int w = 1; w < kReduceWarps; ++w) s = add(s, s_sum[w][lane]);
    *reinterpret_cast<float4 *>(out + col) = s;
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Vectors per thread and threads of a row: as many threads as there are
// vectors, up to row_threads.  Rows of more than 896 vectors take four a thread,
// with their weights through L1: 8192 x 7176 bf16 99 us where 8192 x 7168 takes 87.
struct RowShape {
  int vpt, nt;
};
RowShape row_shape(int nvec) {
  RowShape s;
  s.vpt = nvec <= row_threads(1) ? 1 : (nvec <= 2 * row_threads(2) ? 2 : 4);
  s.nt = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  return s;
}
// The backward pass keeps its sums in registers, so it takes fewer threads with
// 128 registers each: 16381 x 4096, with 256 threads of two vectors 165 us, with
// 512 of one, whose 64 registers spilled, 208.  `most`: the threads a kernel is
// compiled for; for 512 in place of 448 rows of 4096 took 135 us for 130 (14333
// rows), so it is for the rows that need it.
struct GradShape {
  int vpt, most, nt;
};
GradShape grad_shape(int nvec) {
  GradShape s;
  s.vpt = nvec <= 256 ? 1 : (nvec <= 1024 ? 2 : 4);
  s.most = s.vpt == 1 ? 256 : (nvec <= 896 ? 448 : 512);
  s.nt = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  return s;
}
// Rows in a ring: two, three where they leave the L1 cache enough for what goes
// through it (weights of long rows, spilled registers).  Two against as many as
// fit: gradient, 8189 x 7168 128 us against 150 (of three), 14333 x 4096 129 either
// way; forward, 4775 x 12288 90 against 128 (of four).  Three against two: forward
// without an h, 14333 x 4096 57 against 61.  One against two: gradient, 4775 x
// 12288 185 against 218 (192 KB), 5731 x 10240 208 against 198 (160 KB).
int stages_for(size_t row_bytes, size_t weight_bytes, int ctas_per_sm, bool weights_in_l1) {
  const size_t limit[2] = {weights_in_l1 ? 160u << 10 : kRingLimit,
                           weights_in_l1 ? 128u << 10 : 160u << 10};
  int n = 1;
  while (n < kMaxStages && ctas_per_sm * (weight_bytes + (n + 1) * row_bytes) <= limit[n - 1]) ++n;
  return n;
}
// CTAs of the backward pass: up to 512 threads and 16 CTAs an SM, and no more
// CTAs than rows.
int grad_ctas(const moe_norm_config &c) {
  const GradShape r = grad_shape(c.d / (c.dtype == MOE_F32 ? 4 : 8));
  const int per_sm = std::max(1, std::min(16, 512 / r.nt));
  return std::min(c.T, kNormSms * per_sm);
}

template <typename T, int VPT, bool POST, bool PRE>
cudaError_t run_norm(const NormArgs &a0, int nt, cudaStream_t s) {
  NormArgs a = a0;
  constexpr bool kKept = Weights<T, VPT>::kKept;
  const int tensors = 1 + POST + (POST && gate_in_ring(a.gate, a.span, a.T, kKept));
  const size_t row = (size_t)tensors * VPT * nt * 16;
  const int per_sm = std::max(1, std::min(16, (VPT == 4 ? 512 : 1024) / nt));
  const size_t kept = kKept ? (size_t)(2 * POST + PRE) * VPT * nt * 16 : 0;
  a.stages = stages_for(row, kept, per_sm, !kKept);
  const size_t smem = kept + a.stages * row;
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = tc::set_smem_once(attr_set, k_norm<T, VPT, POST, PRE>, kRingLimit)) return e;
  const int grid = a.T < kNormSms * per_sm ? a.T : kNormSms * per_sm;
  launch_k(k_norm<T, VPT, POST, PRE>, grid, nt, smem, s, a);
  return cudaGetLastError();
}

template <typename T, int VPT>
cudaError_t run_norm_parts(const NormArgs &a, int nt, cudaStream_t s) {
  const bool pre = a.h || a.hq;
  if (a.y && pre) return run_norm<T, VPT, true, true>(a, nt, s);
  if (a.y) return run_norm<T, VPT, true, false>(a, nt, s);
  return run_norm<T, VPT, false, true>(a, nt, s);
}

template <typename T, int VPT, int THREADS, bool POST, bool PRE>
cudaError_t run_grad(const NormGradArgs &a0, int nt, int ctas, cudaStream_t s) {
  NormGradArgs a = a0;
  constexpr bool kKept = Weights<T, VPT>::kKept;
  const int tensors = (a.dz != nullptr) + 2 * PRE + POST +
                      (POST && gate_in_ring(a.gate, a.span, a.T, kKept));
  const size_t row = (size_t)tensors * VPT * nt * 16;
  const int per_sm = (ctas + kNormSms - 1) / kNormSms;
  const size_t kept = kKept ? (size_t)(2 * POST + PRE) * VPT * nt * 16 : 0;
  a.stages = stages_for(row, kept, per_sm, !kKept);
  const size_t smem = kept + a.stages * row;
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e =
          tc::set_smem_once(attr_set, k_norm_grad<T, VPT, THREADS, POST, PRE>, kRingLimit))
    return e;
  launch_k(k_norm_grad<T, VPT, THREADS, POST, PRE>, ctas, nt, smem, s, a);
  return cudaGetLastError();
}

template <typename T, int VPT, int THREADS>
cudaError_t run_grad_parts(const NormGradArgs &a, int nt, int ctas, cudaStream_t s) {
  if (a.y && a.dh) return run_grad<T, VPT, THREADS, true, true>(a, nt, ctas, s);
  if (a.y) return run_grad<T, VPT, THREADS, true, false>(a, nt, ctas, s);
  return run_grad<T, VPT, THREADS, false, true>(a, nt, ctas, s);
}

template <typename T>
cudaError_t run_grad_shape(const NormGradArgs &a, int ctas, cudaStream_t s) {
  const GradShape r = grad_shape(a.d / Vec<T>::N);
  if (r.vpt == 1) return run_grad_parts<T, 1, 256>(a, r.nt, ctas, s);
  if (r.vpt == 4) return run_grad_parts<T, 4, 512>(a, r.nt, ctas, s);
  return r.most == 448 ? run_grad_parts<T, 2, 448>(a, r.nt, ctas, s)
                       : run_grad_parts<T, 2, 512>(a, r.nt, ctas, s);
}

}  // namespace

size_t norm_workspace_bytes(const moe_norm_config &c) {
  // partial sums: dw_post, dw_pre, two gate slots
  return (size_t)grad_ctas(c) * c.d * sizeof(float) * 4;
}

cudaError_t launch_norm(const moe_norm_config &c, const moe_norm_io &io, cudaStream_t s) {
  NormArgs a{io.x, io.y, io.w_post, io.gate, io.w_pre, io.z, io.h, io.hq, io.h_scale,
             io.rstd_post, io.rstd_pre, c.T, c.d, std::min(c.gate_span, c.T), 1, c.post_norm,
             c.residual_scale, c.eps_post, c.eps_pre};
  if (c.dtype == MOE_F32) {
    const RowShape r = row_shape(c.d / 4);
    if (r.vpt == 1) return run_norm_parts<float, 1>(a, r.nt, s);
    if (r.vpt == 2) return run_norm_parts<float, 2>(a, r.nt, s);
    return run_norm_parts<float, 4>(a, r.nt, s);
  }
  const RowShape r = row_shape(c.d / 8);
  if (r.vpt == 1) return run_norm_parts<__nv_bfloat16, 1>(a, r.nt, s);
  if (r.vpt == 2) return run_norm_parts<__nv_bfloat16, 2>(a, r.nt, s);
  return run_norm_parts<__nv_bfloat16, 4>(a, r.nt, s);
}

cudaError_t launch_norm_grad(const moe_norm_config &c, const moe_norm_grad_io &io, void *ws,
                             cudaStream_t s) {
  const int ctas = grad_ctas(c);
  float *parts = static_cast<float *>(ws);
  const size_t block = (size_t)ctas * c.d;
  const int span = std::min(c.gate_span, c.T);  // row 0 for every token either way
  NormGradArgs a{io.dz, io.dh, io.z, io.y, io.w_post, io.gate, io.w_pre, io.rstd_post,
                 io.rstd_pre, io.dx, io.dy, io.dgate, io.dw_post ? parts : nullptr,
                 io.dw_pre ? parts + block : nullptr, parts + 2 * block, c.T, c.d, span, 1,
                 c.post_norm, c.residual_scale};
  const cudaError_t e = c.dtype == MOE_F32 ? run_grad_shape<float>(a, ctas, s)
                                           : run_grad_shape<__nv_bfloat16>(a, ctas, s);
  if (e != cudaSuccess) return e;
  if (!io.dw_post && !io.dw_pre && !io.dgate) return cudaSuccess;
  // gate rows to look at: all of them, or one per CTA when there are more rows
  int gates = 0, by_group = 1;
  if (io.dgate && span > 1) {
    gates = (c.T - 1) / span + 1;
    if (gates > ctas) {
      gates = ctas;
      by_group = 0;
    }
  }
  if (!io.dw_post && !io.dw_pre && !gates) return cudaSuccess;
  NormReduceArgs ra{a.part_post, a.part_pre, a.part_gate, io.dw_post, io.dw_pre, io.dgate, ctas,
                    c.T, c.d, span, by_group};
  launch_k(k_norm_reduce, dim3((c.d + 127) / 128, 2 + gates), kReduceWarps * 32, 0, s, ra);
  return cudaGetLastError();
}

}  // namespace moe
