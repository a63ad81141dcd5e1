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
#include <algorithm>

#include "quantize_rows.cuh"

namespace moe {
namespace {

constexpr int kMaxStages = 4;
constexpr size_t kRingLimit = 216u << 10;  // shared memory for the rings of one SM
constexpr int kNormSms = 148;

__device__ __forceinline__ void copy16(void *smem, const void *gmem) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Wait until at most n of this thread's copy groups are still in flight.
__device__ __forceinline__ void copy_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// Sums of NV values over the block, in a fixed order.  `red`: one of two
// buffers of 32 float4 that consecutive calls take in turn.
template <int NV>
__device__ __forceinline__ void block_sums(float (&v)[NV], float4 *red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int q = 0; q < NV; ++q) v[q] += __shfl_xor_sync(0xffffffffu, v[q], off);
  const int nw = blockDim.x / 32;
  if (nw == 1) return;
  if (threadIdx.x % 32 == 0) {
    float4 f = make_float4(v[0], 0.f, 0.f, 0.f);
    if (NV > 1) f.y = v[NV > 1 ? 1 : 0];
    if (NV > 2) f.z = v[NV > 2 ? 2 : 0];
    red[threadIdx.x / 32] = f;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < NV; ++q) v[q] = 0.f;
  for (int w = 0; w < nw; ++w) {
    const float4 f = red[w];
    v[0] += f.x;
    if (NV > 1) v[NV > 1 ? 1 : 0] += f.y;
    if (NV > 2) v[NV > 2 ? 2 : 0] += f.z;
  }
}
__device__ __forceinline__ float block_max(float v, float4 *red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  const int nw = blockDim.x / 32;
  if (nw == 1) return v;
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32].x = v;
  __syncthreads();
  for (int w = 0; w < nw; ++w) v = fmaxf(v, red[w].x);
  return v;
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
  int T, d, span, stages;
  float alpha, eps_post, eps_pre;
};

template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 128 : 512) k_norm(const NormArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using V = Vec<T>;
  constexpr int N = V::N;
  extern __shared__ uint4 s_ring[];  // [stages][tensors][VPT * blockDim.x]
  __shared__ float4 s_red[2][32];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = a.d / N;
  const int span_vecs = VPT * nt;
  const bool post = a.y != nullptr, pre = a.h || a.hq;
  const bool gate_rows = a.gate && a.span < a.T;  // a gate row per span: through the ring
  const int tensors = 1 + post + gate_rows;
  const uint4 *src[3] = {static_cast<const uint4 *>(a.x), static_cast<const uint4 *>(a.y),
                         static_cast<const uint4 *>(a.gate)};

  uint4 wpost[VPT], gate[VPT], wpre[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nt + tid;
    if (v < nvec) {
      if (a.w_post) wpost[i] = static_cast<const uint4 *>(a.w_post)[v];
      if (a.gate && !gate_rows) gate[i] = src[2][v];
      if (a.w_pre) wpre[i] = static_cast<const uint4 *>(a.w_pre)[v];
    }
  }
  const int r0 = first_row(blockIdx.x, gridDim.x, a.T);
  const int r1 = first_row(blockIdx.x + 1, gridDim.x, a.T);
  const float inv_d = 1.0f / (float)a.d;
  int red = 0;

  auto issue = [&](int r) {  // this thread's vectors of row r into its ring slot
    if (r < r1) {
      uint4 *st = s_ring + (size_t)((r - r0) % a.stages) * tensors * span_vecs;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + tid;
        if (v < nvec) {
          copy16(st + v, src[0] + (size_t)r * nvec + v);
          if (post) copy16(st + span_vecs + v, src[1] + (size_t)r * nvec + v);
          if (gate_rows)
            copy16(st + 2 * span_vecs + v, src[2] + (size_t)(r / a.span) * nvec + v);
        }
      }
    }
    copy_commit();
  };
  for (int s = 0; s < a.stages - 1; ++s) issue(r0 + s);

  for (int r = r0; r < r1; ++r) {
    issue(r + a.stages - 1);
    copy_wait(a.stages - 1);
    const uint4 *st = s_ring + (size_t)((r - r0) % a.stages) * tensors * span_vecs;
    uint4 z[VPT];
    float sum[1] = {0.f};
    if (post) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + tid;
        if (v < nvec) {
          float f[N];
          V::get(st[span_vecs + v], f);
#pragma unroll
          for (int q = 0; q < N; ++q) sum[0] = fmaf(f[q], f[q], sum[0]);
        }
      }
      block_sums(sum, s_red[red ^= 1]);
      const float rs = rsqrtf(fmaf(sum[0], inv_d, a.eps_post));
      if (tid == 0 && a.rstd_post) a.rstd_post[r] = rs;
      sum[0] = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + tid;
        if (v < nvec) {
          float fx[N], f[N], w[N];
          V::get(st[v], fx);
          V::get(st[span_vecs + v], f);
#pragma unroll
          for (int q = 0; q < N; ++q) f[q] *= rs;
          if (a.w_post) {
            V::get(wpost[i], w);
#pragma unroll
            for (int q = 0; q < N; ++q) f[q] *= w[q];
          }
          if (a.gate) {
            V::get(gate_rows ? st[2 * span_vecs + v] : gate[i], w);
#pragma unroll
            for (int q = 0; q < N; ++q) f[q] *= w[q];
          }
#pragma unroll
          for (int q = 0; q < N; ++q) f[q] = fmaf(a.alpha, fx[q], f[q]);
          z[i] = V::put(f);
          static_cast<uint4 *>(a.z)[(size_t)r * nvec + v] = z[i];
          V::get(z[i], f);  // z as stored
#pragma unroll
          for (int q = 0; q < N; ++q) sum[0] = fmaf(f[q], f[q], sum[0]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + tid;
        if (v < nvec) {
          float f[N];
          z[i] = st[v];
          V::get(z[i], f);
#pragma unroll
          for (int q = 0; q < N; ++q) sum[0] = fmaf(f[q], f[q], sum[0]);
        }
      }
    }
    if (!pre) continue;
    block_sums(sum, s_red[red ^= 1]);
    const float rs = rsqrtf(fmaf(sum[0], inv_d, a.eps_pre));
    if (tid == 0 && a.rstd_pre) a.rstd_pre[r] = rs;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + tid;
      if (v < nvec) {
        float f[N], w[N];
        V::get(z[i], f);
#pragma unroll
        for (int q = 0; q < N; ++q) f[q] *= rs;
        if (a.w_pre) {
          V::get(wpre[i], w);
#pragma unroll
          for (int q = 0; q < N; ++q) f[q] *= w[q];
        }
        z[i] = V::put(f);  // h from here on
        if (a.h) static_cast<uint4 *>(a.h)[(size_t)r * nvec + v] = z[i];
        if (a.hq) {
          V::get(z[i], f);
#pragma unroll
          for (int q = 0; q < N; ++q) top = fmaxf(top, i8::magnitude(f[q]));
        }
      }
    }
    if (!a.hq) continue;
    const i8::RowScale q8 = i8::row_scale(block_max(top, s_red[red ^= 1]));
    if (tid == 0) a.h_scale[r] = q8.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + tid;
      if (v < nvec) {
        float f[N];
        V::get(z[i], f);
        uint32_t c[N / 4];
        i8::codes<N>(f, q8, c);
        i8::store<N>(a.hq + (size_t)r * a.d + (size_t)v * N, c);
      }
    }
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
  int T, d, span, stages;
  float alpha;
};

template <typename T, int VPT, bool POST, bool PRE>
__global__ void __launch_bounds__(VPT == 1 ? 128 : 512) k_norm_grad(const NormGradArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using V = Vec<T>;
  constexpr int N = V::N;
  extern __shared__ uint4 s_ring[];  // [stages][tensors][VPT * blockDim.x]
  __shared__ float4 s_red[2][32];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = a.d / N;
  const int span_vecs = VPT * nt;
  const bool gate_rows = POST && a.gate && a.span < a.T;
  // ring tensors, in order: dz, dh, z, y, gate (those that there are)
  const bool has_dz = a.dz != nullptr;
  const int at_dh = has_dz, at_z = at_dh + PRE, at_y = at_z + PRE, at_g = at_y + POST;
  const int tensors = at_g + gate_rows;

  uint4 wpost[VPT], gate[VPT], wpre[VPT];
  float acc_post[POST ? VPT : 1][N] = {}, acc_gate[POST ? VPT : 1][N] = {};
  float acc_pre[PRE ? VPT : 1][N] = {};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nt + tid;
    if (v < nvec) {
      if (POST && a.w_post) wpost[i] = static_cast<const uint4 *>(a.w_post)[v];
      if (POST && a.gate && !gate_rows) gate[i] = static_cast<const uint4 *>(a.gate)[v];
      if (PRE && a.w_pre) wpre[i] = static_cast<const uint4 *>(a.w_pre)[v];
    }
  }
  const int r0 = first_row(blockIdx.x, gridDim.x, a.T);
  const int r1 = first_row(blockIdx.x + 1, gridDim.x, a.T);
  const float inv_d = 1.0f / (float)a.d;
  int red = 0, seg0 = r0;  // seg0: first row of the gate row at hand

  auto issue = [&](int r) {
    if (r < r1) {
      uint4 *st = s_ring + (size_t)((r - r0) % a.stages) * tensors * span_vecs;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nt + tid;
        if (v < nvec) {
          const size_t at = (size_t)r * nvec + v;
          if (has_dz) copy16(st + v, static_cast<const uint4 *>(a.dz) + at);
          if (PRE) {
            copy16(st + at_dh * span_vecs + v, static_cast<const uint4 *>(a.dh) + at);
            copy16(st + at_z * span_vecs + v, static_cast<const uint4 *>(a.z) + at);
          }
          if (POST) copy16(st + at_y * span_vecs + v, static_cast<const uint4 *>(a.y) + at);
          if (gate_rows)
            copy16(st + at_g * span_vecs + v,
                   static_cast<const uint4 *>(a.gate) + (size_t)(r / a.span) * nvec + v);
        }
      }
    }
    copy_commit();
  };
  for (int s = 0; s < a.stages - 1; ++s) issue(r0 + s);
  float next_pre = 0.f, next_post = 0.f;
  if (r0 < r1) {
    if (PRE) next_pre = a.rstd_pre[r0];
    if (POST) next_post = a.rstd_post[r0];
  }

  for (int r = r0; r < r1; ++r) {
    issue(r + a.stages - 1);
    const float rs_pre = next_pre, rs_post = next_post;
    if (r + 1 < r1) {
      if (PRE) next_pre = a.rstd_pre[r + 1];
      if (POST) next_post = a.rstd_post[r + 1];
    }
    copy_wait(a.stages - 1);
    const uint4 *st = s_ring + (size_t)((r - r0) % a.stages) * tensors * span_vecs;
    // per vector: dz, dv = dh * w_pre, v, u, and c = gate * w_post
    auto load = [&](int i, int v, float (&dz)[N], float (&dv)[N], float (&vv)[N], float (&u)[N],
                    float (&c)[N], float (&wp)[N], float (&gt)[N], float (&dh)[N]) {
      if (has_dz) {
        V::get(st[v], dz);
      } else {
#pragma unroll
        for (int q = 0; q < N; ++q) dz[q] = 0.f;
      }
      if (PRE) {
        float w[N];
        V::get(st[at_dh * span_vecs + v], dh);
        V::get(st[at_z * span_vecs + v], vv);
        if (a.w_pre) {
          V::get(wpre[i], w);
#pragma unroll
          for (int q = 0; q < N; ++q) dv[q] = dh[q] * w[q];
        } else {
#pragma unroll
          for (int q = 0; q < N; ++q) dv[q] = dh[q];
        }
#pragma unroll
        for (int q = 0; q < N; ++q) vv[q] *= rs_pre;
      }
      if (POST) {
        V::get(st[at_y * span_vecs + v], u);
#pragma unroll
        for (int q = 0; q < N; ++q) u[q] *= rs_post;
        if (a.w_post) {
          V::get(wpost[i], wp);
        } else {
#pragma unroll
          for (int q = 0; q < N; ++q) wp[q] = 1.f;
        }
        if (a.gate) {
          V::get(gate_rows ? st[at_g * span_vecs + v] : gate[i], gt);
        } else {
#pragma unroll
          for (int q = 0; q < N; ++q) gt[q] = 1.f;
        }
#pragma unroll
        for (int q = 0; q < N; ++q) c[q] = wp[q] * gt[q];
      }
    };
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + tid;
      if (v < nvec) {
        float dz[N], dv[N], vv[N], u[N], c[N], wp[N], gt[N], dh[N];
        load(i, v, dz, dv, vv, u, c, wp, gt, dh);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          if (PRE) s[0] = fmaf(dv[q], vv[q], s[0]);
          if (POST) {
            const float cu = c[q] * u[q];
            s[1] = fmaf(cu, PRE ? fmaf(rs_pre, dv[q], dz[q]) : dz[q], s[1]);
            if (PRE) s[2] = fmaf(cu, vv[q], s[2]);
          }
        }
      }
    }
    block_sums(s, s_red[red ^= 1]);
    const float m_pre = s[0] * inv_d;
    const float m_post = (s[1] - rs_pre * m_pre * s[2]) * inv_d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nt + tid;
      if (v < nvec) {
        float dz[N], dv[N], vv[N], u[N], c[N], wp[N], gt[N], dh[N], o[N];
        load(i, v, dz, dv, vv, u, c, wp, gt, dh);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          if constexpr (PRE) {
            acc_pre[i][q] = fmaf(dh[q], vv[q], acc_pre[i][q]);
            dz[q] = fmaf(rs_pre, fmaf(-vv[q], m_pre, dv[q]), dz[q]);
          }
          o[q] = POST ? a.alpha * dz[q] : dz[q];
        }
        static_cast<uint4 *>(a.dx)[(size_t)r * nvec + v] = V::put(o);
        if constexpr (POST) {
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const float gu = dz[q] * u[q];
            acc_post[i][q] = fmaf(gu, gt[q], acc_post[i][q]);
            acc_gate[i][q] = fmaf(gu, wp[q], acc_gate[i][q]);
            o[q] = rs_post * fmaf(-u[q], m_post, dz[q] * c[q]);
          }
          static_cast<uint4 *>(a.dy)[(size_t)r * nvec + v] = V::put(o);
        }
      }
    }
    if constexpr (POST) if (a.dgate) {  // the last row of a gate row, or of this range
      const int g = r / a.span;
      const bool ends = r + 1 == a.T || (r + 1) % a.span == 0;
      if (ends || r + 1 == r1) {
        const bool whole = ends && seg0 == g * a.span;
        float *to = whole ? a.dgate + (size_t)g * a.d
                          : a.part_gate + ((size_t)blockIdx.x * 2 + (seg0 != r0)) * a.d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = i * nt + tid;
          if (v < nvec) {
#pragma unroll
            for (int q = 0; q < N; q += 4)
              *reinterpret_cast<float4 *>(to + (size_t)v * N + q) =
                  make_float4(acc_gate[i][q], acc_gate[i][q + 1], acc_gate[i][q + 2],
                              acc_gate[i][q + 3]);
          }
#pragma unroll
          for (int q = 0; q < N; ++q) acc_gate[i][q] = 0.f;
        }
        seg0 = r + 1;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nt + tid;
    if (v < nvec) {
      const size_t at = (size_t)blockIdx.x * a.d + (size_t)v * N;
#pragma unroll
      for (int q = 0; q < N; q += 4) {
        if constexpr (POST) {
          if (a.part_post)
            *reinterpret_cast<float4 *>(a.part_post + at + q) =
                make_float4(acc_post[i][q], acc_post[i][q + 1], acc_post[i][q + 2],
                            acc_post[i][q + 3]);
        }
        if constexpr (PRE) {
          if (a.part_pre)
            *reinterpret_cast<float4 *>(a.part_pre + at + q) = make_float4(
                acc_pre[i][q], acc_pre[i][q + 1], acc_pre[i][q + 2], acc_pre[i][q + 3]);
        }
      }
    }
  }
}

// The partial sums of `ctas` CTAs into dw_post (blockIdx.y 0), dw_pre (1) and
// the gate rows that cross CTA ranges (2 ..).  A block takes 32 columns; its
// warps add every kReduceWarps-th CTA and the warps' sums are added in order.
constexpr int kReduceWarps = 16;
struct NormReduceArgs {
  const float *part_post, *part_pre, *part_gate;
  float *dw_post, *dw_pre, *dgate;
  int ctas, T, d, span, by_group;
};
__global__ void __launch_bounds__(kReduceWarps * 32) k_norm_reduce(const NormReduceArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  __shared__ float s_sum[kReduceWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
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
  float s = 0.f;
  if (col < a.d) {
#pragma unroll 8
    for (int b = b0 + warp; b <= b1; b += kReduceWarps)
      s += part[(size_t)b * step + (b == b0 ? first_off : 0) + col];
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < a.d) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kReduceWarps; ++w) s += s_sum[w][lane];
    out[col] = s;
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Vectors per thread and threads of a row: two vectors each up to 512 threads,
// four above (rows of 16 to 32 KB).
struct RowShape {
  int vpt, nt;
};
RowShape row_shape(int nvec) {
  RowShape s;
  s.vpt = nvec <= 128 ? 1 : (nvec <= 1024 ? 2 : 4);
  s.nt = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  return s;
}
int stages_for(size_t row_bytes, int ctas_per_sm) {
  const size_t n = kRingLimit / ((size_t)ctas_per_sm * row_bytes);
  return n < 1 ? 1 : (n > kMaxStages ? kMaxStages : (int)n);
}
// CTAs of the backward pass: at most 512 threads and 8 CTAs an SM (its sums
// take most of the registers), and no more CTAs than rows.
int grad_ctas(const moe_norm_config &c) {
  const int nvec = c.d / (c.dtype == MOE_F32 ? 4 : 8);
  const int nt = row_shape(nvec).nt;
  int per_sm = 512 / nt;
  per_sm = per_sm < 1 ? 1 : (per_sm > 8 ? 8 : per_sm);
  const int n = kNormSms * per_sm;
  return c.T < n ? c.T : n;
}

template <typename T, int VPT>
cudaError_t run_norm(const NormArgs &a0, int nt, cudaStream_t s) {
  NormArgs a = a0;
  const int tensors = 1 + (a.y != nullptr) + (a.gate && a.span < a.T);
  const size_t row = (size_t)tensors * VPT * nt * 16;
  int per_sm = 1024 / nt;
  per_sm = per_sm < 1 ? 1 : (per_sm > 16 ? 16 : per_sm);
  a.stages = stages_for(row, per_sm);
  const size_t smem = a.stages * row;
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = tc::set_smem_once(attr_set, k_norm<T, VPT>, kRingLimit)) return e;
  const int grid = a.T < kNormSms * per_sm ? a.T : kNormSms * per_sm;
  launch_k(k_norm<T, VPT>, grid, nt, smem, s, a);
  return cudaGetLastError();
}

template <typename T, int VPT, bool POST, bool PRE>
cudaError_t run_grad(const NormGradArgs &a0, int nt, int ctas, cudaStream_t s) {
  NormGradArgs a = a0;
  const int tensors = (a.dz != nullptr) + 2 * PRE + POST + (POST && a.gate && a.span < a.T);
  const size_t row = (size_t)tensors * VPT * nt * 16;
  const int per_sm = (ctas + kNormSms - 1) / kNormSms;
  a.stages = stages_for(row, per_sm);
  const size_t smem = a.stages * row;
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = tc::set_smem_once(attr_set, k_norm_grad<T, VPT, POST, PRE>, kRingLimit))
    return e;
  launch_k(k_norm_grad<T, VPT, POST, PRE>, ctas, nt, smem, s, a);
  return cudaGetLastError();
}

template <typename T, int VPT>
cudaError_t run_grad_parts(const NormGradArgs &a, int nt, int ctas, cudaStream_t s) {
  if (a.y && a.dh) return run_grad<T, VPT, true, true>(a, nt, ctas, s);
  if (a.y) return run_grad<T, VPT, true, false>(a, nt, ctas, s);
  return run_grad<T, VPT, false, true>(a, nt, ctas, s);
}

}  // namespace

size_t norm_workspace_bytes(const moe_norm_config &c) {
  // partial sums: dw_post, dw_pre, two gate slots
  return (size_t)grad_ctas(c) * c.d * sizeof(float) * 4;
}

cudaError_t launch_norm(const moe_norm_config &c, const moe_norm_io &io, cudaStream_t s) {
  NormArgs a{io.x, io.y, io.w_post, io.gate, io.w_pre, io.z, io.h, io.hq, io.h_scale,
             io.rstd_post, io.rstd_pre, c.T, c.d, std::min(c.gate_span, c.T), 1, c.residual_scale, c.eps_post,
             c.eps_pre};
  if (c.dtype == MOE_F32) {
    const RowShape r = row_shape(c.d / 4);
    if (r.vpt == 1) return run_norm<float, 1>(a, r.nt, s);
    if (r.vpt == 2) return run_norm<float, 2>(a, r.nt, s);
    return run_norm<float, 4>(a, r.nt, s);
  }
  const RowShape r = row_shape(c.d / 8);
  if (r.vpt == 1) return run_norm<__nv_bfloat16, 1>(a, r.nt, s);
  if (r.vpt == 2) return run_norm<__nv_bfloat16, 2>(a, r.nt, s);
  return run_norm<__nv_bfloat16, 4>(a, r.nt, s);
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
                 c.residual_scale};
  cudaError_t e;
  if (c.dtype == MOE_F32) {
    const RowShape r = row_shape(c.d / 4);
    e = r.vpt == 1   ? run_grad_parts<float, 1>(a, r.nt, ctas, s)
        : r.vpt == 2 ? run_grad_parts<float, 2>(a, r.nt, ctas, s)
                     : run_grad_parts<float, 4>(a, r.nt, ctas, s);
  } else {
    const RowShape r = row_shape(c.d / 8);
    e = r.vpt == 1   ? run_grad_parts<__nv_bfloat16, 1>(a, r.nt, ctas, s)
        : r.vpt == 2 ? run_grad_parts<__nv_bfloat16, 2>(a, r.nt, ctas, s)
                     : run_grad_parts<__nv_bfloat16, 4>(a, r.nt, ctas, s);
  }
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
  launch_k(k_norm_reduce, dim3((c.d + 31) / 32, 2 + gates), kReduceWarps * 32, 0, s, ra);
  return cudaGetLastError();
}

}  // namespace moe
