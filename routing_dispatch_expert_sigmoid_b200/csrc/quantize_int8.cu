// Int8 codes: the experts' matrices (one scale per output channel) and rows of
// activations (one scale per row).
//
// Weights W [G, K, N] (bf16), prepared once:
//   scale[g, n]  = max_k |W[g, k, n]| / 127      (fp32 division; 1 if all zero)
//   Wq[g, n, k]  = W[g, k, n] / scale[g, n], rounded to the nearest integer
// stored K-contiguous, the order in which the GEMMs read them.  A block takes
// 32 columns of one group; reads along N and writes along K both pass through
// a 32 x 32 tile in shared memory.  Off the hot path.
//
// Rows (quantize_rows.cuh has the formulas): one block per row, the row in
// registers between the maximum and the codes, so it is read from HBM once:
// rows * K * (2 or 4) bytes in, rows * (K + 4) out, bound by HBM.  Rows longer
// than the registers hold are read twice, the second time from L2.  With a
// slot table (the layer's dispatch) a token's codes go to every row that the
// token was sent to, so the expert-ordered rows are written in the same pass.
#include <algorithm>

#include "quantize_rows.cuh"

namespace moe {
namespace {

constexpr int kCols = 32;

__global__ void __launch_bounds__(256)
    k_quantize_int8(const __nv_bfloat16 *__restrict__ W, int K, int N, int8_t *__restrict__ Wq,
                    float *__restrict__ scale) {
  grid_dependency();  // the previous grid is complete; the next may launch
  __shared__ float s_max[8][kCols];
  __shared__ i8::RowScale s_scale[kCols];
  __shared__ int8_t s_tile[kCols][kCols + 4];  // [n][k]
  const int g = blockIdx.y, n0 = blockIdx.x * kCols;
  const int tx = threadIdx.x % kCols, ty = threadIdx.x / kCols;  // ty: 0..7
  const __nv_bfloat16 *Wg = W + (size_t)g * K * N;
  const int n = n0 + tx;
  float amax = 0.0f;
  if (n < N)
    for (int k = ty; k < K; k += 8) {
      const float a = fabsf(__bfloat162float(Wg[(size_t)k * N + n]));
      amax = a < INFINITY ? fmaxf(amax, a) : INFINITY;  // NaN counts as infinite
    }
  s_max[ty][tx] = amax;
  __syncthreads();
  if (ty == 0) {
    float m = s_max[0][tx];
    for (int i = 1; i < 8; ++i) m = fmaxf(m, s_max[i][tx]);
    const i8::RowScale s = i8::row_scale(m);
    s_scale[tx] = s;
    if (n < N) scale[(size_t)g * N + n] = s.scale;
  }
  __syncthreads();
  int8_t *Qg = Wq + (size_t)g * N * K;
  for (int k0 = 0; k0 < K; k0 += kCols) {
    for (int i = ty; i < kCols; i += 8) {
      const int k = k0 + i;
      int8_t c = 0;
      if (k < K && n < N) c = (int8_t)i8::code(__bfloat162float(Wg[(size_t)k * N + n]), s_scale[tx]);
      s_tile[tx][i] = c;
    }
    __syncthreads();
    for (int i = ty; i < kCols; i += 8) {
      const int nn = n0 + i, k = k0 + tx;
      if (nn < N && k < K) Qg[(size_t)nn * K + k] = s_tile[i][tx];
    }
    __syncthreads();
  }
}

struct RowsArgs {
  const void *x;
  const int32_t *n_rows;    // rows to do (device), or nullptr: all of `rows`
  const int32_t *slot_row;  // [rows, k]: where a row's codes go, or nullptr: its own place
  int rows, K, k, out_rows;
  int8_t *xq;
  float *scale;
  int8_t *own;              // with slot_row: the codes in the row's own place too, or nullptr
  float *own_scale;
  uint32_t *err;
};

// VPT 16-byte vectors of the row per thread; 0: longer rows, read twice.
template <typename T, int VPT>
__global__ void __launch_bounds__(512) k_quantize_rows(const RowsArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ float s_red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = a.K / N, nw = nt / 32;
  int R = a.n_rows ? *a.n_rows : a.rows;
  if (R < 0 || R > a.rows) {
    if (blockIdx.x == 0 && tid == 0) raise_error(a.err, kErrIndex);
    R = 0;
  }
  int red = 0;
  for (int r = blockIdx.x; r < R; r += gridDim.x) {
    const uint4 *row = static_cast<const uint4 *>(a.x) + (size_t)r * nvec;
    uint4 u[VPT > 0 ? VPT : 1];
    float top = 0.0f;
    auto peak = [&](const uint4 &q) {
      float f[N];
      V::get(q, f);
#pragma unroll
      for (int i = 0; i < N; ++i) top = fmaxf(top, i8::magnitude(f[i]));
    };
    if constexpr (VPT > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i * nt + tid < nvec) u[i] = row[i * nt + tid];
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i * nt + tid < nvec) peak(u[i]);
    } else {
      for (int v = tid; v < nvec; v += nt) peak(row[v]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (nw > 1) {
      red ^= 1;
      if (tid % 32 == 0) s_red[red][tid / 32] = top;
      __syncthreads();
      for (int w = 0; w < nw; ++w) top = fmaxf(top, s_red[red][w]);
    }
    const i8::RowScale s = i8::row_scale(top);
    auto put = [&](const uint4 &q, int v) {
      float f[N];
      uint32_t c[N / 4];
      V::get(q, f);
      i8::codes<N>(f, s, c);
      const size_t at = (size_t)v * N;
      if (!a.slot_row) {
        i8::store<N>(a.xq + (size_t)r * a.K + at, c);
        return;
      }
      if (a.own) i8::store<N>(a.own + (size_t)r * a.K + at, c);
      for (int j = 0; j < a.k; ++j) {
        const int to = a.slot_row[(size_t)r * a.k + j];
        if (to >= 0 && to < a.out_rows) i8::store<N>(a.xq + (size_t)to * a.K + at, c);
      }
    };
    if constexpr (VPT > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i * nt + tid < nvec) put(u[i], i * nt + tid);
    } else {
      for (int v = tid; v < nvec; v += nt) put(row[v], v);
    }
    if (!a.slot_row) {
      if (tid == 0) a.scale[r] = s.scale;
    } else {
      if (tid == 0 && a.own) a.own_scale[r] = s.scale;
      for (int j = tid; j < a.k; j += nt) {
        const int to = a.slot_row[(size_t)r * a.k + j];
        if (to >= a.out_rows || to < -1) raise_error(a.err, kErrIndex);
        else if (to >= 0) a.scale[to] = s.scale;
      }
    }
  }
}

// Codes that exist already, dispatched: a token's codes and scale to every row
// that it was sent to.  One block per token at a time.
__global__ void __launch_bounds__(128)
    k_scatter_codes(const uint4 *__restrict__ xq, const float *__restrict__ scale,
                    const int32_t *__restrict__ slot_row, int T, int k, int row_vecs, int out_rows,
                    uint4 *__restrict__ out, float *__restrict__ out_scale, uint32_t *err) {
  grid_dependency();  // the previous grid is complete; the next may launch
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const int32_t *to_row = slot_row + (size_t)t * k;
    for (int v = threadIdx.x; v < row_vecs; v += blockDim.x) {
      const uint4 u = xq[(size_t)t * row_vecs + v];
      for (int j = 0; j < k; ++j) {
        const int to = to_row[j];
        if (to >= 0 && to < out_rows) out[(size_t)to * row_vecs + v] = u;
      }
    }
    if ((int)threadIdx.x < k) {
      const int to = to_row[threadIdx.x];
      if (to >= out_rows || to < -1) raise_error(err, kErrIndex);
      else if (to >= 0) out_scale[to] = scale[t];
    }
  }
}

template <typename T>
cudaError_t run_rows(const RowsArgs &a, cudaStream_t s) {
  const int nvec = a.K / Vec<T>::N;
  const int vpt = nvec <= 128 ? 1 : (nvec <= 1024 ? 2 : (nvec <= 2048 ? 4 : 0));
  const int nt = vpt ? ((nvec + vpt - 1) / vpt + 31) / 32 * 32 : 512;
  const int grid = std::min(a.rows, 148 * std::max(1, 2048 / nt));
  if (vpt == 1) launch_k(k_quantize_rows<T, 1>, grid, nt, 0, s, a);
  else if (vpt == 2) launch_k(k_quantize_rows<T, 2>, grid, nt, 0, s, a);
  else if (vpt == 4) launch_k(k_quantize_rows<T, 4>, grid, nt, 0, s, a);
  else launch_k(k_quantize_rows<T, 0>, grid, nt, 0, s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_int8(int G, int K, int N, const void *W, int8_t *Wq, float *scale,
                                 cudaStream_t s) {
  if ((long long)G * K * N == 0) return cudaSuccess;
  const dim3 grid((N + kCols - 1) / kCols, G);
  launch_k(k_quantize_int8, grid, 256, 0, s, static_cast<const __nv_bfloat16 *>(W), K, N, Wq,
           scale);
  return cudaGetLastError();
}

cudaError_t launch_scatter_codes(const int8_t *xq, const float *scale, const int32_t *slot_row,
                                 int T, int k, int K, int out_rows, int8_t *out, float *out_scale,
                                 uint32_t *err, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  launch_k(k_scatter_codes, std::min(T, 148 * 16), 128, 0, s, reinterpret_cast<const uint4 *>(xq),
           scale, slot_row, T, k, K / 16, out_rows, reinterpret_cast<uint4 *>(out), out_scale, err);
  return cudaGetLastError();
}

cudaError_t launch_quantize_rows(int dtype, const void *x, const int32_t *n_rows, int rows, int K,
                                 int8_t *xq, float *scale, uint32_t *err, cudaStream_t s,
                                 const int32_t *slot_row, int k, int out_rows, int8_t *own,
                                 float *own_scale) {
  if (rows <= 0) return cudaSuccess;
  const RowsArgs a{x, n_rows, slot_row, rows, K, k, out_rows, xq, scale, own, own_scale, err};
  return dtype == MOE_F32 ? run_rows<float>(a, s) : run_rows<__nv_bfloat16>(a, s);
}

}  // namespace moe
