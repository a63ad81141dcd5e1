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
// Rows (quantize_rows.cuh has the formulas): a warp or a block per row, the row
// in shared memory between the maximum and the codes, so it is read from HBM
// once: rows * K * (2 or 4) bytes in, rows * (K + 4) out, bound by HBM.  Rows
// longer than shared memory holds are read twice, the second time from L2.  With a
// slot table (the layer's dispatch) a token's codes go to every row that the
// token was sent to, so the expert-ordered rows are written in the same pass.
// bf16 rows: 131072 x 2048 145 us (5.5 TB/s; a copy reaches 6.45), 16384 x 14336
// 153 us; fp32 65536 x 2048 119 us (5.6 TB/s).  bf16 rows are bound by
// instructions, 13 a value.
#include <algorithm>

#include "quantize_rows.cuh"

namespace moe {
namespace {

constexpr int kCols = 32;
constexpr size_t kStagedLimit = 200u << 10;  // shared memory for the rows of a block

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

// The rows to do, checked.
__device__ __forceinline__ int row_count(const RowsArgs &a) {
  const int R = a.n_rows ? *a.n_rows : a.rows;
  if (R >= 0 && R <= a.rows) return R;
  if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrIndex);
  return 0;
}
// Vector v of row r as codes, to every place that it has.
template <typename T, bool SCATTER>
__device__ __forceinline__ void put(const RowsArgs &a, int r, int v, const uint4 &u,
                                    const i8::RowScale &s) {
  constexpr int N = Vec<T>::N;
  float f[N];
  uint32_t c[N / 4];
  Vec<T>::get(u, f);
  i8::codes<N>(f, s, c);
  const size_t at = (size_t)v * N;
  if constexpr (!SCATTER) {
    i8::store<N>(a.xq + (size_t)r * a.K + at, c);
  } else {
    if (a.own) i8::store<N>(a.own + (size_t)r * a.K + at, c);
    for (int j = 0; j < a.k; ++j) {
      const int to = a.slot_row[(size_t)r * a.k + j];
      if (to >= 0 && to < a.out_rows) i8::store<N>(a.xq + (size_t)to * a.K + at, c);
    }
  }
}
template <bool SCATTER>
__device__ __forceinline__ void put_scale(const RowsArgs &a, int r, float scale, int id, int n) {
  if constexpr (!SCATTER) {
    if (id == 0) a.scale[r] = scale;
  } else {
    if (id == 0 && a.own) a.own_scale[r] = scale;
    for (int j = id; j < a.k; j += n) {
      const int to = a.slot_row[(size_t)r * a.k + j];
      if (to >= a.out_rows || to < -1) raise_error(a.err, kErrIndex);
      else if (to >= 0) a.scale[to] = scale;
    }
  }
}

// blockDim.x threads share a row; blockDim.y rows at a time (more than one
// only with a warp per row).  A thread copies its vectors of the next row into
// its own places in shared memory with cp.async while it works on this one;
// nobody else reads them, so the row's maximum is the only thing its threads
// exchange.  STAGED false: rows too long for that, read twice from memory.
template <typename T, bool SCATTER, bool STAGED>
__global__ void __launch_bounds__(512) k_quantize_rows(const RowsArgs a) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using V = Vec<T>;
  extern __shared__ uint4 s_rows[];  // [blockDim.y][2][nvec]
  __shared__ uint32_t s_red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = a.K / V::N, R = row_count(a);
  if (nt > 32) {
    if (tid < 32) s_red[tid / 16][tid % 16] = 0;
    __syncthreads();
  }
  uint4 *const slots = s_rows + (size_t)threadIdx.y * 2 * nvec;
  const int step = gridDim.x * blockDim.y;
  auto issue = [&](int r, int which) {
    uint4 *const to = slots + (which ? nvec : 0);
    if constexpr (STAGED) {
      const uint4 *row = static_cast<const uint4 *>(a.x) + (size_t)r * nvec;
      if (r < R)
        for (int v = tid; v < nvec; v += nt) copy16(tc::smem_addr(to + v), row + v);
      copy_commit();
    }
  };
  int which = 0;
  const int r_first = blockIdx.x * blockDim.y + threadIdx.y;
  issue(r_first, 0);
  for (int r = r_first; r < R; r += step) {
    const uint4 *row = static_cast<const uint4 *>(a.x) + (size_t)r * nvec;
    if constexpr (STAGED) {
      issue(r + step, which ^ 1);
      copy_wait(1);
      row = slots + (which ? nvec : 0);
    }
    uint32_t bits = 0;
#pragma unroll 4
    for (int v = tid; v < nvec; v += nt) bits = V::peak(row[v], bits);
    uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(V::peak_value(bits)));
    if (nt > 32) {
      if (tid % 32 == 0) s_red[which][tid / 32] = top;
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, s_red[which][tid % 16]);
    }
    const i8::RowScale s = i8::row_scale(__uint_as_float(top));
#pragma unroll 2
    for (int v = tid; v < nvec; v += nt) put<T, SCATTER>(a, r, v, row[v], s);
    put_scale<SCATTER>(a, r, s.scale, tid, nt);
    which ^= 1;
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

template <typename T, bool SCATTER>
cudaError_t run_rows(const RowsArgs &a, cudaStream_t s) {
  const int nvec = a.K / Vec<T>::N;
  const size_t row_bytes = (size_t)nvec * 16;
  // Eight vectors a thread keep enough bytes in flight on an SM (two rows of
  // 128 bytes for each of its threads); with few rows, more threads a row.
  const auto warps_of = [](long long threads) { return (threads + 31) / 32 * 32; };
  long long nt = warps_of((nvec + 7) / 8);
  nt = std::max(nt, std::min(warps_of(nvec), warps_of(148 * 1024 / a.rows)));
  nt = std::max<long long>(32, std::min<long long>(nt, 512));
  const bool staged = 2 * row_bytes <= kStagedLimit;
  const int rows = nt == 32 && a.rows > 148 ? (int)std::min<size_t>(8, kStagedLimit / (2 * row_bytes)) : 1;
  const size_t smem = staged ? rows * 2 * row_bytes : 0;
  const int per_sm = std::max(1, std::min<int>((int)(1024 / (nt * rows)),
                                               staged ? (int)((220 << 10) / smem) : 2));
  const int grid = std::min((a.rows + rows - 1) / rows, 148 * per_sm);
  const dim3 block((unsigned)nt, rows);
  static std::atomic<bool> attr_set[64];
  if (staged) {
    if (cudaError_t e = tc::set_smem_once(attr_set, k_quantize_rows<T, SCATTER, true>,
                                          kStagedLimit))
      return e;
    launch_k(k_quantize_rows<T, SCATTER, true>, grid, block, smem, s, a);
  } else {
    launch_k(k_quantize_rows<T, SCATTER, false>, grid, block, smem, s, a);
  }
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
  if (slot_row)
    return dtype == MOE_F32 ? run_rows<float, true>(a, s) : run_rows<__nv_bfloat16, true>(a, s);
  return dtype == MOE_F32 ? run_rows<float, false>(a, s) : run_rows<__nv_bfloat16, false>(a, s);
}

}  // namespace moe
