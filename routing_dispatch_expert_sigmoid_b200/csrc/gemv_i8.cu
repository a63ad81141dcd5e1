// Int8 products of one or two rows (the formulas of grouped_gemm_i8.cu), or of
// about one row in each of a few groups: a decode step of a handful of tokens.
//
// The bound is the stream of weights from HBM, G*N*K bytes, and for small
// matrices the time to get it going: tiles of 128 columns leave most SMs
// without work, and a tensor-core pipeline takes longer to fill than the whole
// product.  So here every warp streams columns with plain 16-byte loads and
// multiplies them with dp4a (four codes an instruction, exact int32 sums, the
// same bits as the other engines); the rows' codes wait in shared memory, and
// with QUANT the block makes them itself from the activations, so that a
// product is one launch.  The block's first weights are already on their way
// while it does.
//
// A warp takes four streams of codes: four columns, or gate and up of two.
// `ksplit` of the eight warps share their columns and split K, so that the
// number of blocks suits the GPU; their parts meet in shared memory.
#include <algorithm>

#include "gemm_i8.cuh"
#include "quantize_rows.cuh"

namespace moe {
namespace tc {
namespace {

constexpr int kWarpsV = 8;
constexpr int kStreams = 4;
constexpr int kUnroll = 4;  // 16-byte loads of a stream in flight per lane
constexpr size_t kCodesLimit = 64u << 10;  // the rows' codes in shared memory

struct ParamsV {
  const int32_t *offsets;
  int G, fixed_rows, rows_cap, K, N;
  const void *x;            // QUANT: rows [rows_cap, K]; else their codes
  const float *row_scale;   // without QUANT
  const int8_t *W1, *W3;    // [G, N, K]
  const float *s1, *s3;     // [G, N]
  void *out;
  int out_bf16, ksplit;
  uint32_t *err;
};

__device__ __forceinline__ uint4 load_stream(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int acc) {
  acc = __dp4a((int)a.x, (int)b.x, acc);
  acc = __dp4a((int)a.y, (int)b.y, acc);
  acc = __dp4a((int)a.z, (int)b.z, acc);
  return __dp4a((int)a.w, (int)b.w, acc);
}

// R rows at a time; T: type of the rows with QUANT (int8_t: codes are given).
template <int R, typename T, bool SWIGLU>
__global__ void __launch_bounds__(kWarpsV * 32, 2) k_gemv_i8(const ParamsV p) {
  grid_dependency();  // the previous grid is complete; the next may launch
  constexpr bool QUANT = sizeof(T) > 1;
  constexpr int kCols = SWIGLU ? kStreams / 2 : kStreams;  // columns of a warp
  extern __shared__ uint4 s_x[];  // [R][K / 16], then the tile tables
  __shared__ int s_part[kWarpsV][kStreams * R];
  __shared__ float s_scale[R];
  __shared__ uint32_t s_peak[kWarpsV][R];
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int kvec = p.K / 16;
  int32_t *s_off = reinterpret_cast<int32_t *>(s_x + (size_t)R * kvec);
  int32_t *s_tstart = s_off + (p.G + 1);
  if (tid == 0) s_abort = 0;
  __syncthreads();
  const int block_cols = kCols * (kWarpsV / p.ksplit);
  const int col_tiles = (p.N + block_cols - 1) / block_cols;
  const int total = build_tiles(p.offsets, p.G, p.fixed_rows, p.rows_cap, R, col_tiles, s_off,
                                s_tstart, &s_abort, p.err);
  // this warp's part of K, in 16-byte vectors, and its columns of a tile
  const int per = (kvec + p.ksplit - 1) / p.ksplit, kpart = warp % p.ksplit;
  const int k_lo = min(kvec, kpart * per), k_hi = min(kvec, k_lo + per);
  int cursor = 0, held = -1;  // held: first row of the rows whose codes are in s_x
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const Tile t = tile_at(tile, R, p.G, s_off, s_tstart, cursor);
    const int col0 = t.c * block_cols + (warp / p.ksplit) * kCols;
    const int8_t *w[kStreams];
#pragma unroll
    for (int q = 0; q < kStreams; ++q) {
      // columns behind the last are read as the last and not written
      const int c = min(col0 + (SWIGLU ? q / 2 : q), p.N - 1);
      const int8_t *W = (SWIGLU && q % 2) ? p.W3 : p.W1;
      w[q] = W + ((size_t)t.g * p.N + c) * p.K;
    }
    uint4 u[kUnroll][kStreams];
    auto load = [&](int k) {
#pragma unroll
      for (int b = 0; b < kUnroll; ++b)
#pragma unroll
        for (int q = 0; q < kStreams; ++q) {
          const int v = k + b * 32 + lane;
          u[b][q] = make_uint4(0, 0, 0, 0);
          if (v < k_hi) u[b][q] = load_stream(w[q] + (size_t)v * 16);
        }
    };
    load(k_lo);

    if (held != t.row0) {
      __syncthreads();  // the last tile's codes have been read
      if constexpr (QUANT) {
        using V = Vec<T>;
        const int nvec = p.K / V::N;
        const uint4 *rows = static_cast<const uint4 *>(p.x) + (size_t)t.row0 * nvec;
        uint32_t bits[R];
#pragma unroll
        for (int r = 0; r < R; ++r) bits[r] = 0;
        for (int v = tid; v < nvec; v += kWarpsV * 32)
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (r < t.nr) bits[r] = V::peak(__ldg(rows + (size_t)r * nvec + v), bits[r]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t m =
              __reduce_max_sync(0xffffffffu, __float_as_uint(V::peak_value(bits[r])));
          if (lane == 0) s_peak[warp][r] = m;
        }
        __syncthreads();
#pragma unroll 1
        for (int r = 0; r < t.nr; ++r) {
          const uint32_t m = __reduce_max_sync(0xffffffffu, s_peak[lane % kWarpsV][r]);
          const i8::RowScale s = i8::row_scale(__uint_as_float(m));
          if (tid == 0) s_scale[r] = s.scale;
          int8_t *to = reinterpret_cast<int8_t *>(s_x + (size_t)r * kvec);
          for (int v = tid; v < nvec; v += kWarpsV * 32) {
            float f[V::N];
            uint32_t c[V::N / 4];
            V::get(__ldg(rows + (size_t)r * nvec + v), f);
            i8::codes<V::N>(f, s, c);
            i8::store<V::N>(to + (size_t)v * V::N, c);
          }
        }
      } else {
        const uint4 *rows = static_cast<const uint4 *>(p.x) + (size_t)t.row0 * kvec;
        for (int i = tid; i < t.nr * kvec; i += kWarpsV * 32) s_x[i] = __ldg(rows + i);
        if (tid < t.nr) s_scale[tid] = p.row_scale[t.row0 + tid];
      }
      __syncthreads();
      held = t.row0;
    }

    int acc[kStreams][R];
#pragma unroll
    for (int q = 0; q < kStreams; ++q)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[q][r] = 0;
    for (int k = k_lo; k < k_hi; k += kUnroll * 32) {
      if (k != k_lo) load(k);
#pragma unroll
      for (int b = 0; b < kUnroll; ++b) {
        const int v = k + b * 32 + lane;
        if (v < k_hi) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (r < t.nr) {
              const uint4 xv = s_x[(size_t)r * kvec + v];
#pragma unroll
              for (int q = 0; q < kStreams; ++q) acc[q][r] = dot16(u[b][q], xv, acc[q][r]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kStreams; ++q)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int sum = __reduce_add_sync(0xffffffffu, acc[q][r]);
        if (lane == 0) s_part[warp][q * R + r] = sum;
      }
    __syncthreads();
    // one output per thread: column of the block, row
    for (int i = tid; i < block_cols * t.nr; i += kWarpsV * 32) {
      const int c = i % block_cols, r = i / block_cols, col = t.c * block_cols + c;
      const int w0 = c / kCols * p.ksplit, cc = c % kCols;
      int a = 0, b = 0;
      for (int s = 0; s < p.ksplit; ++s) {
        if constexpr (SWIGLU) {
          a += s_part[w0 + s][2 * cc * R + r];
          b += s_part[w0 + s][(2 * cc + 1) * R + r];
        } else {
          a += s_part[w0 + s][cc * R + r];
        }
      }
      if (col < p.N) {
        const float rs = s_scale[r];
        const size_t sc = (size_t)t.g * p.N + col;
        float y = __int2float_rn(a) * (rs * p.s1[sc]);
        if constexpr (SWIGLU) y = silu_times(y, __int2float_rn(b) * (rs * p.s3[sc]));
        const size_t at = (size_t)(t.row0 + r) * p.N + col;
        if (SWIGLU || p.out_bf16)
          static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
        else
          static_cast<float *>(p.out)[at] = y;
      }
    }
    __syncthreads();  // s_part is written again by the next tile
  }
}

// Rows of a block's pass.  A group of more rows takes several passes.
int rows_of(const Int8Gemm &a) { return a.rows_cap == 1 ? 1 : 2; }

template <int R, typename T, bool SWIGLU>
cudaError_t run(const Int8Gemm &a, cudaStream_t s) {
  constexpr int kCols = SWIGLU ? kStreams / 2 : kStreams;
  // K is split as far as every block still runs at once (two an SM, 128
  // registers a thread for the loads in flight), into parts of at least two
  // loads per lane: one row 7168 -> 2048 in 256 blocks of eight columns, not in
  // 512 of four, of which some would run second
  const int groups = a.offsets ? std::min(a.G, a.rows_cap) : 1;
  int ksplit = 1;
  while (ksplit < kWarpsV && a.K >= 2048 * ksplit &&
         (long long)groups * a.N * 2 * ksplit <= 2LL * 148 * kWarpsV * kCols)
    ksplit *= 2;
  const int block_cols = kCols * (kWarpsV / ksplit);
  const long long tiles = (long long)(a.offsets ? groups + a.rows_cap / R : 1) *
                          ((a.N + block_cols - 1) / block_cols);
  const size_t smem = (size_t)R * a.K + sizeof(int32_t) * 2 * (size_t)(a.G + 1);
  const ParamsV p{a.offsets, a.G, a.fixed_rows, a.rows_cap, a.K, a.N, a.A, a.row_scale,
                  static_cast<const int8_t *>(a.B1), static_cast<const int8_t *>(a.B3), a.s1,
                  a.s3, a.out, a.out_bf16, ksplit, a.err};
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = set_smem_once(attr_set, k_gemv_i8<R, T, SWIGLU>,
                                    kCodesLimit + sizeof(int32_t) * 2 * (kMaxGroups + 1)))
    return e;
  const int grid = (int)std::max<long long>(1, std::min<long long>(tiles, 148 * 2));
  launch_k(k_gemv_i8<R, T, SWIGLU>, grid, kWarpsV * 32, smem, s, p);
  return cudaGetLastError();
}

template <typename T, bool SWIGLU>
cudaError_t run_rows(const Int8Gemm &a, cudaStream_t s) {
  return rows_of(a) == 1 ? run<1, T, SWIGLU>(a, s) : run<2, T, SWIGLU>(a, s);
}

}  // namespace
}  // namespace tc

// Measured against the swap engine, with the rows' quantisation, on weights that
// are not in L2: one row 7168 -> 2048 7.0 us against 13.1, 14336 -> 4096 14.8
// against 20.0, 4096 -> 2 x 14336 21.9 against 25.3 (18.2 at the measured copy
// rate); four rows 7168 -> 2048 16 against 13.4.  Groups: 2 rows of 8 experts
// 4096 -> 2 x 14336 39.7 against 52.5 (36.4), 8 rows of 8 137 against 153; 8
// rows of 256 experts 7168 -> 2 x 2048 52.4 against 50.9, 64 rows 294 against 278.
// The rule knows the rows and the groups, not how they fall.  One row in each of
// its groups, the sizes are even from 8 of 256 on (8 rows 55 against 53, 32 160
// against 161) and this kernel is ahead in smaller layers (32 of 128, 2048 -> 2 x
// 768, 30 against 34).  All rows in one group read its weights once for every two
// rows: 8 of 256 still 28 against 41 us, but 32 of 256 83 against 42, and 8 of 8
// 4096 -> 2 x 14336 56 against 30.
bool gemv_i8_fits(const Int8Gemm &a) {
  if (a.rows_cap > (a.offsets ? std::min(32, a.G) : 2)) return false;
  return (size_t)tc::rows_of(a) * a.K <= tc::kCodesLimit;
}

cudaError_t launch_gemv_i8(bool swiglu, int dtype, const Int8Gemm &a, cudaStream_t s) {
  if (a.rows_cap <= 0) return cudaSuccess;
  if (a.G < 1 || a.G > tc::kMaxGroups || a.N % 8 || a.K % 16) return cudaErrorInvalidValue;
  switch (dtype) {
    case MOE_F32: return swiglu ? tc::run_rows<float, true>(a, s) : tc::run_rows<float, false>(a, s);
    case MOE_BF16:
      return swiglu ? tc::run_rows<__nv_bfloat16, true>(a, s)
                    : tc::run_rows<__nv_bfloat16, false>(a, s);
    default: return swiglu ? tc::run_rows<int8_t, true>(a, s) : tc::run_rows<int8_t, false>(a, s);
  }
}

}  // namespace moe
