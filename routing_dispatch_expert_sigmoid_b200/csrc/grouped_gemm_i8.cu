// Grouped products of int8 codes (moe_gemm_int8): tcgen05.mma kind::i8.
//
//   acc[r, n] = sum_k a[r, k] * b[g][n, k]            exact, int32
//   y[r, n]   = acc * (row_scale[r] * col_scale[g, n])  fp32
//   plain:  out = y        SwiGLU: out = silu(y of W1) * (y of W3)
// Rows r of group g are offsets[g] .. offsets[g+1]-1; without offsets all rows
// are one group.  Codes of both operands are K-contiguous, so both are K-major
// operands: a k-block of 128 codes is one 128-byte swizzle span.  The sums are
// exact in int32 (|acc| <= 128 * 128 * K, K <= 131056), so their order is free:
// splitting K over CTAs changes no bit of the result.
//
// Two engines, both warp-specialised (one TMA producer thread, one MMA thread,
// epilogue warps), persistent, accumulators double-buffered in tensor memory,
// every mbarrier wait bounded, no TMA multicast:
//
//   pair  CTA pairs (cta_group::2), tiles of 256 rows x 256 accumulator columns
//         (SwiGLU: 128 columns of W1 beside the same 128 of W3): for groups of
//         hundreds of rows, bound by the tensor cores.  Each CTA streams 32 KB
//         per k-block for 4 MMAs of M=256, N=256, K=32.  16381 rows in 8
//         groups, 14336 -> 4096: 690-720 us, 2.7-2.8 POP/s (the power limit;
//         bf16 sustains half of it).
//   swap  single CTAs, the weights as the MMA's M (128 columns) and the rows
//         as its N (16 .. 128): for groups of few rows, bound by the stream of
//         weights from HBM.  A stage holds two code tiles (SwiGLU: W1 and W3;
//         plain: two k-blocks) and the rows' codes.  When there are fewer tiles
//         than SMs, K is split over a cluster of 2 or 4 CTAs, whose int32
//         partial sums meet through distributed shared memory.  128 rows in 8
//         groups, 4096 -> 2 x 14336: 154 us for 0.94 GB, 6.1 TB/s.
#include <algorithm>

#include "gemm_i8.cuh"

namespace moe {
namespace tc {
namespace {

constexpr int kB = 128;  // K per k-block: one 128-byte swizzle span of codes

// kind::i8 instruction descriptor: int32 accumulator (bits 4-5 = 2), A and B
// signed (1 at bits 7-9 and 10-12), both K-major, N >> 3 at bit 17, M >> 4 at
// bit 24; wrapping (no saturation).
__host__ __device__ constexpr uint32_t instr_desc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct ParamsI8 {
  const int32_t *offsets;  // [G+1] or nullptr: one group of fixed_rows rows
  int G, fixed_rows, rows_cap, K, N;
  void *out;               // [rows_cap, N], bf16 or fp32
  const float *row_scale;  // [rows_cap]
  const float *scale1, *scale3;  // [G, N]
  int out_bf16;
  uint32_t *err;
  uint64_t wait_limit_ns;
  // swap engine
  int nt;          // rows per tile, at most (32, 64 or 128)
  int stages;      // ring depth
  int split;       // CTAs of a cluster that share a tile's K
};

// The accumulator value of a tcgen05.ld register as fp32.
__device__ __forceinline__ float acc_f32(float bits) {
  return __int2float_rn(__float_as_int(bits));
}

// 32 floats from shared memory, the same for every lane.
__device__ __forceinline__ void load32(const float *s, float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 f = *reinterpret_cast<const float4 *>(s + 4 * q);
    v[4 * q] = f.x;
    v[4 * q + 1] = f.y;
    v[4 * q + 2] = f.z;
    v[4 * q + 3] = f.w;
  }
}

// One warp, lane = row: 32 columns col .. of rows row0 + lane (rows from
// row_end on are not written), through the warp's staging buffer (32 rows of 64
// bytes) so that stores are whole 64-byte row segments.  A row's 16-byte pieces
// are turned by half its number, which keeps both the writes (8 rows, the same
// piece) and the reads (2 rows, all pieces) free of bank conflicts.
constexpr uint32_t kStageWarpBytes = 32 * 64;
__device__ __forceinline__ uint32_t *stage_at(uint32_t *st, int row, int piece) {
  return st + row * 16 + 4 * (piece ^ ((row >> 1) & 3));
}
__device__ __forceinline__ void store_rows(const float (&v)[32], uint32_t *st, int lane, int row0,
                                           int row_end, int col, int N, void *out, bool bf16) {
  if (bf16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[q * 8 + 2 * i], v[q * 8 + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b2);
      }
      *reinterpret_cast<uint4 *>(stage_at(st, lane, q)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 8 rows x 64 bytes per instruction
      const int r = i * 8 + (lane >> 2), q = lane & 3;
      const int grow = row0 + r, gcol = col + q * 8;
      const uint4 val = *reinterpret_cast<const uint4 *>(stage_at(st, r, q));
      if (grow < row_end && gcol < N)
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + (size_t)grow * N + gcol) =
            val;
    }
    __syncwarp();
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4 *>(stage_at(st, lane, q)) =
          make_float4(v[16 * h + 4 * q], v[16 * h + 4 * q + 1], v[16 * h + 4 * q + 2],
                      v[16 * h + 4 * q + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2), q = lane & 3;
      const int grow = row0 + r, gcol = col + 16 * h + q * 4;
      const uint4 val = *reinterpret_cast<const uint4 *>(stage_at(st, r, q));
      if (grow < row_end && gcol < N)
        *reinterpret_cast<uint4 *>(static_cast<float *>(out) + (size_t)grow * N + gcol) = val;
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// CTA pairs
// ---------------------------------------------------------------------------
constexpr int kPairRows = 256;
constexpr int kPairEpiWarps = 8;  // two per quarter of the tensor memory's lanes
constexpr int kPairThreads = 32 * (2 + kPairEpiWarps);

template <bool SWIGLU, int KPS>
struct PairI8 {
  static constexpr int BN = SWIGLU ? 128 : 256;  // output columns per tile
  static constexpr uint32_t kABytes = 128 * kB;  // this CTA's 128 rows
  static constexpr uint32_t kKbBytes = 2 * kABytes;
  static constexpr int kKbPerStage = KPS;  // k-blocks of a ring stage
  static constexpr uint32_t kStageBytes = kKbPerStage * kKbBytes;
  static constexpr int kStages = 6 / kKbPerStage;
  static constexpr uint32_t kRingBytes = kStages * kStageBytes;
  static constexpr uint32_t kAccCols = 256, kTmemCols = 512;
  static constexpr uint32_t kIdesc = instr_desc_i8(kPairRows, 256);
  // per epilogue warp: the output staging, and its 128 columns' scales
  static constexpr uint32_t kEpiBytes = kPairEpiWarps * (kStageWarpBytes + 512);
  static constexpr size_t kSmemFixed = 1024 + kRingBytes + 256 + kEpiBytes;
  static_assert(kSmemFixed + 8 * (kMaxGroups + 1) <= 232448, "shared memory of a CTA");
};

template <bool SWIGLU, int KPS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_gemm_i8_pair(const __grid_constant__ CUtensorMap tmA,   // codes [rows_cap, K]
                   const __grid_constant__ CUtensorMap tmB1,  // codes [G, N, K]
                   const __grid_constant__ CUtensorMap tmB3, const ParamsI8 p) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using S = PairI8<SWIGLU, KPS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(ring + S::kRingBytes);
  // bars: full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S::kStages + 5);
  int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
  uint32_t *s_epi = reinterpret_cast<uint32_t *>(ring + S::kRingBytes + 256);
  int32_t *s_off = reinterpret_cast<int32_t *>(ring + S::kRingBytes + 256 + S::kEpiBytes);
  int32_t *s_tstart = s_off + (p.G + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + S::kStages);
  const uint32_t accf0 = smem_addr(bars + 2 * S::kStages);
  const uint32_t acce0 = smem_addr(bars + 2 * S::kStages + 2);
  const uint32_t drain = smem_addr(bars + 2 * S::kStages + 4);
  // A pair stops only on the long limit: its CTAs complete copies on each
  // other's barriers, so one CTA stopping early must not outrun its peer.
  const Ctl ctl{abort_flag, p.err, kWaitLimitNs};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);   // the leader's arrive.expect_tx (both CTAs' bytes)
      mbar_init(empty0 + 8 * s, 1);  // the leader's multicast commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);                  // the leader's multicast commit
      mbar_init(acce0 + 8 * b, 2 * kPairEpiWarps);  // both CTAs' warps (leader's copy is used)
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB1);
    if (SWIGLU) prefetch_tmap(&tmB3);
  }
  if (warp == 1) tmem_alloc_pair(smem_addr(tmem_slot), S::kTmemCols);
  __syncthreads();
  const int col_tiles = (p.N + S::BN - 1) / S::BN;
  const int total = build_tiles(p.offsets, p.G, p.fixed_rows, p.rows_cap, kPairRows,
                                col_tiles, s_off, s_tstart, abort_flag, p.err);
  if (warp == 1) tmem_relinquish_pair();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int num_kb = (p.K + kB - 1) / kB;
  const uint32_t leader_full0 = mapa_shared(full0, 0);
  const uint32_t leader_acce0 = mapa_shared(acce0, 0);

  if (warp == 0) {
    // ------------------------------------------------------------ producers (both CTAs)
    if (lane == 0) {
      int s = 0, issued = 0, cursor = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        const Tile t = tile_at(tile, kPairRows, p.G, s_off, s_tstart, cursor);
        const int row = t.row0 + (int)rank * 128;
        const CUtensorMap *mb = (SWIGLU && rank == 1) ? &tmB3 : &tmB1;
        const int col = t.c * S::BN + (SWIGLU ? 0 : (int)rank * 128);
        for (int kb0 = 0; kb0 < num_kb; kb0 += S::kKbPerStage) {
          if (!wait(empty0 + 8 * s, ph ^ 1, ctl)) {
            ok = false;
            break;
          }
          const int nk = min(S::kKbPerStage, num_kb - kb0);
          const uint32_t lfb = leader_full0 + 8 * s;
          if (rank == 0) mbar_expect_tx(full0 + 8 * s, 2 * S::kKbBytes * (uint32_t)nk);
          for (int h = 0; h < nk; ++h) {
            const uint32_t st = smem_addr(ring + s * S::kStageBytes + h * S::kKbBytes);
            tma_load_2d_pair(st, &tmA, lfb, (kb0 + h) * kB, row);
            tma_load_3d_pair(st + S::kABytes, mb, lfb, (kb0 + h) * kB, col, t.g);
          }
          ++issued;
          if (++s == S::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok && issued > 0) {
        // Stopped early.  The leader waits for the stages it armed; both CTAs'
        // copies complete there.  The peer gives its copies a moment to land.
        if (rank == 0) {
          for (int q = 0; q < S::kStages && q < issued; ++q) {
            int st_i = s - 1 - q;
            uint32_t par = ph;
            if (st_i < 0) {
              st_i += S::kStages;
              par ^= 1;
            }
            wait_drain(full0 + 8 * st_i, par, p.err);
          }
        } else {
          const uint64_t t0 = global_timer();
          while (global_timer() - t0 < 2000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && lane == 0) {
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true, any = false;
      const uint64_t a_d0 = smem_desc(smem_addr(ring), 16, 1024);
      constexpr uint32_t kStageStep = S::kStageBytes >> 4, kKbStep = S::kKbBytes >> 4;
      constexpr uint32_t kBStep = S::kABytes >> 4, kStep = 32 >> 4;  // a K step of 32 codes
      for (int tile = pair; tile < total && ok; tile += npairs) {
        if (!wait(acce0 + 8 * buf, acc_ph ^ 1, ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * S::kAccCols;
        for (int kb0 = 0; kb0 < num_kb; kb0 += S::kKbPerStage) {
          if (!wait(full0 + 8 * s, ph, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int nk = min(S::kKbPerStage, num_kb - kb0);
          for (int h = 0; h < nk; ++h) {
            const uint64_t ad = a_d0 + s * kStageStep + h * kKbStep;
            const uint32_t acc0 = (kb0 + h) != 0;
#pragma unroll
            for (int kk = 0; kk < kB / 32; ++kk)
              umma_i8_pair(d_tmem, ad + kk * kStep, ad + kBStep + kk * kStep, S::kIdesc,
                           kk ? 1u : acc0);
          }
          any = true;
          umma_commit_pair_both(empty0 + 8 * s);
          if (++s == S::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit_pair_both(accf0 + 8 * buf);
        buf ^= 1;
        if (buf == 0) acc_ph ^= 1;
      }
      if (!ok && any) {
        umma_commit_pair_self(drain);
        wait_drain(drain, 0, p.err);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // lane = row of this CTA's 128, TMEM column = column of the tile; the two
    // warps of a quarter take half of the columns each
    const int quarter = warp & 3, half = (warp - 2) / 4;
    int buf = 0, cursor = 0;
    uint32_t acc_ph = 0;
    uint32_t *stg = s_epi + (warp - 2) * (kStageWarpBytes / 4);
    // the scales of this warp's columns wait in shared memory (SwiGLU: 64 of W1,
    // then 64 of W3), fetched before the accumulator is waited for
    float *s_scale = reinterpret_cast<float *>(s_epi) +
                     kPairEpiWarps * (kStageWarpBytes / 4) + (warp - 2) * 128;
    for (int tile = pair; tile < total; tile += npairs) {
      const Tile t = tile_at(tile, kPairRows, p.G, s_off, s_tstart, cursor);
      const int row0 = t.row0 + (int)rank * 128 + quarter * 32;
      const int row_end = t.row0 + t.nr;
      const float rs = row0 + lane < row_end ? p.row_scale[row0 + lane] : 0.f;
      {
        const bool third = SWIGLU && lane >= 16;
        const int c = t.c * S::BN + half * (S::BN / 2) + 4 * (SWIGLU ? lane & 15 : lane);
        const float *sc = (third ? p.scale3 : p.scale1) + (size_t)t.g * p.N;
        const float4 f = c < p.N ? __ldg(reinterpret_cast<const float4 *>(sc + c))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(s_scale + 4 * lane) = f;
        __syncwarp();
      }
      int ready = 0;
      if (lane == 0) ready = wait(accf0 + 8 * buf, acc_ph, ctl) ? 1 : 0;
      ready = __shfl_sync(0xffffffffu, ready, 0);
      if (!ready) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + buf * S::kAccCols + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < S::BN / 2; c0 += 32) {
        const int c = half * (S::BN / 2) + c0, col = t.c * S::BN + c;
        float v[32], sc[32];
        if (SWIGLU) {
          float u[32];
          tmem_ld32x2(tb + c, tb + S::BN + c, v, u);
          load32(s_scale + c0, sc);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = acc_f32(v[i]) * (rs * sc[i]);
          load32(s_scale + 64 + c0, sc);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = silu_times(v[i], acc_f32(u[i]) * (rs * sc[i]));
        } else {
          tmem_ld32(tb + c, v);
          load32(s_scale + c0, sc);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = acc_f32(v[i]) * (rs * sc[i]);
        }
        store_rows(v, stg, lane, row0, row_end, col, p.N, p.out, SWIGLU || p.out_bf16);
      }
      tc_fence_before();
      __syncwarp();  // (and the scales have been read)
      if (lane == 0) {
        if (rank == 0)
          mbar_arrive(acce0 + 8 * buf);
        else
          mbar_arrive_cluster(leader_acce0 + 8 * buf);
      }
      buf ^= 1;
      if (buf == 0) acc_ph ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer's MMAs or arrivals may reach it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, S::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Swap-AB: weights as M, rows as N
// ---------------------------------------------------------------------------
constexpr int kSwapThreads = 192;
constexpr int kSwapMaxStages = 8;
constexpr uint32_t kCodeBytes = 128 * kB;  // a code tile: 128 weight columns x one k-block
constexpr int kSwapRowWords = 36;
constexpr uint32_t kSwapEpiBytes = 4 * 32 * kSwapRowWords * 4;
// full, empty per stage; acc full and empty (2 each); drain; TMEM slot, abort
constexpr uint32_t kSwapBarBytes = 256;

template <bool SWIGLU>
struct SwapI8 {
  static constexpr int kKbPerStage = SWIGLU ? 1 : 2;  // two code tiles a stage either way
  static constexpr int kSpans = SWIGLU ? 2 : 1;       // accumulators: gate and up
};
__host__ __device__ constexpr uint32_t swap_stage_bytes(bool swiglu, int nt) {
  return 2 * kCodeBytes + (swiglu ? 1 : 2) * (uint32_t)nt * kB;
}
__host__ __device__ constexpr uint32_t swap_tmem_cols(bool swiglu, int nt) {
  return 2u * (swiglu ? 2 : 1) * nt;  // double-buffered; a power of two, 64 .. 512
}

template <bool SWIGLU, bool SPLIT>
__global__ void __launch_bounds__(kSwapThreads, 1)
    k_gemm_i8_swap(const __grid_constant__ CUtensorMap tmA,   // codes [rows_cap, K], 16-row boxes
                   const __grid_constant__ CUtensorMap tmW1,  // codes [G, N, K]
                   const __grid_constant__ CUtensorMap tmW3, const ParamsI8 p) {
  grid_dependency();  // the previous grid is complete; the next may launch
  using S = SwapI8<SWIGLU>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t stage_bytes = swap_stage_bytes(SWIGLU, p.nt);
  const uint32_t ring_bytes = p.stages * stage_bytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(ring + ring_bytes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kSwapMaxStages + 5);
  int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
  float *s_epi = reinterpret_cast<float *>(ring + ring_bytes + kSwapBarBytes);
  int32_t *s_off = reinterpret_cast<int32_t *>(ring + ring_bytes + kSwapBarBytes + kSwapEpiBytes);
  int32_t *s_tstart = s_off + (p.G + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + kSwapMaxStages);
  const uint32_t accf0 = smem_addr(bars + 2 * kSwapMaxStages);
  const uint32_t acce0 = smem_addr(bars + 2 * kSwapMaxStages + 2);
  const uint32_t drain = smem_addr(bars + 2 * kSwapMaxStages + 4);
  const Ctl ctl{abort_flag, p.err, p.wait_limit_ns};
  const uint32_t tmem_cols = swap_tmem_cols(SWIGLU, p.nt), acc_cols = S::kSpans * p.nt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmW1);
    if (SWIGLU) prefetch_tmap(&tmW3);
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), tmem_cols);
  __syncthreads();
  const int col_tiles = (p.N + 127) / 128;
  const int total = build_tiles(p.offsets, p.G, p.fixed_rows, p.rows_cap, p.nt, col_tiles,
                                s_off, s_tstart, abort_flag, p.err);
  if (warp == 1) tmem_relinquish();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // With SPLIT a cluster of p.split CTAs shares one tile, each with its part of
  // the k-blocks, and there is a cluster for every tile.
  const uint32_t rank = SPLIT ? cluster_ctarank() : 0;
  const int first = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int step = SPLIT ? gridDim.x / p.split : gridDim.x;
  const int num_kb = (p.K + kB - 1) / kB;
  const int kb_lo = SPLIT ? (int)((long long)num_kb * rank / p.split) : 0;
  const int kb_hi = SPLIT ? (int)((long long)num_kb * (rank + 1) / p.split) : num_kb;
  bool mine = false;  // SPLIT: this epilogue thread holds a finished accumulator

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0, cursor = 0;
      uint32_t ph = 0, issued_parity = 0, issued_mask = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = tile_at(tile, p.nt, p.G, s_off, s_tstart, cursor);
        const int boxes = (t.nr + 15) / 16;
        for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += S::kKbPerStage) {
          if (!wait(empty0 + 8 * s, ph ^ 1, ctl)) {
            ok = false;
            break;
          }
          const int nk = min(S::kKbPerStage, kb_hi - kb0);
          const uint32_t st = smem_addr(ring + s * stage_bytes), fb = full0 + 8 * s;
          mbar_expect_tx(fb, nk * (S::kSpans * kCodeBytes + boxes * 16 * kB));
          for (int h = 0; h < nk; ++h) {
            const int k = (kb0 + h) * kB;
            if (SWIGLU) {
              tma_load_3d(st, &tmW1, fb, k, t.c * 128, t.g);
              tma_load_3d(st + kCodeBytes, &tmW3, fb, k, t.c * 128, t.g);
            } else {
              tma_load_3d(st + h * kCodeBytes, &tmW1, fb, k, t.c * 128, t.g);
            }
            const uint32_t rows = st + 2 * kCodeBytes + h * p.nt * kB;
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(rows + b * 16 * kB, &tmA, fb, k, t.row0 + b * 16);
          }
          issued_mask |= 1u << s;
          issued_parity = (issued_parity & ~(1u << s)) | (ph << s);
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {  // stopped early: let the copies already issued land first
        for (int q = 0; q < p.stages; ++q)
          if ((issued_mask >> q) & 1u) wait_drain(full0 + 8 * q, (issued_parity >> q) & 1u, p.err);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int s = 0, buf = 0, cursor = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true, any = false;
      const uint64_t d0 = smem_desc(smem_addr(ring), 16, 1024);
      const uint32_t stage_step = stage_bytes >> 4, rows_step = (uint32_t)(p.nt * kB) >> 4;
      constexpr uint32_t kStep = 32 >> 4, kSpan = kCodeBytes >> 4;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = tile_at(tile, p.nt, p.G, s_off, s_tstart, cursor);
        // N: the rows rounded up to 16, above 32 to 32; rows behind the tile's
        // only reach accumulator columns that the epilogue does not read
        const int n = t.nr <= 16 ? 16 : (t.nr + 31) & ~31;
        const uint32_t idesc = instr_desc_i8(128, n);
        if (!wait(acce0 + 8 * buf, acc_ph ^ 1, ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * acc_cols;
        for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += S::kKbPerStage) {
          if (!wait(full0 + 8 * s, ph, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t sd = d0 + s * stage_step;
          const int nk = min(S::kKbPerStage, kb_hi - kb0);
          for (int h = 0; h < nk; ++h) {
            const uint64_t rd = sd + 2 * kSpan + h * rows_step;
            const uint32_t acc0 = (kb0 + h) != kb_lo;
#pragma unroll
            for (int kk = 0; kk < kB / 32; ++kk) {
              const uint32_t acc = kk ? 1u : acc0;
              umma_i8(d_tmem, sd + h * kSpan + kk * kStep, rd + kk * kStep, idesc, acc);
              if (SWIGLU)
                umma_i8(d_tmem + p.nt, sd + kSpan + kk * kStep, rd + kk * kStep, idesc, acc);
            }
          }
          any = true;
          umma_commit(empty0 + 8 * s);
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(accf0 + 8 * buf);
        buf ^= 1;
        if (buf == 0) acc_ph ^= 1;
      }
      if (!ok && any) {
        umma_commit(drain);
        wait_drain(drain, 0, p.err);
      }
    }
    __syncwarp();
  } else if (SPLIT) {
    int ready = 0;
    if (first < total) {
      if (lane == 0) ready = wait(accf0, 0, ctl) ? 1 : 0;
      ready = __shfl_sync(0xffffffffu, ready, 0);
    }
    mine = ready;
  } else {
    // ------------------------------------------------------------ epilogue
    // TMEM lane = weight column, TMEM column = row of the tile; transposed
    // through shared memory into row-major output
    const int quarter = warp & 3;
    int buf = 0, cursor = 0;
    uint32_t acc_ph = 0;
    float *stg = s_epi + (warp - 2) * 32 * kSwapRowWords;
    for (int tile = first; tile < total; tile += step) {
      const Tile t = tile_at(tile, p.nt, p.G, s_off, s_tstart, cursor);
      const int col0 = t.c * 128 + quarter * 32, col = col0 + lane;
      float sc1 = 0.f, sc3 = 0.f;
      if (col < p.N) {
        sc1 = p.scale1[(size_t)t.g * p.N + col];
        if (SWIGLU) sc3 = p.scale3[(size_t)t.g * p.N + col];
      }
      int ready = 0;
      if (lane == 0) ready = wait(accf0 + 8 * buf, acc_ph, ctl) ? 1 : 0;
      ready = __shfl_sync(0xffffffffu, ready, 0);
      if (!ready) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + buf * acc_cols + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
      for (int j0 = 0; j0 < t.nr; j0 += 32) {
        const float rs = j0 + lane < t.nr ? p.row_scale[t.row0 + j0 + lane] : 0.f;
        float v[32];
        if (SWIGLU) {
          float u[32];
          tmem_ld32x2(tb + j0, tb + p.nt + j0, v, u);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float r = __shfl_sync(0xffffffffu, rs, j);
            v[j] = silu_times(acc_f32(v[j]) * (r * sc1), acc_f32(u[j]) * (r * sc3));
          }
        } else {
          tmem_ld32(tb + j0, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = acc_f32(v[j]) * (__shfl_sync(0xffffffffu, rs, j) * sc1);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) stg[j * kSwapRowWords + lane] = v[j];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // 4 rows per step, 4 columns a lane
          const int j = i * 4 + (lane >> 3), q = lane & 7;
          const int gcol = col0 + q * 4;
          const float4 f = *reinterpret_cast<const float4 *>(stg + j * kSwapRowWords + 4 * q);
          if (j0 + j < t.nr && gcol < p.N) {
            const size_t at = (size_t)(t.row0 + j0 + j) * p.N + gcol;
            if (SWIGLU || p.out_bf16) {
              const __nv_bfloat162 lo = __floats2bfloat162_rn(f.x, f.y);
              const __nv_bfloat162 hi = __floats2bfloat162_rn(f.z, f.w);
              *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                  make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                             *reinterpret_cast<const uint32_t *>(&hi));
            } else {
              *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = f;
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce0 + 8 * buf);
      buf ^= 1;
      if (buf == 0) acc_ph ^= 1;
    }
  }

  if constexpr (SPLIT) {
    // The partial sums of a tile: every CTA sends each of its 128 columns to
    // the CTA that owns it (128 / split columns each), which adds the parts
    // and writes the outputs.  The parts lie where the rings were: the first
    // cluster barrier says that every CTA's MMAs have read theirs.
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    const int width = 128 / p.split;
    int32_t *part = reinterpret_cast<int32_t *>(ring);  // [src][span][row][width]
    int cursor = 0;
    Tile t{0, 0, 0, 0};
    if (first < total) t = tile_at(first, p.nt, p.G, s_off, s_tstart, cursor);
    if (mine) {
      tc_fence_after();
      const int quarter = warp & 3, c = quarter * 32 + lane;
      const uint32_t tb = tmem_base + ((uint32_t)(quarter * 32) << 16);
      const uint32_t to = mapa_shared(smem_addr(part), c / width);
#pragma unroll 1
      for (int sp = 0; sp < S::kSpans; ++sp) {
#pragma unroll 1
        for (int j0 = 0; j0 < t.nr; j0 += 32) {
          float v[32];
          tmem_ld32(tb + sp * p.nt + j0, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j0 + j < t.nr) {
              const uint32_t at =
                  ((((uint32_t)rank * S::kSpans + sp) * t.nr + j0 + j) * width + c % width) * 4;
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + at),
                           "r"(__float_as_uint(v[j]))
                           : "memory");
            }
          }
        }
      }
      tc_fence_before();
    }
    cluster_sync_all();
    // An aborted CTA's parts are missing: the device error word says so, and
    // the sums that need them are not meaningful.
    const int col0 = t.c * 128 + (int)rank * width;
    for (int i = threadIdx.x; i < t.nr * width; i += kSwapThreads) {
      const int j = i / width, c = i - j * width;
      if (col0 + c >= p.N) continue;
      int sum[S::kSpans];
#pragma unroll
      for (int sp = 0; sp < S::kSpans; ++sp) {
        sum[sp] = 0;
        for (int q = 0; q < p.split; ++q)
          sum[sp] += part[((q * S::kSpans + sp) * t.nr + j) * width + c];
      }
      const float r = p.row_scale[t.row0 + j];
      const size_t sc = (size_t)t.g * p.N + col0 + c;
      float y = __int2float_rn(sum[0]) * (r * p.scale1[sc]);
      if constexpr (SWIGLU)
        y = silu_times(y, __int2float_rn(sum[S::kSpans - 1]) * (r * p.scale3[sc]));
      const size_t at = (size_t)(t.row0 + j) * p.N + col0 + c;
      if (SWIGLU || p.out_bf16)
        static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
      else
        static_cast<float *>(p.out)[at] = y;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// 2-D map over codes [rows, K], box 128 (K) x box_rows, 128-byte swizzle.
bool make_map_rows_i8(CUtensorMap *m, const void *q, int rows, int K, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {(cuuint32_t)kB, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// 3-D map over codes [G, N, K], box 128 (K) x 128 (N) x 1, 128-byte swizzle.
bool make_map_codes_i8(CUtensorMap *m, const void *q, int G, int N, int K) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)G};
  cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)N * K};
  cuuint32_t box[3] = {(cuuint32_t)kB, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool SWIGLU, int KPS>
cudaError_t launch_i8_pair_kps(const Int8Gemm &a, cudaStream_t s) {
  using S = PairI8<SWIGLU, KPS>;
  CUtensorMap ma, mb1, mb3;
  if (!make_map_rows_i8(&ma, a.A, a.rows_cap, a.K, 128) ||
      !make_map_codes_i8(&mb1, a.B1, a.G, a.N, a.K) ||
      !make_map_codes_i8(&mb3, SWIGLU ? a.B3 : a.B1, a.G, a.N, a.K))
    return cudaErrorInvalidValue;
  const size_t smem = S::kSmemFixed + sizeof(int32_t) * 2 * (size_t)(a.G + 1);
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = set_smem_once(attr_set, k_gemm_i8_pair<SWIGLU, KPS>,
                                    S::kSmemFixed + sizeof(int32_t) * 2 * (kMaxGroups + 1)))
    return e;
  ParamsI8 p{a.offsets, a.G, a.fixed_rows, a.rows_cap, a.K, a.N, a.out, a.row_scale, a.s1, a.s3,
             a.out_bf16, a.err, kWaitLimitNs, 0, 0, 1};
  const long long max_tiles =
      (long long)((a.rows_cap + kPairRows - 1) / kPairRows + (a.offsets ? a.G : 0)) *
      ((a.N + S::BN - 1) / S::BN);
  const long long pairs = std::max<long long>(1, std::min<long long>(sm_count() / 2, max_tiles));
  launch_k(k_gemm_i8_pair<SWIGLU, KPS>, (int)(2 * pairs), kPairThreads, smem, s, ma, mb1, mb3, p);
  return cudaGetLastError();
}

// Two k-blocks per ring stage for long, even K: half the barrier round trips a
// byte.  Call by call, one k-block against two: 16384 x 4096 -> 2 x 14336 of 8
// experts 1538 and 1366 us, 131072 x 2048 -> 2 x 768 of 128 345 and 333, but
// 65536 x 2880 (23 blocks) -> 2 x 720 of 512 527 and 583; no difference for
// fewer than 16 blocks.
template <bool SWIGLU>
cudaError_t launch_i8_pair(const Int8Gemm &a, cudaStream_t s) {
  const int num_kb = (a.K + kB - 1) / kB;
  return num_kb >= 16 && num_kb % 2 == 0 ? launch_i8_pair_kps<SWIGLU, 2>(a, s)
                                         : launch_i8_pair_kps<SWIGLU, 1>(a, s);
}

template <bool SWIGLU>
cudaError_t launch_i8_swap(const Int8Gemm &a, cudaStream_t s) {
  CUtensorMap ma, mw1, mw3;
  if (!make_map_rows_i8(&ma, a.A, a.rows_cap, a.K, 16) ||
      !make_map_codes_i8(&mw1, a.B1, a.G, a.N, a.K) ||
      !make_map_codes_i8(&mw3, SWIGLU ? a.B3 : a.B1, a.G, a.N, a.K))
    return cudaErrorInvalidValue;
  constexpr size_t kFixed = 1024 + kSwapBarBytes + kSwapEpiBytes;
  constexpr size_t kLimit = 232448;
  const size_t tables = sizeof(int32_t) * 2 * (size_t)(a.G + 1);
  // rows per tile: twice the average group, so that most groups are one tile
  // and their weights are read once
  const int avg = (a.rows_cap + a.G - 1) / a.G;
  int nt = 32;  // the epilogue reads 32 accumulator columns at a time
  while (nt < 128 && nt < (a.offsets ? 2 * avg : avg)) nt *= 2;
  const uint32_t stage = swap_stage_bytes(SWIGLU, nt);
  const int stages =
      std::min<int>(kSwapMaxStages, (int)((kLimit - kFixed - tables) / stage));
  const int sms = sm_count();
  const long long max_tiles = (long long)((a.rows_cap + nt - 1) / nt + (a.offsets ? a.G - 1 : 0)) *
                              ((a.N + 127) / 128);
  // K over a cluster when the tiles leave SMs idle; at least four k-blocks each
  const int num_kb = (a.K + kB - 1) / kB;
  int split = 1;
  // (not eight: clusters of eight CTAs that fill their SMs do not all fit at
  // once, 18 us against 11 us with four for one row, 7168 -> 2048)
  while (split < 4 && 2 * split * max_tiles <= sms && num_kb >= 8 * split) split *= 2;
  // the parts of a split tile lie in the ring: 512 bytes a row and span
  while (split > 1 && (size_t)(SWIGLU ? 2 : 1) * nt * 512 > (size_t)stages * stage) split /= 2;
  ParamsI8 p{a.offsets, a.G, a.fixed_rows, a.rows_cap, a.K, a.N, a.out, a.row_scale, a.s1, a.s3,
             a.out_bf16, a.err, pipeline_wait_limit_ns(), nt, stages, split};
  const size_t smem = kFixed + tables + (size_t)stages * stage;
  if (split > 1) {
    static std::atomic<bool> attr_set[64];
    if (cudaError_t e = set_smem_once(attr_set, k_gemm_i8_swap<SWIGLU, true>, kLimit)) return e;
    launch_cluster(k_gemm_i8_swap<SWIGLU, true>, (int)(max_tiles * split), kSwapThreads, split,
                   smem, s, ma, mw1, mw3, p);
  } else {
    static std::atomic<bool> attr_set[64];
    if (cudaError_t e = set_smem_once(attr_set, k_gemm_i8_swap<SWIGLU, false>, kLimit)) return e;
    const int grid = (int)std::max<long long>(1, std::min<long long>(sms, max_tiles));
    launch_k(k_gemm_i8_swap<SWIGLU, false>, grid, kSwapThreads, smem, s, ma, mw1, mw3, p);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace tc

// MOE_INT8_ENGINE=swap|pair|gemv forces one engine (gemv where it fits).
bool use_gemv_i8(const Int8Gemm &a) {
  const char *env = getenv("MOE_INT8_ENGINE");
  return (!env || (env[0] != 's' && env[0] != 'p')) && gemv_i8_fits(a);
}

cudaError_t launch_gemm_i8(bool swiglu, const Int8Gemm &a, cudaStream_t s) {
  if (a.rows_cap <= 0) return cudaSuccess;
  if (a.G < 1 || a.G > tc::kMaxGroups || a.N % 8 || a.K % 16) return cudaErrorInvalidValue;
  if (use_gemv_i8(a)) return launch_gemv_i8(swiglu, -1, a, s);  // a few rows: no tensor cores
  // Groups of up to 96 rows on average stream their weights (swap); larger
  // ones fill 256-row tiles (pair).  On codes, swap against pair, us: 8 groups
  // 4096 -> 2 x 14336 of 96 rows 168 and 202, of 128 175 and 204, of 192 309 and
  // 208; 32 groups 2048 -> 2048 of 64 rows 36 and 37, of 96 46 and 37.  The rule
  // looks at the rows alone: one matrix is few tiles, where swap splits K and pair
  // does not, 7168 -> 2048 of 16 rows 12 and 22, 64 20 and 23, 96 25 and 23, 128 31
  // and 23, 512 45 and 23; 7168 -> 2 x 2048 of 64 rows 33 and 25, 96 40 and 24;
  // 2048 -> 7168 of 64 25 and 12, 96 29 and 12.  Pair takes one time there from 4 to
  // 1024 rows, that of the one tile a pair of CTAs has.
  const char *env = getenv("MOE_INT8_ENGINE");
  bool swap = (a.rows_cap + a.G - 1) / a.G <= 96;
  if (env && env[0] == 's') swap = true;
  if (env && env[0] == 'p') swap = false;
  if (swap) return swiglu ? tc::launch_i8_swap<true>(a, s) : tc::launch_i8_swap<false>(a, s);
  return swiglu ? tc::launch_i8_pair<true>(a, s) : tc::launch_i8_pair<false>(a, s);
}

}  // namespace moe
