// General gating (MOE_GATE_SOFTMAX .. MOE_GATE_SIGMOID_RENORM) and the gradient
// of the combine weights, for every gating mode.
//
// Forward, per token with logits l[E] and k_t slots:
//   s_e = softmax(l)_e or sigmoid(l_e);  u_e = s_e + sel_bias_e
//   with n_groups > 1: a group's score is the sum of its group_score_topk
//   largest u; the topk_groups best groups stay
//   the k_t largest u among the experts that stay; w = scale * s (divided by
//   the sum of the selected s in the _RENORM modes)
// The order is that of the scores in 64 bits.  Without a bias u is increasing in
// l, so the logits themselves are compared.
//
// Forward and backward run one warp per token; lane l holds experts l, l+32,
// ... so rows are read in 128-byte lines.  The selection is bound by instructions
// (HBM would take T*E logits in, T*k indices and weights out), so it is made on
// one 32-bit word per expert: the key in 22-bit fixed point below the row's
// largest, above 1023 - expert.  One unsigned comparison then ranks two experts,
// no two words are equal, a lane sorts its own with plain minima and maxima, and
// a selection round is one warp reduction.  What the 22 bits and the fp32
// scores behind them may be off by is known; a token where two neighbours of the
// resulting order (or the last group kept and the first one dropped) are closer
// than that is selected again: without a bias on the fp32 logits' own bits, with
// one on scores in fp64; only the groups if they are close, and of the experts
// only those that may be among the k_t best.  For normal logits 0.1 to 1% of the
// tokens are.  A bias that leaves little of the scores (it all but cancels them,
// or holds finite values far beyond them, as masks of -1e9 do) sends every token
// there: 16384 x 256 (4 of 8 groups) 140 us for 24.5; masks of -inf cost 25.
// Against selecting everything on 64-bit words: 16384 x 128 (softmax, bias)
// 16.5 -> 12.0 us, 16384 x 256 (sigmoid, groups, bias) 44 -> 24.5, 8192 x 512
// (softmax, bias, top-16) 36 -> 21, 4096 x 1024 (top-32) 69 -> 27.  With the
// second selection over all experts, these took 13, 29, 27 and 57: the tokens
// are few, but the last of them is waited for.
//
// Backward, with g_j = scale * dL/dw_j of the selected slots:
//   renormalised: g_j <- (g_j - sum_i g_i n_i) / S,  S = sum of the selected s,
//   n_i = s_i / S;  then ds_j = g_j.  sigmoid: dl_j = ds_j s_j (1 - s_j);
//   softmax: dl_e = s_e (ds_e - sum_i ds_i s_i) for every e; its renormalised
//   form needs the selected logits alone, since the softmax over all experts
//   cancels: dl_j = n_j (g_j - sum_i g_i n_i).
// The selection and its bias get no gradient.  Only the MOE_GATE_SOFTMAX form
// reads whole rows of logits; the others read k logits and write the row.  Bound
// by HBM: 65536 x 512 (softmax) 55 us, 5.0 TB/s (with the fast exponential 52, but
// scores far below the largest then lose up to seven bits).
#include <limits.h>
#include <math.h>

#include "gating.cuh"

namespace moe {
namespace {

using gating::GatingArgs;
using gating::kFull;
using gating::warp_sum;

constexpr int kGateWarps = 4;  // tokens per CTA

// ---- ordered keys ----------------------------------------------------------
// fp64 keys as unsigned integers in their order (-0 as +0); 0 is no candidate.
typedef unsigned long long u64;
__device__ __forceinline__ u64 order64(double k) {
  u64 b = (u64)__double_as_longlong(k);
  const u64 sign = 0x8000000000000000ull;
  if (b == sign) b = 0;
  const u64 u = (b & sign) ? ~b : (b | sign);
  return u ? u : 1;
}
__device__ __forceinline__ u64 top64(u64 u) {
  const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(u >> 32));
  const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(u >> 32) == hi ? (uint32_t)u : 0u);
  return ((u64)hi << 32) | lo;
}
// An fp32 candidate: its ordered key above 1023 - expert, so that one unsigned
// comparison ranks by larger key, then lower index, and no two are equal.
__device__ __forceinline__ u64 candidate(float k, int e) {
  return ((u64)gating::order_key(k) << 32) | (uint32_t)(1023 - e);
}
__device__ __forceinline__ float key_of(uint32_t hi) {
  return __uint_as_float((hi & 0x80000000u) ? (hi & 0x7fffffffu) : ~hi);
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
template <typename R>
__device__ __forceinline__ R warp_sum_of(R v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
// sigmoid without overflow on either side (-inf gives 0).
template <typename R>
__device__ __forceinline__ R sigmoid_of(R v) {
  const R e = exp_of(v < R(0) ? v : -v);
  return (v < R(0) ? e : R(1)) / (R(1) + e);
}

// ---- candidates of a lane -------------------------------------------------------
// The larger of two first (32-bit words or 64-bit candidates).
template <typename U>
__device__ __forceinline__ void order2(U &a, U &b) {
  const U hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}
// The four largest of c[0 .. NPL), largest first (0: none); with BELOW those
// below `bound` only.  Sorted fours merge two and two: the larger ones of a list
// and the other reversed are the four largest of both, in bitonic order.
template <int NPL, bool BELOW, typename U>
__device__ __forceinline__ void best_four(const U (&c)[NPL], U bound, U (&h)[4]) {
#pragma unroll
  for (int i = 0; i < NPL; i += 4) {
    U f[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[q] = i + q < NPL ? c[i + q < NPL ? i + q : 0] : 0;
      if (BELOW && f[q] >= bound) f[q] = 0;
    }
    if (NPL > 1) order2(f[0], f[1]);
    if (NPL > 2) {
      order2(f[2], f[3]);
      order2(f[0], f[2]);
      order2(f[1], f[3]);
      order2(f[1], f[2]);
    }
    if (i == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = f[q];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = max(h[q], f[3 - q]);
      order2(h[0], h[2]);
      order2(h[1], h[3]);
      order2(h[0], h[1]);
      order2(h[2], h[3]);
    }
  }
}

// Lanes of a group when several share one: a power of two.
__device__ __forceinline__ int group_lanes(int n_groups) {
  int L = 1;
  while (2 * L * n_groups <= 32) L *= 2;
  return L;
}
// A logit as the selection sees it: NaN ranks as -inf.
__device__ __forceinline__ float clean(float v) { return fmaxf(v, -INFINITY); }

// A token's row, for the selections that look at it again.
struct Row {
  const float *l;
  u64 *s_u;       // [E] of this warp's shared memory, with groups
  float top;      // the largest logit; 0 if there is none
  bool sigmoid, by_score;
};

// fp64 scores: the softmax's sum, and u_e without the bias.
__device__ __forceinline__ double sum64(const Row w, int E) {
  double z = 0.0;
  if (!w.sigmoid) {
#pragma unroll 2
    for (int e = threadIdx.x % 32; e < E; e += 32)
      z += exp((double)clean(w.l[e]) - (double)w.top);
    z = warp_sum_of(z);
  }
  return z;
}
__device__ __forceinline__ double score64(const Row w, float v, double z) {
  if (w.sigmoid) return sigmoid_of((double)v);
  return z > 0.0 ? exp((double)v - (double)w.top) / z : 0.0;
}

// The topk_groups best groups' bits, by scores in fp64 (by_score) or logits.
__device__ __noinline__ uint32_t best_groups64(const GatingArgs &g, const Row w) {
  const int lane = threadIdx.x % 32, E = g.E, gsz = E / g.n_groups;
  double *s_u = reinterpret_cast<double *>(w.s_u);
  const double z = w.by_score ? sum64(w, E) : 0.0;
  __syncwarp();
#pragma unroll 2
  for (int e = lane; e < E; e += 32) {
    const float v = clean(w.l[e]);
    double u = v;
    if (w.by_score) {
      u = score64(w, v, z);
      if (g.sel_bias) u += (double)clean(g.sel_bias[e]);
    }
    s_u[e] = u;
  }
  __syncwarp();
  // L lanes scan a group, once for each score that is summed
  const int L = group_lanes(g.n_groups), gi = lane / L;
  const double *mine = s_u + gi * gsz;
  double score = 0.0, bound = 0.0;
  int bound_at = -1;
  for (int j = 0; j < g.group_score_topk; ++j) {
    double best = -INFINITY;
    int at = 1 << 20;
    if (gi < g.n_groups) {
      for (int e = lane % L; e < gsz; e += L) {
        const double v = mine[e];
        const bool left = bound_at < 0 || v < bound || (v == bound && e > bound_at);
        if (left && (at == 1 << 20 || v > best)) {
          best = v;
          at = e;
        }
      }
    }
    for (int off = L / 2; off > 0; off /= 2) {
      const double v = __shfl_xor_sync(kFull, best, off);
      const int e = __shfl_xor_sync(kFull, at, off);
      if (v > best || (v == best && e < at)) {
        best = v;
        at = e;
      }
    }
    score = j ? score + best : best;
    bound = best;
    bound_at = at;
  }
  score = __shfl_sync(kFull, score, (lane * L) % 32);  // lane i: group i's
  u64 gu = lane < g.n_groups ? order64(score) : 0;
  uint32_t kept = 0;
  for (int r = 0; r < g.topk_groups; ++r) {
    const u64 top = top64(gu);
    const int win = __ffs(__ballot_sync(kFull, gu == top)) - 1;
    kept |= 1u << win;
    if (lane == win) gu = 0;
  }
  __syncwarp();
  return kept;
}

// The topk_groups best groups' bits, from scores in steps (lane i: group i's, at
// least 1; 0 for none); where the last one kept and the first one dropped differ
// by at most tol, on the exact scores.
__device__ __forceinline__ uint32_t best_groups(const GatingArgs &g, uint32_t gu, int tol,
                                                const Row row) {
  const int lane = threadIdx.x % 32;
  uint32_t kept = 0, last = 0;
  for (int r = 0; r < g.topk_groups; ++r) {
    last = __reduce_max_sync(kFull, gu);
    const int win = __ffs(__ballot_sync(kFull, gu == last)) - 1;
    kept |= 1u << win;
    if (lane == win) gu = 0;
  }
  if (g.topk_groups < g.n_groups) {
    const uint32_t next = __reduce_max_sync(kFull, gu);
    if ((int)(last - next) <= tol) kept = best_groups64(g, row);
  }
  return kept;
}

// Sets the candidates of groups that are not kept to 0.
template <int NPL, typename U>
__device__ __forceinline__ void drop_groups(U (&c)[NPL], uint32_t kept, int E, int gsz) {
  const uint32_t recip = (uint32_t)((0x100000000ull + gsz - 1) / gsz);  // e / gsz for e < 1024
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const uint32_t e = i * 32 + threadIdx.x % 32, of = gsz == 1 ? e : __umulhi(e, recip);
    if (e < (uint32_t)E && !((kept >> of) & 1u)) c[i] = 0;
  }
}

// ---- selection on 32-bit words --------------------------------------------------
constexpr int kKeyBits = 22;
constexpr float kKeyTop = (float)((1 << kKeyBits) - 2);  // words stay below 2^32 - 1
constexpr float kKeySteps = kKeyTop - 8.f;  // finite keys: steps 8 and above, but for rounding
constexpr float kLogitRange = 64.f;
constexpr float kRangeLimit = 1e37f;  // of the keys; steps of larger ranges leave fp32's
// The step of a key of -inf (an expert that a bias masks), below every finite
// one: a group that has to count it has the score -inf, and not the sum of the
// steps, which could pass for that of a group of small keys.
constexpr uint32_t kMaskedStep = 1;

// The words of keys u: kKeyTop for `top`, the largest key, less by steps of
// range / kKeySteps; one and the same for everything `range` or more below it.
// 1.5 * 2^23 + v holds the nearest integer to v in its low bits.  Every step is
// monotone: a larger word means a larger u.
template <int NPL>
__device__ __forceinline__ void words(const float (&u)[NPL], float top, float range,
                                      float per_step, int E, uint32_t (&c)[NPL]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    const float d = fmaxf(u[i] - top, -range);
    const float v = fmaf(d, per_step, 12582912.0f + kKeyTop);
    c[i] = e < E ? (__float_as_uint(v) << 10) | (uint32_t)(1023 - e) : 0;
  }
}
// The words of keys that are -inf, where there are any.
template <int NPL>
__device__ __forceinline__ void masked_words(const float (&u)[NPL], int E, uint32_t (&c)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + (int)threadIdx.x % 32;
    if (e < E && u[i] == -INFINITY) c[i] = (kMaskedStep << 10) | (uint32_t)(1023 - e);
  }
}

// Groups of PER whole registers across the lanes: their scores, the sum of the
// group_score_topk largest keys in steps, and dropped groups' words set to 0.
template <int NPL, int PER>
__device__ __forceinline__ void groups_of_registers(const GatingArgs &g, uint32_t (&c)[NPL],
                                                    bool masked, int tol, const Row row) {
  const int lane = threadIdx.x % 32;
  uint32_t gu = 0, k[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) k[i] = c[i];
  for (int j = 0; j < g.group_score_topk; ++j) {
#pragma unroll
    for (int gi = 0; gi < NPL / PER; ++gi) {  // (behind the last group: zeros)
      uint32_t best = k[gi * PER];
#pragma unroll
      for (int q = 1; q < PER; ++q) best = max(best, k[gi * PER + q]);
      const uint32_t top = __reduce_max_sync(kFull, best);
      if (lane == gi) gu += top >> 10;
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (k[gi * PER + q] == top) k[gi * PER + q] = 0;  // not counted again
    }
  }
  if (masked) {
#pragma unroll
    for (int gi = 0; gi < NPL / PER; ++gi) {
      int left = 0;  // experts with a finite key
#pragma unroll
      for (int q = 0; q < PER; ++q)
        left += __popc(__ballot_sync(kFull, c[gi * PER + q] >= (kMaskedStep + 1) << 10));
      if (lane == gi && gu != 0 && left < g.group_score_topk) gu = kMaskedStep;
    }
  }
  const uint32_t kept = best_groups(g, gu, tol, row);
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (!((kept >> (i / PER)) & 1u)) c[i] = 0;
}

// Groups of any other size: 32 / n_groups lanes (a power of two) scan a group
// in this warp's shared memory.
template <int NPL>
__device__ __forceinline__ void groups_in_memory(const GatingArgs &g, uint32_t (&c)[NPL],
                                                 int tol, const Row row) {
  const int lane = threadIdx.x % 32, E = g.E, gsz = E / g.n_groups;
  uint32_t *s_c = reinterpret_cast<uint32_t *>(row.s_u);
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (i * 32 + lane < E) s_c[i * 32 + lane] = c[i];
  __syncwarp();
  const int L = group_lanes(g.n_groups), gi = lane / L, sub = lane % L;
  const uint32_t *mine = s_c + gi * gsz;
  uint32_t score = 0, bound = 0xffffffffu;
  for (int j = 0; j < g.group_score_topk; ++j) {
    uint32_t best = 0;
    if (gi < g.n_groups)
      for (int e = sub; e < gsz; e += L)
        if (mine[e] < bound) best = max(best, mine[e]);
    for (int off = L / 2; off > 0; off /= 2)
      best = max(best, __shfl_xor_sync(kFull, best, off));
    score += best >> 10;
    bound = best;
  }
  if (bound >> 10 == kMaskedStep) score = kMaskedStep;  // the last one counted is masked
  score = __shfl_sync(kFull, score, (lane * L) % 32);  // lane i: group i's
  drop_groups<NPL>(c, best_groups(g, lane < g.n_groups ? score : 0u, tol, row), E, gsz);
  __syncwarp();
}

// Lane j gets the j-th best expert of the `n` words (n >= k_t).  Where two
// neighbours of the first k_t + 1 differ by at most tol steps, `floor` is the
// smallest word that may be among the k_t best, else 0.
template <int NPL>
__device__ __forceinline__ int take_best(const uint32_t (&c)[NPL], int kt, int n, int tol,
                                         uint32_t &floor) {
  const int lane = threadIdx.x % 32;
  uint32_t h[4];
  best_four<NPL, false>(c, 0u, h);
  uint32_t mine = 0, extra = 0;
  const int rounds = n > kt ? kt + 1 : kt;
  for (int j = 0; j < rounds; ++j) {
    extra = __reduce_max_sync(kFull, h[0]);
    if (lane == j) mine = extra;
    const bool won = h[0] == extra;
    h[0] = won ? h[1] : h[0];
    h[1] = won ? h[2] : h[1];
    h[2] = won ? h[3] : h[2];
    h[3] = won ? 0 : h[3];
    if (NPL > 4 && won && h[0] == 0) best_four<NPL, true>(c, extra, h);  // its next ones
  }
  const uint32_t after = __shfl_down_sync(kFull, mine, 1);
  const uint32_t next = lane == kt - 1 ? (rounds > kt ? extra : 0u) : after;
  const bool close = lane < kt && (next != 0 && (int)((mine >> 10) - (next >> 10)) <= tol);
  const int last = (int)(__shfl_sync(kFull, mine, kt - 1) >> 10);
  floor = __any_sync(kFull, close) ? (uint32_t)max(last - tol, 1) << 10 : 0u;
  return lane < kt ? 1023 - (int)(mine & 1023u) : -1;
}

// s_list gets the experts whose words are at least `floor` (>= 1), in their
// order, the first kListed of them; returns their number.
constexpr int kListed = 64;
template <int NPL>
__device__ __forceinline__ int list_from(const uint32_t (&c)[NPL], uint32_t floor, int *s_list) {
  const int lane = threadIdx.x % 32;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const bool in = c[i] >= floor;
    const uint32_t all = __ballot_sync(kFull, in);
    const int at = n + __popc(all & ((1u << lane) - 1u));
    if (in && at < kListed) s_list[at] = i * 32 + lane;
    n += __popc(all);
  }
  __syncwarp();
  return n;
}

// ---- the listed experts in their exact order ------------------------------------
// Of the n <= kListed experts in s_list, two a lane, lane j gets the j-th best:
// on the logits' own bits, with a bias on the scores in fp64.  A lane counts
// those ahead of its own; equal keys stay in the list's order.
__device__ __noinline__ int choose_listed(const GatingArgs &g, const Row w, int *s_list, int n,
                                          int kt) {
  const int lane = threadIdx.x % 32;
  const double z = g.sel_bias ? sum64(w, g.E) : 0.0;
  u64 key[2] = {0, 0};
  int e[2] = {0, 0}, ahead[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = h * 32 + lane;
    e[h] = at < n ? s_list[at] : 0;
    const float v = clean(w.l[e[h]]);
    key[h] = g.sel_bias ? order64(score64(w, v, z) + (double)clean(g.sel_bias[e[h]]))
                        : (u64)gating::order_key(v);
    if (n <= 32) break;
  }
  for (int q = 0; q < n; ++q) {
    const u64 other = __shfl_sync(kFull, q < 32 ? key[0] : key[1], q % 32);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (other > key[h] || (other == key[h] && q < h * 32 + lane)) ++ahead[h];
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (h * 32 + lane < n) s_list[ahead[h]] = e[h];
  __syncwarp();
  return lane < kt ? s_list[lane] : -1;
}

// ---- selection on the logits' own bits --------------------------------------------
// For rows holding a NaN or +inf, and for tokens without a bias whose words leave
// more than kListed experts open.  64-bit candidates, equal logits in expert
// order.
template <int NPL>
__device__ __noinline__ int choose_logits(const GatingArgs &g, const Row row, int kt) {
  const int lane = threadIdx.x % 32, E = g.E;
  u64 c[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    c[i] = i * 32 + lane < E ? candidate(clean(row.l[i * 32 + lane]), i * 32 + lane) : 0;
  if (g.n_groups > 1) drop_groups<NPL>(c, best_groups64(g, row), E, E / g.n_groups);
  u64 h[4];
  best_four<NPL, false>(c, (u64)0, h);
  int mine = -1;
  for (int j = 0; j < kt; ++j) {
    const u64 top = top64(h[0]);
    if (lane == j) mine = 1023 - (int)(top & 1023);
    if (h[0] == top) {
      if (NPL > 4 && h[1] == 0) {
        best_four<NPL, true>(c, top, h);
      } else {
        h[0] = h[1];
        h[1] = h[2];
        h[2] = h[3];
        h[3] = 0;
      }
    }
  }
  return mine;
}

// ---- fp64 selection -----------------------------------------------------------
// For tokens with a bias whose words leave more than kListed experts open, or
// whose keys are infinite: plain scans.
template <int NPL>
__device__ __forceinline__ int take_best64(const double (&u)[NPL], uint32_t alive, int kt) {
  const int lane = threadIdx.x % 32;
  int mine = -1;
  for (int j = 0; j < kt; ++j) {
    u64 best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const u64 o = ((alive >> i) & 1u) ? order64(u[i]) : 0;
      if (o > best) {
        best = o;
        at = i;
      }
    }
    const u64 top = top64(best);
    if (top == 0) break;  // no candidate left
    const int win = __reduce_min_sync(kFull, best == top ? at * 32 + lane : 0x7fffffff);
    if (lane == (win & 31)) alive &= ~(1u << (win >> 5));
    if (lane == j) mine = win;
  }
  return mine;
}

template <int NPL>
__device__ __noinline__ int choose_scores(const GatingArgs &g, const Row w, int kt) {
  const int lane = threadIdx.x % 32, E = g.E;
  const double z = sum64(w, E);
  const uint32_t kept = g.n_groups > 1 ? best_groups64(g, w) : 1u;
  const int gsz = E / g.n_groups;
  double u[NPL];
  uint32_t alive = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = i * 32 + lane;
    u[i] = 0.0;
    if (e < E) {
      u[i] = score64(w, clean(w.l[e]), z) + (double)clean(g.sel_bias[e]);
      if ((kept >> (e / gsz)) & 1u) alive |= 1u << i;
    }
  }
  return take_best64<NPL>(u, alive, kt);
}

// fp32 scores are within these factors of the largest score (sigmoid: of 1) and
// the largest finite key.  Softmax: the fast exponential is off by
// (2 + 1.16 |x|) units of 2^-23, times e^-|x| at most 2 of them; the sum by that
// and at most NPL + 5 roundings (37 * 2^-24), the fast reciprocal and the product
// by three more.  Sigmoid: the exponential's error times s (1 - s), and 2 units
// for the fast division.  Each sum with a bias rounds once.
constexpr float kTolSoftmax = 4e-6f, kTolSigmoid = 6e-7f, kTolSum = 1.2e-7f;

// Warps on an SM: the registers are held down for them (what spills is around the
// second selections).  With 8, 5 and 3 CTAs in place of 9, 6 and 4: 12.1 -> 12.5,
// 102 -> 110 (65536 x 512) and 27 -> 31 us; 10 or 12 CTAs gain nothing.
template <int NPL>
__global__ void __launch_bounds__(kGateWarps * 32,
                                  NPL <= 8 ? 9 : NPL == 16 ? 6 : 4)
    k_gate(const __grid_constant__ GatingArgs g, const bool sigmoid, const bool renorm) {
  grid_dependency();  // the previous grid is complete; the next may launch
  extern __shared__ u64 s_gate[];  // [kGateWarps][E], with groups
  __shared__ int s_list[kGateWarps][kListed];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kGateWarps + warp;
  if (t >= g.T) return;  // whole warp leaves together
  const int E = g.E;
  const float *l = g.logits + (size_t)t * E;
  u64 *s_u = s_gate + (size_t)warp * E;
  int kt = g.k_per_token ? g.k_per_token[t] : g.k_max;
  if (kt < 1 || kt > g.k_max) {
    if (lane == 0) raise_error(g.err, kErrRouting);
    kt = kt < 1 ? 1 : g.k_max;
  }
  float u[NPL];
  float top = -INFINITY;
  bool bad = false;  // a NaN or +inf logit
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    u[i] = i * 32 + lane < E ? l[i * 32 + lane] : -INFINITY;
    bad |= !(u[i] < INFINITY);
    top = fmaxf(top, u[i]);  // NaN is skipped
  }
  // narrow rows: the bias is on its way while the row is looked at (128 tokens of
  // 256 experts 4.8 -> 3.5 us); wide ones have no registers left for it
  constexpr bool kEarly = NPL <= 8;
  float bias[kEarly ? NPL : 1];
  if constexpr (kEarly) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      bias[i] = g.sel_bias && i * 32 + lane < E ? g.sel_bias[i * 32 + lane] : 0.f;
  }
  bad = __any_sync(kFull, bad);
  // a row with such a logit has no scores: its experts are picked by the
  // logits, its weights are NaN
  const bool by_score = g.sel_bias || (g.n_groups > 1 && g.group_score_topk > 1);
  top = key_of(__reduce_max_sync(kFull, gating::order_key(top)));
  const float row_top = top;  // the largest logit
  if (top == -INFINITY) top = 0.f;  // nothing but -inf: every e^(l - top) is 0
  float z = 0.f;
  int my_idx = -1;
  bool open = bad;  // not selected yet
  const Row row = {l, s_u, top, sigmoid, by_score && !bad};
  if (!bad) {
    float key_top = row_top, range = kLogitRange, per_step = kKeySteps / kLogitRange;
    int tol = 0;  // logits: only equal keys leave their order open
    bool masked = false;  // by the bias: keys of -inf
    bool cut = false;  // finite keys below the range: they share the smallest word
    float smax = 0.f;  // softmax: the largest score
    if (!sigmoid && (by_score || !renorm)) {
      float e[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        e[i] = __expf(u[i] - top);
        z += e[i];
      }
      z = warp_sum(z);
      if (by_score) {
        smax = z > 0.f ? __fdividef(1.f, z) : 0.f;  // e^0 over the sum
#pragma unroll
        for (int i = 0; i < NPL; ++i) u[i] = e[i] * smax;
      }
    } else if (by_score) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) u[i] = __fdividef(1.f, 1.f + __expf(-u[i]));
    }
    if (by_score) {
      float size = 0.f, hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = i * 32 + lane;
        if (g.sel_bias && e < E) u[i] += clean(kEarly ? bias[kEarly ? i : 0] : g.sel_bias[e]);
        size = fmaxf(size, fabsf(u[i]));
        if (e < E) hi = fmaxf(hi, u[i]);
      }
      // (magnitudes are not negative: ordered as their bits are)
      size = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(size)));
      if (!(size < INFINITY)) {  // experts that a bias masks
        size = 0.f;
        masked = true;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          size = fmaxf(size, fabsf(u[i]) < INFINITY ? fabsf(u[i]) : 0.f);
        size = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(size)));
      }
      key_top = key_of(__reduce_max_sync(kFull, gating::order_key(hi)));
      // every finite key lies within it; its last limit is for the steps' sake (a
      // sum of words behind it says nothing about the sum of the keys)
      range = fminf(fmaxf(2.f * size, 1e-30f), kRangeLimit);
      cut = 2.f * size > kRangeLimit;
      per_step = __fdividef(kKeySteps, range);
      // twice the error of a key, in steps: of the score, and less than one step
      // from rounding the difference to the largest and the step
      const float err = (sigmoid ? kTolSigmoid : kTolSoftmax * smax) + kTolSum * size;
      // (at most all steps: every order is open)
      tol = 3 + (int)fminf(2.f * err * per_step, kKeyTop);
    }
    if (fabsf(key_top) < INFINITY) {
      uint32_t c[NPL];
      words<NPL>(u, key_top, range, per_step, E, c);
      if (masked) masked_words<NPL>(u, E, c);
      int n = E;
      if (g.n_groups > 1) {
        const int gtol = cut ? INT_MAX : tol * g.group_score_topk, gsz = E / g.n_groups;
        if (gsz == 32)
          groups_of_registers<NPL, 1>(g, c, masked, gtol, row);
        else if (NPL >= 4 && gsz == 64)
          groups_of_registers<NPL, NPL >= 4 ? 2 : 1>(g, c, masked, gtol, row);
        else if (NPL >= 8 && gsz == 128)
          groups_of_registers<NPL, NPL >= 8 ? 4 : 1>(g, c, masked, gtol, row);
        else
          groups_in_memory<NPL>(g, c, gtol, row);
        n = g.topk_groups * gsz;
        if (by_score && !g.sel_bias) {  // inside the groups the logits decide
          uint32_t w[NPL];
#pragma unroll
          for (int i = 0; i < NPL; ++i) u[i] = i * 32 + lane < E ? l[i * 32 + lane] : -INFINITY;
          words<NPL>(u, row_top, kLogitRange, kKeySteps / kLogitRange, E, w);
          open = !(row_top > -INFINITY);
#pragma unroll
          for (int i = 0; i < NPL; ++i) c[i] = c[i] ? w[i] : 0;
          tol = 0;
        }
      }
      uint32_t floor = 0;
      if (!open) my_idx = take_best<NPL>(c, kt, n, tol, floor);
      if (floor) {
        n = list_from<NPL>(c, floor, s_list[warp]);
        if (n <= kListed) my_idx = choose_listed(g, row, s_list[warp], n, kt);
        else open = true;
      }
    } else {
      open = true;  // no finite key, or an infinite one
    }
  }
  if (open)
    my_idx = (g.sel_bias && !bad) ? choose_scores<NPL>(g, row, kt) : choose_logits<NPL>(g, row, kt);

  // Weights, from the selected logits, in fp32: a few units of 2^-24 for the
  // exponential, the fast division and the sum z (whose fast exponentials err by
  // kTolSoftmax at most), and |l - top| of them from rounding that difference.
  const bool mine = lane < kt && my_idx >= 0;
  const float v = mine ? l[my_idx] : -INFINITY;
  float w = 0.f;
  if (bad) {
    w = __int_as_float(0x7fc00000);
  } else if (!renorm) {
    if (sigmoid) {
      w = sigmoid_of(v);
    } else {
      w = (mine && z > 0.f) ? __fdividef(expf(v - top), z) : 0.f;
    }
  } else {
    // s_j over their sum, both times e^-M with M = min(0, largest selected
    // logit): rows of very negative logits keep their ratios
    const float big = warp_max(v);
    if (big > -INFINITY) {
      float s;
      if (!sigmoid) {
        s = expf(v - big);
      } else {
        const float M = fminf(big, 0.f);
        s = v < 0.f ? __fdividef(expf(v - M), 1.f + expf(v)) : __fdividef(1.f, 1.f + expf(-v));
      }
      w = __fdividef(s, warp_sum(mine ? s : 0.f));
    }
  }
  if (lane < g.k_max) {
    g.topk_idx[(size_t)t * g.k_max + lane] = mine ? my_idx : -1;
    g.topk_w[(size_t)t * g.k_max + lane] = mine ? g.routed_scale * w : 0.f;
  }
}

template <int NPL>
cudaError_t run_gate(const GatingArgs &a, bool sigmoid, bool renorm, cudaStream_t s) {
  const int blocks = (a.T - 1) / kGateWarps + 1;
  const size_t smem = a.n_groups > 1 ? sizeof(u64) * kGateWarps * (size_t)a.E : 0;
  launch_k(k_gate<NPL>, blocks, kGateWarps * 32, smem, s, a, sigmoid, renorm);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
struct GateGradArgs {
  const float *logits, *dw;
  const int32_t *topk_idx;
  float *dlogits;
  int T, E, k;
  float scale;
  uint32_t *err;
};

// One warp per token: the gradients of the selected scores are put into a row
// of shared memory, which leaves as whole lines (16-byte stores when `vec`).
template <bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kGateWarps * 32)
    k_gate_grad(const GateGradArgs a, const bool vec) {
  grid_dependency();  // the previous grid is complete; the next may launch
  constexpr bool kDense = !SIGMOID && !RENORM;  // every expert's logit gets a gradient
  extern __shared__ float s_rows[];             // [kGateWarps][E rounded up to 4]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = a.E;
  const int t = blockIdx.x * kGateWarps + warp;
  if (t >= a.T) return;  // whole warp leaves together
  float *row = s_rows + (size_t)warp * ((E + 3) / 4 * 4);
  const float *l = a.logits + (size_t)t * E;
  float *out = a.dlogits + (size_t)t * E;

  int e = -1;
  float gj = 0.f;
  if (lane < a.k) {
    e = a.topk_idx[(size_t)t * a.k + lane];
    gj = a.scale * a.dw[(size_t)t * a.k + lane];
    if (e >= E || e < -1) {
      raise_error(a.err, kErrRouting);
      e = -1;
    }
  }
  const bool mine = e >= 0;
  if (!mine) gj = 0.f;
  const float v = mine ? l[e] : -INFINITY;

  float top = v, inv_z = 0.f;
  if constexpr (kDense) {
    if (vec) {
      for (int q = lane; q < E / 4; q += 32) {
        const float4 f = reinterpret_cast<const float4 *>(l)[q];
        reinterpret_cast<float4 *>(row)[q] = f;
        top = fmaxf(top, fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)));
      }
    } else {
      for (int q = lane; q < E; q += 32) {
        const float f = l[q];
        row[q] = f;
        top = fmaxf(top, f);
      }
    }
    top = warp_max(top);
    if (top == -INFINITY) top = 0.f;  // nothing but -inf: every e^(l - top) is 0
    float z = 0.f;
    __syncwarp();
    // the row becomes e^(l - top)
    if (vec) {
      for (int q = lane; q < E / 4; q += 32) {
        float4 f = reinterpret_cast<float4 *>(row)[q];
        f.x = expf(f.x - top);
        f.y = expf(f.y - top);
        f.z = expf(f.z - top);
        f.w = expf(f.w - top);
        reinterpret_cast<float4 *>(row)[q] = f;
        z += (f.x + f.y) + (f.z + f.w);
      }
    } else {
      for (int q = lane; q < E; q += 32) {
        const float p = expf(row[q] - top);
        row[q] = p;
        z += p;
      }
    }
    z = warp_sum(z);
    inv_z = z == 0.f ? 0.f : 1.f / z;  // NaN for a row with NaN or +inf
  } else {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = lane; q < (E + 3) / 4; q += 32) reinterpret_cast<float4 *>(row)[q] = zero;
    top = warp_max(top);
  }

  // what a selected slot adds to its logit
  float d = 0.f, dot = 0.f;
  if constexpr (kDense) {
    const float p = mine ? expf(v - top) * inv_z : 0.f;
    dot = warp_sum(gj * p);
    d = gj * p;
  } else if constexpr (!SIGMOID) {
    const float ex = (mine && top > -INFINITY) ? expf(v - top) : 0.f;
    const float sum = warp_sum(ex);
    const float n = sum == 0.f ? 0.f : ex / sum;
    d = n * (gj - warp_sum(gj * n));
  } else if constexpr (!RENORM) {
    const float s = mine ? sigmoid_of(v) : 0.f;
    d = gj * s * sigmoid_of(-v);  // 1 - s = sigmoid(-v), without cancellation
  } else {
    // shares n_j as in the forward pass: dl_j = (g_j - sum g_i n_i) n_j (1 - s_j)
    const float M = fminf(top, 0.f);
    float s = 0.f;
    if (mine && top > -INFINITY)
      s = v < 0.f ? expf(v - M) / (1.f + expf(v)) : 1.f / (1.f + expf(-v));
    const float sum = warp_sum(s);
    const float n = sum == 0.f ? 0.f : s / sum;
    d = (gj - warp_sum(gj * n)) * n * (mine ? sigmoid_of(-v) : 0.f);
  }
  // the forward pass has no weights for such a row
  if (!kDense && __any_sync(kFull, mine && !(v < INFINITY))) d = __int_as_float(0x7fc00000);
  __syncwarp();
  if constexpr (kDense) {
    const float c = -dot * inv_z;  // dl_e = p_e (ds_e - dot), p_e = row_e * inv_z
    if (!__any_sync(kFull, mine)) {  // no slot: zeros, whatever the logits are
      for (int q = lane; q < E; q += 32) row[q] = 0.f;
    } else if (vec) {
      for (int q = lane; q < E / 4; q += 32) {
        const float4 f = reinterpret_cast<float4 *>(row)[q];
        reinterpret_cast<float4 *>(row)[q] = make_float4(f.x * c, f.y * c, f.z * c, f.w * c);
      }
    } else {
      for (int q = lane; q < E; q += 32) row[q] *= c;
    }
    __syncwarp();
  }
  // Add the slots in; an expert named by several slots gets them in slot order.
  const uint32_t same = __match_any_sync(kFull, e);
  float sum = d;
  if (__any_sync(kFull, mine && same != (1u << lane))) {
    sum = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float o = __shfl_sync(kFull, d, j);
      if ((same >> j) & 1u) sum += o;
    }
  }
  if (mine && lane == __ffs(same) - 1) row[e] += sum;
  __syncwarp();
  if (vec) {
    for (int q = lane; q < E / 4; q += 32)
      reinterpret_cast<float4 *>(out)[q] = reinterpret_cast<const float4 *>(row)[q];
  } else {
    for (int q = lane; q < E; q += 32) out[q] = row[q];
  }
}

template <bool SIGMOID, bool RENORM>
cudaError_t run_grad(const GateGradArgs &a, cudaStream_t s) {
  const int blocks = (a.T - 1) / kGateWarps + 1;
  const size_t smem = sizeof(float) * kGateWarps * (size_t)((a.E + 3) / 4 * 4);
  const bool vec = a.E % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) |
                                     reinterpret_cast<uintptr_t>(a.dlogits)) & 15u) == 0;
  launch_k(k_gate_grad<SIGMOID, RENORM>, blocks, kGateWarps * 32, smem, s, a, vec);
  return cudaGetLastError();
}

}  // namespace

bool general_gating(int gating) {
  return gating >= MOE_GATE_SOFTMAX && gating <= MOE_GATE_SIGMOID_RENORM;
}

cudaError_t launch_gate_general(const moe_config &c, const float *logits, const float *sel_bias,
                                const int32_t *k_per_token, int32_t *topk_idx, float *topk_w,
                                uint32_t *err, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const bool sigmoid = c.gating == MOE_GATE_SIGMOID || c.gating == MOE_GATE_SIGMOID_RENORM;
  const bool renorm = c.gating == MOE_GATE_SOFTMAX_RENORM || c.gating == MOE_GATE_SIGMOID_RENORM;
  GatingArgs a{logits,  sel_bias, k_per_token, topk_idx,      topk_w,
               c.T,     c.E,      c.k_max,     c.gating,      c.n_groups,
               c.topk_groups,     c.group_score_topk, c.routed_scale, err};
  const int npl = (c.E + 31) / 32;
  if (npl <= 1) return run_gate<1>(a, sigmoid, renorm, s);
  if (npl <= 2) return run_gate<2>(a, sigmoid, renorm, s);
  if (npl <= 4) return run_gate<4>(a, sigmoid, renorm, s);
  if (npl <= 8) return run_gate<8>(a, sigmoid, renorm, s);
  if (npl <= 16) return run_gate<16>(a, sigmoid, renorm, s);
  return run_gate<32>(a, sigmoid, renorm, s);
}

cudaError_t launch_gate_grad(const moe_config &c, const float *logits, const int32_t *topk_idx,
                             const float *dtopk_w, float *dlogits, uint32_t *err,
                             cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const bool scaled = c.gating == MOE_SIGMOID_GROUPED || general_gating(c.gating);
  GateGradArgs a{logits, dtopk_w, topk_idx, dlogits, c.T, c.E, c.k_max,
                 scaled ? c.routed_scale : 1.0f, err};
  switch (c.gating) {
    case MOE_GATE_SOFTMAX: return run_grad<false, false>(a, s);
    case MOE_GATE_SIGMOID: return run_grad<true, false>(a, s);
    case MOE_SIGMOID_GROUPED:
    case MOE_GATE_SIGMOID_RENORM: return run_grad<true, true>(a, s);
    default: return run_grad<false, true>(a, s);
  }
}

}  // namespace moe
