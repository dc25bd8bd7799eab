// The top-k router: expert ids, weights and load statistics from logits, and
// the gradient to the logits.
//
//   key_e    = logit_e + bias_e (one fp32 addition; bias only selects)
//   ids      = the k largest keys, ties to the lowest id, in descending order;
//              a key of -inf is never chosen (id -1, weight 0)
//   score    = softmax(logits) or sigmoid(logits)
//   weights  = score of the chosen, divided by their sum if renormalised, times scale
//   p        = score / sum of the scores (softmax: the score itself)
//   balance  = E / (k T^2) * sum_e count_e * sum_t p_te,   z = sum_t lse_t^2 / T
//
// T counts the live tokens: those the mask keeps that have a key above -inf.
// A row with a key that is NaN or +inf has no order: its ids are -1 and its
// weights NaN.
//
// Layout: a token belongs to 16 lanes (8 where that is faster, see
// eight_lanes; the wave above 512 experts), lane l of G holding experts l, l +
// G, ... in registers, so a wave runs four or eight tokens at once and every
// reduction over a token is three or four DPP instructions.
//
// The choice. Per token it costs instructions, not bytes, so it decides the
// kernel's time beyond about 64 experts. Up to k = 16 it is a sorting
// network on 32-bit words, the key's order-preserving bits with the lowest 8
// (9 and 10 above 256 and 512 experts) replaced by the complement of the expert id: a
// comparator is one max and one min, a lane sorts its experts' words to the
// 8 or 16 largest, and merges with the lists of other lanes (max with a DPP
// operand, then a half-cleaner) leave the token's list in every lane.
// For bf16 logits without a bias the words order exactly as the keys do. For
// fp32 keys two words may agree in the key bits they keep while the keys
// differ below: that is checked for (neighbours in the list, and the first
// word behind it), and a wave that meets it, or a k above 16, runs k exact
// rounds of (largest key, lowest id that has it, take it out) instead.
#include <algorithm>
#include <type_traits>

#include "mok_internal.h"
#include "wave_ops.h"

namespace mok {
namespace {

// exp(x) for x <= 0 on the hardware's exponential (1 ulp): the rounding of x
// * log2(e) is an error of |x| 2^-24 of the value. For fp32 logits that is no
// more than the rounding of their difference, which x is; differences of bf16
// logits are mostly exact, and there it is the largest error of a score. -inf
// gives 0. (Sums and quotients of scores come out within 1e-7 of the float64
// definition, relative in the 2-norm, for logits of a few units.)
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// Over a token's group of G lanes (8, 16 or the wave).
template <int G>
__device__ __forceinline__ float grp_sum(float x) {
  if constexpr (G == 8) return octet_sum(x);
  if constexpr (G == 16) return row_sum(x);
  return wave_sum(x);
}
template <int G>
__device__ __forceinline__ float grp_max(float x) {
  if constexpr (G == 8) return octet_maxf(x);
  if constexpr (G == 16) return row_max(x);
  return wave_max(x);
}
template <int G>
__device__ __forceinline__ int grp_min(int x) {
  if constexpr (G == 8) return octet_min(x);
  if constexpr (G == 16) return row_min(x);
  return wave_min(x);
}
// Whether any lane of the group says so.
template <int G>
__device__ __forceinline__ bool grp_any(bool x) {
  const uint64_t b = __ballot(x);
  if constexpr (G < 64) return ((uint32_t)(b >> (lane_id() & (64 - G))) & ((1u << G) - 1u)) != 0;
  return b != 0;
}
#if defined(__HIP_DEVICE_COMPILE__)
// NaN or +inf, in one instruction.
__device__ __forceinline__ bool is_nan_or_inf(float x) { return __builtin_amdgcn_classf(x, 0x203); }
#else
__device__ bool is_nan_or_inf(float x);  // device only
#endif
constexpr float kInf = __builtin_inff();
// words of the statistics' scratch before the partial rows (router_stats)
constexpr int kStatsHead = 128, kStatsZ = 96;

struct RouterFwd {
  const void* logits;
  int64_t T, ld;
  int E, k;
  const float* bias;      // null: none
  const uint8_t* mask;    // null: every token
  int sigmoid, renorm;
  int exact_words;        // the network's words order exactly as the keys: bf16 logits, no bias
  float scale;
  float* weights;
  int64_t* ids;
  float* part;            // statistics (router_stats)
};

// Bits of a key in its order (larger key, larger word). The key must not be
// -0, which is equal to +0: callers add +0. -inf is kNone, words of numbers
// lie above it.
constexpr uint32_t kNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t ordered(float key) {
  const uint32_t u = f2u(key);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// The bits of a word that hold the complement of the expert id, with G lanes
// of V experts each.
constexpr uint32_t word_ids(int G, int V) { return G * V <= 256 ? 255u : G * V - 1u; }
// The key that a word without lost bits came from (bf16 keys).
__device__ __forceinline__ float key_of(uint32_t word, uint32_t ids) {
  return u2f(word & 0x80000000u ? (word ^ 0x80000000u) & ~ids : ~(word | ids));
}

// A token's logits, lane gl of its group holding experts gl, gl + G, ... (-inf
// past E), and what they say of the token.
template <typename LT, int G, int VPL, bool WORDS>
struct Row {
  float l[VPL];
  uint32_t word[VPL];  // WORDS: the keys' words for the network
  float top;           // largest logit
  bool live;           // kept by the mask, and some key above -inf or no order
  bool broken;         // a key that is NaN or +inf

  // `p`: the workgroup's first token of this turn, `off` this token's offset
  // from it, `last` the last one that may be read.
  __device__ __forceinline__ void load(const LT* p, uint32_t off, uint32_t last, const float* bias, int E, int gl,
                                       bool keep) {
    constexpr uint32_t kIds = word_ids(G, VPL);
    const char* b = (const char*)p;  // (bytes in 32 bits: a scalar base and one register of offset)
    if (E == G * VPL) {
      const uint32_t o = (off + (uint32_t)gl) * (uint32_t)sizeof(LT);
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = load1((const LT*)(b + o) + i * G);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        l[i] = load1((const LT*)(b + min(off + (uint32_t)(i * G + gl), last) * (uint32_t)sizeof(LT)));
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = i * G + gl < E ? l[i] : -kInf;
    }
    top = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = __builtin_fmaxf(top, l[i]);
    top = grp_max<G>(top);
    float most = top;
    bool odd = false;
    auto see = [&](int i, float key) {
      odd |= is_nan_or_inf(key);
      if constexpr (WORDS) word[i] = (ordered(key) & ~kIds) | (kIds - (uint32_t)(i * G + gl));
    };
    if (bias) {
      most = -kInf;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float key = l[i] + bias[min(i * G + gl, E - 1)] + 0.0f;  // (-0 + -0 is -0)
        most = __builtin_fmaxf(most, key);
        see(i, key);
      }
      most = grp_max<G>(most);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) see(i, l[i] + 0.0f);
    }
    broken = keep && grp_any<G>(odd);
    live = keep && (broken || most > -kInf);
  }
};

// Score of a logit up to a factor common to its token, from the token's
// largest logit `top` (for sigmoid at most 0): e^(l - top), or sigmoid(l) /
// e^top = e^(min(l, 0) - top) / (1 + e^-|l|), which is not 0 / 0 where every
// logit is far below 0. l = -inf gives 0 (in a token that has a number).
template <bool SIGMOID>
__device__ __forceinline__ float score_of(float l, float top) {
  if constexpr (!SIGMOID) return exp_neg(l - top);
  return exp_neg(__builtin_fminf(l, 0.f) - top) * __builtin_amdgcn_rcpf(1.f + exp_neg(-__builtin_fabsf(l)));
}
// 1 - sigmoid(l)
__device__ __forceinline__ float one_minus(float l) {
  return exp_neg(__builtin_fminf(-l, 0.f)) * __builtin_amdgcn_rcpf(1.f + exp_neg(-__builtin_fabsf(l)));
}

// ---- the sorting network --------------------------------------------
// A bitonic list of N words into descending order.
template <int N>
__device__ __forceinline__ void merge_desc(uint32_t (&w)[N]) {
#pragma unroll
  for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & h) == 0) {
        const uint32_t a = w[i], b = w[i + h];
        w[i] = max(a, b);
        w[i + h] = min(a, b);
      }
}
// The comparators of Batcher's odd-even merge sort of N words (19 for 8, 63
// for 16; a bitonic sort has 24 and 80).
template <int N>
struct OddEvenSort {
  int n = 0;
  signed char lo[80] = {}, hi[80] = {};
  constexpr OddEvenSort() {
    for (int p = 1; p < N; p *= 2)
      for (int d = p; d >= 1; d /= 2)
        for (int j = d % p; j + d < N; j += 2 * d)
          for (int i = 0; i < d && i + j + d < N; ++i)
            if ((i + j) / (2 * p) == (i + j + d) / (2 * p)) lo[n] = (signed char)(i + j), hi[n++] = (signed char)(i + j + d);
  }
};
// N words into descending order.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&w)[N]) {
  constexpr OddEvenSort<N> c{};
#pragma unroll
  for (int i = 0; i < c.n; ++i) {
    const uint32_t x = w[c.lo[i]], y = w[c.hi[i]];
    w[c.lo[i]] = max(x, y);
    w[c.hi[i]] = min(x, y);
  }
}
// The N largest of a lane's list and another lane's (both descending): the
// larger of opposite ends is a bitonic list of exactly those.
template <int N, int CTRL>
__device__ __forceinline__ void merge_dpp(uint32_t (&w)[N]) {
  uint32_t m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = max(w[i], (uint32_t)dpp_mov<CTRL>((int)w[N - 1 - i]));
  merge_desc<N>(m);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = m[i];
}
template <int N>
__device__ __forceinline__ void merge_xor(uint32_t (&w)[N], int d) {
  uint32_t m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = max(w[i], (uint32_t)__shfl_xor((int)w[N - 1 - i], d));
  merge_desc<N>(m);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = m[i];
}

// The word of choice gl of the token (kNone or less: none) in lane gl of the
// group, for k <= N <= 16. False (for the whole wave) if some token's order
// hangs on key bits that the words do not keep.
template <int N, int G, int VPL>
__device__ __forceinline__ bool choose_network(const uint32_t (&word)[VPL], int gl, int k, bool exact, bool keep,
                                               uint32_t& mine) {
  constexpr uint32_t kIds = word_ids(G, VPL);
  uint32_t top[N];
#pragma unroll
  for (int c = 0; c < VPL; c += N) {
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = c + i < VPL ? word[c + i < VPL ? c + i : 0] : 0u;
    sort_desc<N>(w);
    if (c == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) top[i] = w[i];
    } else {
      uint32_t m[N];
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] = max(top[i], w[N - 1 - i]);
      merge_desc<N>(m);
#pragma unroll
      for (int i = 0; i < N; ++i) top[i] = m[i];
    }
  }
  // each step pairs a lane with one whose list covers other lanes: the next
  // one, the next two, the mirrored four, the mirrored eight
  merge_dpp<N, kQuadXor1>(top);
  merge_dpp<N, kQuadXor2>(top);
  merge_dpp<N, kHalfMirror>(top);
  if constexpr (G >= 16) merge_dpp<N, kMirror>(top);
  if constexpr (G == 64) {
    merge_xor<N>(top, 16);
    merge_xor<N>(top, 32);
  }
  mine = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) mine = gl == j && j < k ? top[j] : mine;
  if (exact) return true;
  // neighbours in the list, and the first word behind the k chosen
  auto close = [](uint32_t a, uint32_t b) { return b > kNone && ((a ^ b) & ~kIds) == 0; };
  uint32_t last = 0, behind = 0;
  bool any = false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    last = j == k - 1 ? top[j] : last;
    if (j + 1 < N) any |= j + 1 < k && close(top[j], top[j + 1 < N ? j + 1 : j]);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) behind = max(behind, word[i] < last ? word[i] : 0u);
  any |= close(last, behind);
  return __ballot(keep && any) == 0;
}

// NET: width of the sorting network, 8 for k <= 8, else 16.
// STATS: the sums behind the losses and counts. A workgroup then keeps them
// in registers and LDS over its tokens and writes one partial row.
template <typename LT, int G, int VPL, int BLOCK, bool STATS, bool SIGMOID, int NET>
__global__ void __launch_bounds__(BLOCK) router_rows(RouterFwd a) {
  constexpr int GPB = BLOCK / G;
  constexpr int KQ = NET == 8 ? 1 : 64 / G;  // choices a lane may hold (k <= 8, or <= 64)
  extern __shared__ float lds[];  // STATS: int cnt[E + 1], then float sums[waves][E + 1]
  const int E = a.E, k = a.k;
  const int lane = (int)threadIdx.x % G, group = (int)threadIdx.x / G;
  int* cnt = (int*)lds;
  float psum[VPL];
  float zsum = 0.f;
  int nlive = 0;
  if constexpr (STATS) {
    for (int i = threadIdx.x; i <= E; i += BLOCK) cnt[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPL; ++i) psum[i] = 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < a.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + group;
    const bool in = t < a.T;
    // (a new value to the compiler in each turn: what follows from it for each
    // of the lane's experts would otherwise be computed before the loop and
    // held, in more registers than there are)
    const int gl = opaque(lane);
    const bool keep = in && (!a.mask || a.mask[t]);
    // (a workgroup's tokens lie within 2^31 elements: the host checks ld)
    const LT* rows = (const LT*)a.logits + t0 * a.ld;
    const uint32_t ld = (uint32_t)a.ld, ngrp = (uint32_t)min<int64_t>(GPB, a.T - t0);
    const uint32_t off = min((uint32_t)group, ngrp - 1) * ld, last = (ngrp - 1) * ld + (uint32_t)E - 1;
    const LT* row = rows + off;
    Row<LT, G, VPL, true> r;
    r.load(rows, off, last, a.bias, E, gl, keep);
    int pick[KQ];
#pragma unroll
    for (int q = 0; q < KQ; ++q) pick[q] = -1;
    uint32_t mine = 0;
    const bool done = k <= NET && choose_network<NET, G, VPL>(r.word, gl, k, a.exact_words, keep, mine);
    if (done) pick[0] = mine > kNone ? (int)(word_ids(G, VPL) - (mine & word_ids(G, VPL))) : -1;
    if (!done) {
      float key[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        key[i] = a.bias ? r.l[i] + a.bias[min(i * G + gl, E - 1)] : r.l[i];
      }
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        pick[q] = -1;
        for (int j = 0; j < G; ++j) {
          if (q * G + j >= k) break;
          float m = key[0];
#pragma unroll
          for (int i = 1; i < VPL; ++i) m = __builtin_fmaxf(m, key[i]);
          m = grp_max<G>(m);
          int at = 0x7FFFFFFF;
#pragma unroll
          for (int i = VPL - 1; i >= 0; --i) at = key[i] == m ? i * G + gl : at;
          at = grp_min<G>(at);
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = i * G + gl == at ? -kInf : key[i];
          if (gl == j && m > -kInf) pick[q] = at;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < KQ; ++q) pick[q] = keep && !r.broken ? pick[q] : -1;
    // weights of the choices: lane j of the group holds choice j, j + G, ...
    const float nan = r.broken ? __builtin_nanf("") : 0.f;
    float w[KQ], ltop = -kInf;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      if (q * G >= k) break;
      w[q] = pick[q] < 0 ? -kInf : done && a.exact_words ? key_of(mine, word_ids(G, VPL)) : load1(row + pick[q]);
      ltop = __builtin_fmaxf(ltop, w[q]);
    }
    // the scores over all experts, where anything needs them
    float den = 0.f, score[VPL];
    const float ptop = SIGMOID ? __builtin_fminf(r.top, 0.f) : r.top;
    if (STATS || (!SIGMOID && !a.renorm)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        score[i] = score_of<SIGMOID>(r.l[i], ptop);
        den += score[i];
      }
      den = grp_sum<G>(den);
    }
    const float wtop = a.renorm ? grp_max<G>(ltop) : SIGMOID ? 0.f : ptop;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      if (q * G >= k) break;
      w[q] = pick[q] < 0 ? 0.f : score_of<SIGMOID>(w[q], SIGMOID ? __builtin_fminf(wtop, 0.f) : wtop);
      sum += w[q];
    }
    const float total = a.scale * __builtin_amdgcn_rcpf(a.renorm ? grp_sum<G>(sum) : SIGMOID ? 1.f : den);
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      if (q * G >= k) break;
      const int j = q * G + gl;
      if (in && j < k) {
        const int64_t o = t * k + j;
        a.ids[o] = pick[q];
        a.weights[o] = (pick[q] >= 0 ? w[q] * total : 0.f) + nan;
      }
      if (STATS && pick[q] >= 0) atomicAdd(cnt + pick[q], 1);  // integers: any order gives the same count
    }
    if constexpr (STATS) {
      if (r.live) {
        const float inv = __builtin_amdgcn_rcpf(den) + nan;
#pragma unroll
        for (int i = 0; i < VPL; ++i) psum[i] = __builtin_fmaf(score[i], inv, psum[i]);
        if (gl == 0) {
          const float lse = r.top + __logf(den) + nan;
          zsum = __builtin_fmaf(lse, lse, zsum);
          ++nlive;
        }
      }
    }
  }
  if constexpr (STATS) {
    // a wave's tokens, then the waves in order
    constexpr int WAVES = BLOCK / 64;
    float* sums = lds + (E + 1);
    const int wave = threadIdx.x >> 6, wl = lane_id();
#pragma unroll
    for (int d = G; d < 64; d *= 2)
#pragma unroll
      for (int i = 0; i < VPL; ++i) psum[i] += __shfl_xor(psum[i], d);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (wl < G && i * G + wl < E) sums[wave * (E + 1) + i * G + wl] = psum[i];
    zsum = wave_sum(zsum);
    if (wl == 0) sums[wave * (E + 1) + E] = zsum;
    if (lane == 0 && nlive) atomicAdd(cnt + E, nlive);
    __syncthreads();
    float* part = a.part + kStatsHead + (int64_t)blockIdx.x * 2 * (E + 1);
    for (int i = threadIdx.x; i <= E; i += BLOCK) {
      float s = 0.f;
#pragma unroll
      for (int wv = 0; wv < WAVES; ++wv) s += sums[wv * (E + 1) + i];
      part[i] = s;
      ((int*)part)[E + 1 + i] = cnt[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *(uint32_t*)a.part = 0;  // router_stats' counter
  }
}

// Adds the workgroups' partial rows in a fixed order and forms the losses.
// A workgroup takes 16 columns, 64 adders each, so that every load of a
// thread is in flight at once; the workgroup that finishes last (a counter
// that the launch before cleared) adds the columns' products in order, so
// one launch does both.
//
// The scratch: kStatsHead words, [0] the counter, [1 + b] workgroup b's sum
// of count_e * (sum of p_e), [kStatsZ] the sum of lse^2, [kStatsZ + 1] the
// live tokens; then per workgroup of the forward 2 (E + 1) words, the sums of
// p and of lse^2 and the counts and live tokens.
__global__ void __launch_bounds__(1024) router_stats(float* part, int nparts, int E, int k, int sigmoid,
                                                     int32_t* counts, float* losses) {
  __shared__ float fs[16][16];
  __shared__ int is[16][16];
  const int wl = lane_id(), wave = threadIdx.x >> 6;
  const int c = (int)blockIdx.x * 16 + (wl & 15);
  const int g = wave * 4 + (wl >> 4);
  const int W = 2 * (E + 1);
  const float* rows = part + kStatsHead;
  float f = 0.f;
  int n = 0;
  if (c <= E)
#pragma unroll 4
    for (int r = g; r < nparts; r += 64) {
      f += rows[(int64_t)r * W + c];
      n += ((const int*)rows)[(int64_t)r * W + E + 1 + c];
    }
  f += __shfl_xor(f, 16), n += __shfl_xor(n, 16);
  f += __shfl_xor(f, 32), n += __shfl_xor(n, 32);
  if (wl < 16) fs[wave][wl] = f, is[wave][wl] = n;
  __syncthreads();
  if (wave != 0) return;
  f = 0.f, n = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) f += fs[i][wl & 15], n += is[i][wl & 15];
  if (wl < 16 && c <= E) counts[c] = n;
  const float dot = row_sum(c < E ? (float)n * f : 0.f);
  if (wl < 16 && c == E) {
    __hip_atomic_store(part + kStatsZ, f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store((int*)part + kStatsZ + 1, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (wl == 0) __hip_atomic_store(part + 1 + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __threadfence();  // every lane's stores, before the count
  uint32_t done = 0;
  if (wl == 0) done = __hip_atomic_fetch_add((uint32_t*)part, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1;
  done = (uint32_t)lane_value((int)done, 0);
  if (done != gridDim.x) return;
  float s = 0.f;
  for (uint32_t b = wl; b < gridDim.x; b += 64)
    s += __hip_atomic_load(part + 1 + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = wave_sum(s);
  if (wl != 0) return;
  const float z = __hip_atomic_load(part + kStatsZ, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float live = (float)max(__hip_atomic_load((int*)part + kStatsZ + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), 1);
  losses[0] = s / live / live * ((float)E / (float)k);
  losses[1] = sigmoid ? 0.f : z / live;
}

struct RouterBwd {
  const void* logits;
  int64_t T, ld;
  int E, k;
  const float* bias;
  const uint8_t* mask;
  int sigmoid, renorm;
  float scale;
  const float* d_weights;   // [T, k]
  const int64_t* ids;       // [T, k]
  const int32_t* counts;    // [E + 1]; null: no losses
  const float* d_losses;    // [2]
  void* d_logits;           // [T, E], the logits' type
};

// d_logits of one token, for chosen c_j with dw_j = scale * d_weights_j:
//   softmax, renormalised, q = softmax over the chosen:  q_c (dw_c - sum q dw) at the chosen
//   softmax:        p_e (dw_e [e chosen] - sum_j p_cj dw_j)
//   sigmoid:        s (1 - s) dw;  renormalised: (1 - s_c) q_c (dw_c - sum q dw), q = s / sum of the chosen s
//   losses:         a_e = d_balance * E / (k T^2) * count_e:  p_e (a_e - sum p a), for sigmoid times (1 - s_e);
//                   softmax: + d_z * 2 lse / T * p_e
// KQ: choices a lane may hold (k <= KQ * G).
template <typename LT, int G, int VPL, int BLOCK, bool SIGMOID, int KQ>
__global__ void __launch_bounds__(BLOCK) router_bwd_rows(RouterBwd a) {
  constexpr int GPB = BLOCK / G;
  const int E = a.E, k = a.k;
  const int lane = (int)threadIdx.x % G, group = (int)threadIdx.x / G;
  const bool losses = a.counts != nullptr;
  // a token's row by expert: first its logits, for the chosen ones, then the
  // gradients to the chosen ones (rows padded so that the four tokens of a
  // wave meet different banks)
  __shared__ float by_expert[GPB][G * VPL + 16];
  float gz = 0.f, ga[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) ga[i] = 0.f;
  if (losses) {
    const float n = (float)max(a.counts[E], 1);
    const float g = a.d_losses[0] * ((float)E / (float)k) / n / n;
    gz = SIGMOID ? 0.f : a.d_losses[1] * 2.f / n;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i * G + lane < E) ga[i] = g * (float)a.counts[i * G + lane];
  }
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < a.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + group;
    const bool in = t < a.T;
    // (a new value to the compiler in each turn: what follows from it for each
    // of the lane's experts would otherwise be computed before the loop and
    // held, in more registers than there are)
    const int gl = opaque(lane);
    const bool keep = in && (!a.mask || a.mask[t]);
    // (a workgroup's tokens lie within 2^31 elements: the host checks ld)
    const LT* rows = (const LT*)a.logits + t0 * a.ld;
    const uint32_t ld = (uint32_t)a.ld, ngrp = (uint32_t)min<int64_t>(GPB, a.T - t0);
    const uint32_t off = min((uint32_t)group, ngrp - 1) * ld, last = (ngrp - 1) * ld + (uint32_t)E - 1;
    // the choices, one or more per lane; an id outside [0, E) has no gradient
    int id[KQ];
    float c[KQ], lc[KQ], ltop = -kInf;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const int j = q * G + gl;
      id[q] = -1;
      c[q] = 0.f;
      if (q * G < k && keep && j < k) {
        const int64_t v = a.ids[t * k + j];
        const float d = a.d_weights[t * k + j];  // (without an expert anything: a weight of 0 has an infinite logarithm)
        id[q] = v >= 0 && v < E ? (int)v : -1;
        c[q] = d * a.scale;
      }
    }
    Row<LT, G, VPL, false> r;
    r.load(rows, off, last, a.bias, E, gl, keep);
    float* mine = by_expert[group];
#pragma unroll
    for (int i = 0; i < VPL; ++i) mine[i * G + gl] = r.l[i];
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      lc[q] = id[q] >= 0 ? mine[id[q]] : -kInf;
      c[q] = id[q] >= 0 ? c[q] : 0.f;
      ltop = __builtin_fmaxf(ltop, lc[q]);
    }
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < VPL; ++i) mine[i * G + gl] = 0.f;
    wave_lds_fence();
    const float ptop = SIGMOID ? __builtin_fminf(r.top, 0.f) : r.top;
    const float nan = r.broken ? __builtin_nanf("") : 0.f;
    float p[VPL], den = 0.f;
    const bool full = losses || (!SIGMOID && !a.renorm);
    if (full) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        p[i] = score_of<SIGMOID>(r.l[i], ptop);
        den += p[i];
      }
      den = grp_sum<G>(den);
      const float inv = __builtin_amdgcn_rcpf(den);
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] *= inv;
    }
    // c becomes the gradient to the chosen logits
    float along = 0.f;  // softmax without renormalisation: sum_j p_cj dw_j
    {
      const float wtop = a.renorm ? grp_max<G>(ltop) : SIGMOID ? 0.f : ptop;
      float sc[KQ], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        sc[q] = id[q] < 0 ? 0.f : score_of<SIGMOID>(lc[q], SIGMOID ? __builtin_fminf(wtop, 0.f) : wtop);
        sum += sc[q];
        dot = __builtin_fmaf(sc[q], c[q], dot);
      }
      if (a.renorm) {
        sum = grp_sum<G>(sum);
        sum = sum > 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f;
        dot = grp_sum<G>(dot) * sum;
      } else {
        sum = SIGMOID ? 1.f : __builtin_amdgcn_rcpf(den);
        if (!SIGMOID) along = grp_sum<G>(dot) * sum;
        dot = 0.f;
      }
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        if (id[q] < 0) continue;
        float v = sc[q] * sum * (c[q] - dot);
        if (SIGMOID) v *= one_minus(lc[q]);
        atomicAdd(mine + id[q], v);  // (an id is given once, or adds up)
      }
      wave_lds_fence();
    }
    float dl[VPL];
    if (losses) {
      float pa = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) pa = __builtin_fmaf(p[i], ga[i], pa);
      pa = grp_sum<G>(pa);
      const float more = (SIGMOID ? 0.f : gz * (r.top + __logf(den)) - along) - pa;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        dl[i] = p[i] * (ga[i] + more);
        if (SIGMOID && r.l[i] > -kInf) dl[i] *= one_minus(r.l[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) dl[i] = full ? -p[i] * along : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) dl[i] += mine[i * G + gl];
    wave_lds_fence();
    if (!in) continue;
    LT* out = (LT*)a.d_logits + t * E;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * G + gl;
      if (e < E) store1(out + e, r.live ? dl[i] + nan : 0.f);
    }
  }
}

// Whether up to 128 experts take 8 lanes per token instead of 16: twice the
// tokens per wave for one merge less (65536 tokens, k 8: 64 experts 11.2 -> 7.5
// us, 128 experts 11.8 -> 8.9), once there are enough tokens for four such
// waves per SIMD (8192 tokens of 128 experts: 6.8 us with 16, 7.8 with 8). A
// lane then holds one choice, so k is at most 8.
bool eight_lanes(int64_t T, int k) { return k <= 8 && T >= 32768; }

// Lanes per token and experts per lane for E experts: calls f(G, VPL) with
// both as compile-time constants.
template <bool EIGHT, typename F>
void with_layout(int E, F&& f) {
  using std::integral_constant;
  auto go = [&](auto g, auto v) { f(g, v); };
  if constexpr (EIGHT) {
    if (E <= 64) return go(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (E <= 128) return go(integral_constant<int, 8>{}, integral_constant<int, 16>{});
  } else {
    if (E <= 64) return go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if (E <= 128) return go(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  }
  if (E <= 256) go(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512) go(integral_constant<int, 16>{}, integral_constant<int, 32>{});
  else go(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

template <typename F>
void with_types(int fp32, int sigmoid, F&& f) {
  if (fp32)
    sigmoid ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
  else
    sigmoid ? f(uint16_t{}, std::true_type{}) : f(uint16_t{}, std::false_type{});
}

// Workgroup of the forward with statistics: one per compute unit, its LDS
// (one row of sums per wave) below 64 KiB and its registers enough at every E.
constexpr int stats_block(int E) { return E <= 256 ? 1024 : 512; }
constexpr int lanes_of(int E, bool eight) { return eight && E <= 128 ? 8 : E <= 512 ? 16 : 64; }
constexpr int kStatsParts = 256;

}  // namespace

// Workgroups of the forward with statistics, at most: a constant, so the
// order of the sums does not depend on the device.
static int64_t router_parts(int64_t T, int64_t E, bool eight) {
  const int64_t gpb = stats_block((int)E) / lanes_of((int)E, eight);
  return std::min<int64_t>((std::max<int64_t>(T, 1) + gpb - 1) / gpb, kStatsParts);
}
int64_t router_scratch_words(int64_t T, int64_t E) {  // (for every k: more lanes per token, more workgroups)
  return kStatsHead + router_parts(T, E, false) * 2 * (E + 1);
}

hipError_t launch_router(const RouterArgs& r, int cus, hipStream_t s) {
  RouterFwd a{r.logits, r.T, r.ld, r.E, r.k, r.bias, r.mask, r.sigmoid, r.renorm,
              !r.logits_fp32 && !r.bias, r.scale, r.weights, r.ids, r.part};
  const bool stats = r.counts != nullptr;
  if (r.T == 0 && !stats) return hipSuccess;
  const bool eight = eight_lanes(r.T, r.k);
  const int parts = (int)router_parts(r.T, r.E, eight);
  auto go = [&](auto tag, auto sig) {
    using LT = decltype(tag);
    constexpr bool SIG = decltype(sig)::value;
    auto run = [&](auto g, auto v, auto net) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value, NET = decltype(net)::value;
      if (stats) {
        constexpr int B = stats_block(G * V);
        const size_t lds = sizeof(float) * (size_t)(r.E + 1) * (1 + B / 64);
        router_rows<LT, G, V, B, true, SIG, NET><<<parts, B, lds, s>>>(a);
      } else {
        const int64_t gpb = 256 / G;
        const int grid = (int)std::min<int64_t>((r.T + gpb - 1) / gpb, (int64_t)cus * 64);
        router_rows<LT, G, V, 256, false, SIG, NET><<<grid, 256, 0, s>>>(a);
      }
    };
    if (eight)
      with_layout<true>(r.E, [&](auto g, auto v) { run(g, v, std::integral_constant<int, 8>{}); });
    else if (r.k <= 8)
      with_layout<false>(r.E, [&](auto g, auto v) { run(g, v, std::integral_constant<int, 8>{}); });
    else
      with_layout<false>(r.E, [&](auto g, auto v) { run(g, v, std::integral_constant<int, 16>{}); });
  };
  with_types(r.logits_fp32, r.sigmoid, go);
  MOK_HIP_TRY(hipGetLastError());
  if (stats) {
    router_stats<<<r.E / 16 + 1, 1024, 0, s>>>(r.part, parts, r.E, r.k, r.sigmoid, r.counts, r.losses);
    MOK_HIP_TRY(hipGetLastError());
  }
  return hipSuccess;
}

hipError_t launch_router_bwd(const RouterBwdArgs& r, int cus, hipStream_t s) {
  if (r.T == 0) return hipSuccess;
  RouterBwd a{r.logits, r.T,   r.ld,        r.E,   r.k,      r.bias,     r.mask,    r.sigmoid,
              r.renorm, r.scale, r.d_weights, r.ids, r.counts, r.d_losses, r.d_logits};
  auto go = [&](auto tag, auto sig) {
    using LT = decltype(tag);
    constexpr bool SIG = decltype(sig)::value;
    with_layout<false>(r.E, [&](auto g, auto v) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value;
      const int64_t gpb = 256 / G;
      const int grid = (int)std::min<int64_t>((r.T + gpb - 1) / gpb, (int64_t)cus * 8);
      if (r.k <= G)
        router_bwd_rows<LT, G, V, 256, SIG, 1><<<grid, 256, 0, s>>>(a);
      else if constexpr (G < 64)
        router_bwd_rows<LT, G, V, 256, SIG, 64 / G><<<grid, 256, 0, s>>>(a);
    });
  };
  with_types(r.logits_fp32, r.sigmoid, go);
  return hipGetLastError();
}

}  // namespace mok
