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
// A row with a NaN key or a +inf logit has no order: its ids are -1 and its
// weights NaN.
//
// Layout: a token belongs to 16 lanes (E <= 256) or to a whole wave, lane l
// holding experts l, l + 16, ... in registers, so a wave runs four tokens at
// once and every reduction over a token is four DPP instructions.
//
// The choice. Per token it costs instructions, not bytes, so it decides the
// kernel's time beyond about 64 experts. Up to k = 16 it is a sorting
// network on 32-bit words, the key's order-preserving bits with the lowest 8
// (10 with a wave per token) replaced by the complement of the expert id: a
// comparator is one max and one min, a lane sorts its experts' words to the
// 8 or 16 largest, and four merges with the lists of other lanes (max with a
// DPP operand, then a half-cleaner) leave the token's list in every lane.
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
// * log2(e) is an error of |x| 2^-24 of the value, no more than that of the
// rounded difference of logits that x is. -inf gives 0.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

template <int G>
__device__ __forceinline__ float grp_sum(float x) {
  if constexpr (G == 16) return row_sum(x);
  return wave_sum(x);
}
template <int G>
__device__ __forceinline__ float grp_max(float x) {
  if constexpr (G == 16) return row_max(x);
  return wave_max(x);
}
template <int G>
__device__ __forceinline__ int grp_min(int x) {
  if constexpr (G == 16) return row_min(x);
  return wave_min(x);
}

constexpr float kInf = __builtin_inff();
constexpr int kStatsHead = 64;  // words of the statistics' scratch before the partial rows

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

// Bits of a key in its order (larger key, larger word; both zeros alike).
__device__ __forceinline__ uint32_t ordered(float key) {
  const uint32_t u = f2u(key + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// The bits of a word that hold the complement of the expert id.
constexpr uint32_t word_ids(int G) { return G == 16 ? 255u : 1023u; }

// A token's logits and whether it is live or without an order.
template <typename LT, int G, int VPL, bool WORDS>
struct Row {
  static constexpr uint32_t kIds = word_ids(G);
  float l[VPL];
  uint32_t word[VPL];  // the keys' words for the network, 0 for -inf
  float top;   // largest logit
  bool live;   // kept by the mask, and some key above -inf or no order
  bool broken; // NaN key or +inf logit

  __device__ __forceinline__ void load(const LT* p, const float* bias, int E, int gl, bool keep) {
    float mk = -kInf;
    int bad = 0;
    top = -kInf;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * G + gl;
      l[i] = (keep && e < E) ? load1(p + e) : -kInf;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * G + gl;
      const float key = (bias && e < E) ? l[i] + bias[e] : l[i];
      bad |= !(key == key) | (l[i] == kInf);
      mk = __builtin_fmaxf(mk, key);
      if constexpr (WORDS) word[i] = key > -kInf ? (ordered(key) & ~kIds) | (kIds - (uint32_t)e) : 0u;
      top = __builtin_fmaxf(top, l[i]);
    }
    top = grp_max<G>(top);
    mk = grp_max<G>(mk);
    broken = grp_min<G>(-bad) < 0;
    live = broken || mk > -kInf;
  }
};

// Score of a logit up to a factor common to its token, from the token's
// largest logit `top` (for sigmoid at most 0): e^(l - top), or sigmoid(l) /
// e^top = e^(min(l, 0) - top) / (1 + e^-|l|), which is not 0 / 0 where every
// logit is far below 0. l = -inf gives 0.
__device__ __forceinline__ float score_of(float l, float top, int sigmoid) {
  if (!sigmoid) return exp_neg(l - top);
  return exp_neg(__builtin_fminf(l, 0.f) - top) / (1.f + exp_neg(-__builtin_fabsf(l)));
}
// 1 - sigmoid(l)
__device__ __forceinline__ float one_minus(float l) {
  return exp_neg(__builtin_fminf(-l, 0.f)) / (1.f + exp_neg(-__builtin_fabsf(l)));
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
// N words into descending order (bitonic sort).
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&w)[N]) {
#pragma unroll
  for (int size = 2; size <= N; size *= 2)
#pragma unroll
    for (int h = size / 2; h > 0; h /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & h) == 0) {
          const bool up = (i & size) != 0;  // this run ascends
          const uint32_t a = w[i], b = w[i + h];
          w[i] = up ? min(a, b) : max(a, b);
          w[i + h] = up ? max(a, b) : min(a, b);
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

// Choice gl of the token (-1: none) in lane gl of the group, for k <= N <=
// 16. False (for the whole wave) if some token's order hangs on key bits
// that the words do not keep.
template <int N, int G, int VPL>
__device__ __forceinline__ bool choose_network(const uint32_t (&word)[VPL], int gl, int k, bool exact, int& pick) {
  constexpr uint32_t kIds = word_ids(G);
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
  // rotations by 8, 4, 2, 1 pair lists of different lanes each time: after a
  // rotation by r, lanes r apart hold the same list
  merge_dpp<N, kRor8>(top);
  merge_dpp<N, kRor4>(top);
  merge_dpp<N, kRor2>(top);
  merge_dpp<N, kRor1>(top);
  if constexpr (G == 64) {
    merge_xor<N>(top, 16);
    merge_xor<N>(top, 32);
  }
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) mine = gl == j && j < k ? top[j] : mine;
  pick = mine ? (int)(kIds - (mine & kIds)) : -1;
  if (exact) return true;
  // the first word behind the k chosen
  uint32_t last = 0, behind = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) last = j == k - 1 ? top[j] : last;
#pragma unroll
  for (int i = 0; i < VPL; ++i) behind = max(behind, word[i] < last ? word[i] : 0u);
  bool close = behind != 0 && ((behind ^ last) & ~kIds) == 0;
#pragma unroll
  for (int j = 0; j + 1 < N; ++j) close |= j + 1 < k && top[j + 1] != 0 && ((top[j] ^ top[j + 1]) & ~kIds) == 0;
  return __ballot(close) == 0;
}

// STATS: the sums behind the losses and counts. A workgroup then keeps them
// in registers and LDS over its tokens and writes one partial row.
template <typename LT, int G, int VPL, int BLOCK, bool STATS>
__global__ void __launch_bounds__(BLOCK) router_rows(RouterFwd a) {
  constexpr int GPB = BLOCK / G;
  constexpr int KQ = 64 / G;  // choices a lane may hold (k <= 64)
  extern __shared__ float lds[];  // STATS: int cnt[E + 1], then float sums[waves][E + 1]
  const int E = a.E, k = a.k;
  const int gl = (int)threadIdx.x % G, group = (int)threadIdx.x / G;
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
    const bool keep = in && (!a.mask || a.mask[t]);
    const LT* row = (const LT*)a.logits + (in ? t : 0) * a.ld;
    Row<LT, G, VPL, true> r;
    r.load(row, a.bias, E, gl, keep);
    int pick[KQ];
#pragma unroll
    for (int q = 0; q < KQ; ++q) pick[q] = -1;
    bool done = false;
    if (k <= 8)
      done = choose_network<8, G, VPL>(r.word, gl, k, a.exact_words, pick[0]);
    else if (k <= 16)
      done = choose_network<16, G, VPL>(r.word, gl, k, a.exact_words, pick[0]);
    if (!done) {
      float key[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = i * G + gl;
        key[i] = (a.bias && e < E) ? r.l[i] + a.bias[e] : r.l[i];
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
    for (int q = 0; q < KQ; ++q) pick[q] = r.broken ? -1 : pick[q];
    // weights of the choices: lane j of the group holds choice j, j + G, ...
    const float nan = r.broken ? __builtin_nanf("") : 0.f;
    float w[KQ], ltop = -kInf;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      if (q * G >= k) break;
      w[q] = pick[q] >= 0 ? load1(row + pick[q]) : -kInf;
      ltop = __builtin_fmaxf(ltop, w[q]);
    }
    // the scores over all experts, where anything needs them
    float den = 0.f, score[VPL];
    const float ptop = a.sigmoid ? __builtin_fminf(r.top, 0.f) : r.top;
    if (STATS || (!a.sigmoid && !a.renorm)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        score[i] = score_of(r.l[i], ptop, a.sigmoid);
        den += score[i];
      }
      den = grp_sum<G>(den);
    }
    const float wtop = a.renorm ? grp_max<G>(ltop) : a.sigmoid ? 0.f : ptop;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      if (q * G >= k) break;
      w[q] = pick[q] < 0 ? 0.f : score_of(w[q], a.sigmoid ? __builtin_fminf(wtop, 0.f) : wtop, a.sigmoid);
      sum += w[q];
    }
    const float total = a.renorm ? grp_sum<G>(sum) : a.sigmoid ? 1.f : den;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      if (q * G >= k) break;
      const int j = q * G + gl;
      if (in && j < k) {
        const int64_t o = t * k + j;
        a.ids[o] = pick[q];
        a.weights[o] = (pick[q] >= 0 ? w[q] / total * a.scale : 0.f) + nan;
      }
      if (STATS && pick[q] >= 0) atomicAdd(cnt + pick[q], 1);  // integers: any order gives the same count
    }
    if constexpr (STATS) {
      if (r.live) {
        const float inv = 1.f / den + nan;
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
    // a wave's four tokens (or one), then the waves in order
    constexpr int WAVES = BLOCK / 64;
    float* sums = lds + (E + 1);
    const int wave = threadIdx.x >> 6, lane = lane_id();
    if constexpr (G == 16) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        psum[i] += __shfl_xor(psum[i], 16);
        psum[i] += __shfl_xor(psum[i], 32);
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane < G && i * G + gl < E) sums[wave * (E + 1) + i * G + gl] = psum[i];
    zsum = wave_sum(zsum);
    if (lane == 0) sums[wave * (E + 1) + E] = zsum;
    if (gl == 0 && nlive) atomicAdd(cnt + E, nlive);
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
// A workgroup takes 64 columns, 16 adders each; the one that finishes last
// (a counter that the launch before cleared) adds the columns' products in
// order, so one launch does both.
//
// The scratch: kStatsHead words, [0] the counter, [1 + b] workgroup b's sum
// of count_e * (sum of p_e), [32] the sum of lse^2, [33] the live tokens;
// then per workgroup of the forward 2 (E + 1) words, the sums of p and of
// lse^2 and the counts and live tokens.
__global__ void __launch_bounds__(1024) router_stats(float* part, int nparts, int E, int k, int sigmoid,
                                                     int32_t* counts, float* losses) {
  __shared__ float fs[16][64];
  __shared__ int is[16][64];
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int W = 2 * (E + 1);
  const int c = (int)blockIdx.x * 64 + lane;
  const float* rows = part + kStatsHead;
  float f = 0.f;
  int n = 0;
  if (c <= E)
#pragma unroll 8
    for (int r = g; r < nparts; r += 16) {
      f += rows[(int64_t)r * W + c];
      n += ((const int*)rows)[(int64_t)r * W + E + 1 + c];
    }
  fs[g][lane] = f;
  is[g][lane] = n;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) f += fs[i][lane], n += is[i][lane];
  if (c <= E) counts[c] = n;
  const float dot = wave_sum(c < E ? (float)n * f : 0.f);
  if (c == E) {
    __hip_atomic_store(part + 32, f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store((int*)part + 33, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (lane == 0) __hip_atomic_store(part + 1 + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  uint32_t done = 0;
  __threadfence();  // every lane's stores, before the count
  if (lane == 0) done = __hip_atomic_fetch_add((uint32_t*)part, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1;
  if (lane != 0 || done != gridDim.x) return;
  float s = 0.f;
  for (uint32_t b = 0; b < gridDim.x; ++b)
    s += __hip_atomic_load(part + 1 + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float z = __hip_atomic_load(part + 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float live = (float)max(__hip_atomic_load((int*)part + 33, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), 1);
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
template <typename LT, int G, int VPL, int BLOCK>
__global__ void __launch_bounds__(BLOCK) router_bwd_rows(RouterBwd a) {
  constexpr int GPB = BLOCK / G;
  constexpr int KQ = 64 / G;
  const int E = a.E, k = a.k;
  const int gl = (int)threadIdx.x % G, group = (int)threadIdx.x / G;
  const bool losses = a.counts != nullptr;
  float ga = 0.f, gz = 0.f;
  if (losses) {
    const float n = (float)max(a.counts[E], 1);
    ga = a.d_losses[0] * ((float)E / (float)k) / n / n;
    gz = a.sigmoid ? 0.f : a.d_losses[1] * 2.f / n;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < a.T; t0 += (int64_t)gridDim.x * GPB) {
    const int64_t t = t0 + group;
    const bool in = t < a.T;
    const bool keep = in && (!a.mask || a.mask[t]);
    const LT* row = (const LT*)a.logits + (in ? t : 0) * a.ld;
    Row<LT, G, VPL, false> r;
    r.load(row, a.bias, E, gl, keep);
    // the choices, one or more per lane; an id outside [0, E) has no gradient
    int id[KQ];
    float c[KQ], lc[KQ], ltop = -kInf;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      id[q] = -1;
      if (q * G >= k) break;
      const int j = q * G + gl;
      c[q] = 0.f;
      lc[q] = -kInf;
      if (keep && j < k) {
        const int64_t v = a.ids[t * k + j];
        if (v >= 0 && v < E) {
          id[q] = (int)v;
          c[q] = a.d_weights[t * k + j] * a.scale;
          lc[q] = load1(row + v);
        }
      }
      ltop = __builtin_fmaxf(ltop, lc[q]);
    }
    const float ptop = a.sigmoid ? __builtin_fminf(r.top, 0.f) : r.top;
    const float nan = r.broken ? __builtin_nanf("") : 0.f;
    float p[VPL], den = 0.f;
    const bool full = losses || (!a.sigmoid && !a.renorm);
    if (full) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        p[i] = score_of(r.l[i], ptop, a.sigmoid);
        den += p[i];
      }
      den = grp_sum<G>(den);
      const float inv = 1.f / den;
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] *= inv;
    }
    // c becomes the gradient to the chosen logits
    float along = 0.f;  // softmax without renormalisation: sum_j p_cj dw_j
    {
      const float wtop = a.renorm ? grp_max<G>(ltop) : a.sigmoid ? 0.f : ptop;
      float sc[KQ], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        if (q * G >= k) break;
        sc[q] = id[q] < 0 ? 0.f : score_of(lc[q], a.sigmoid ? __builtin_fminf(wtop, 0.f) : wtop, a.sigmoid);
        sum += sc[q];
        dot = __builtin_fmaf(sc[q], c[q], dot);
      }
      if (a.renorm) {
        sum = grp_sum<G>(sum);
        dot = sum > 0.f ? grp_sum<G>(dot) / sum : 0.f;
      } else if (!a.sigmoid) {
        along = grp_sum<G>(dot) / den;
      }
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        if (q * G >= k) break;
        if (id[q] < 0) continue;
        c[q] = a.renorm ? sc[q] / sum * (c[q] - dot) : a.sigmoid ? sc[q] * c[q] : sc[q] / den * c[q];
        if (a.sigmoid) c[q] *= one_minus(lc[q]);
      }
    }
    float dl[VPL];
    if (losses) {
      float pa = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = i * G + gl;
        dl[i] = e < E ? ga * (float)a.counts[e] : 0.f;
        pa = __builtin_fmaf(p[i], dl[i], pa);
      }
      pa = grp_sum<G>(pa);
      const float more = (a.sigmoid ? 0.f : gz * (r.top + __logf(den)) - along) - pa;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        dl[i] = p[i] * (dl[i] + more);
        if (a.sigmoid && r.l[i] > -kInf) dl[i] *= one_minus(r.l[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) dl[i] = full ? -p[i] * along : 0.f;
    }
    // each choice to the lane that owns its expert (a repeated id adds up)
#pragma unroll
    for (int q = 0; q < KQ; ++q)
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (q * G + j >= k) break;
        int e;
        float v;
        if constexpr (G == 16) {
          e = row_lane_of(id[q], j);
          v = u2f((uint32_t)row_lane_of((int)f2u(c[q]), j));
        } else {
          e = lane_value(id[q], j);
          v = lane_valuef(c[q], j);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) dl[i] += e == i * G + gl ? v : 0.f;
      }
    if (!in) continue;
    LT* out = (LT*)a.d_logits + t * E;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * G + gl;
      if (e < E) store1(out + e, r.live ? dl[i] + nan : 0.f);
    }
  }
}

// Lanes per token and experts per lane for E experts: calls f(G, VPL) with
// both as compile-time constants.
template <typename F>
void with_layout(int E, F&& f) {
  using std::integral_constant;
  auto go = [&](auto g, auto v) { f(g, v); };
  if (E <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (E <= 32) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else if (E <= 64) go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128) go(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256) go(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512) go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else go(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

// Workgroup of the forward with statistics, for G lanes per token: one per
// compute unit, its LDS (one row of sums per wave) below 64 KiB at every E.
constexpr int stats_block(int G) { return G == 16 ? 1024 : 512; }
constexpr int kStatsParts = 256;

}  // namespace

// Workgroups of the forward with statistics, at most: a constant, so the
// order of the sums does not depend on the device.
static int64_t router_parts(int64_t T, int64_t E) {
  const int64_t gpb = E <= 256 ? stats_block(16) / 16 : stats_block(64) / 64;
  return std::min<int64_t>((std::max<int64_t>(T, 1) + gpb - 1) / gpb, kStatsParts);
}
int64_t router_scratch_words(int64_t T, int64_t E) { return kStatsHead + router_parts(T, E) * 2 * (E + 1); }

hipError_t launch_router(const RouterArgs& r, int cus, hipStream_t s) {
  RouterFwd a{r.logits, r.T, r.ld, r.E, r.k, r.bias, r.mask, r.sigmoid, r.renorm,
              !r.logits_fp32 && !r.bias, r.scale, r.weights, r.ids, r.part};
  const bool stats = r.counts != nullptr;
  if (r.T == 0 && !stats) return hipSuccess;
  const int parts = (int)router_parts(r.T, r.E);
  auto go = [&](auto tag) {
    using LT = decltype(tag);
    with_layout(r.E, [&](auto g, auto v) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value;
      if (stats) {
        constexpr int B = stats_block(G);
        const size_t lds = sizeof(float) * (size_t)(r.E + 1) * (1 + B / 64);
        router_rows<LT, G, V, B, true><<<parts, B, lds, s>>>(a);
      } else {
        const int64_t gpb = 256 / G;
        const int grid = (int)std::min<int64_t>((r.T + gpb - 1) / gpb, (int64_t)cus * 64);
        router_rows<LT, G, V, 256, false><<<grid, 256, 0, s>>>(a);
      }
    });
  };
  r.logits_fp32 ? go(float{}) : go(uint16_t{});
  MOK_HIP_TRY(hipGetLastError());
  if (stats) {
    router_stats<<<r.E / 64 + 1, 1024, 0, s>>>(r.part, parts, r.E, r.k, r.sigmoid, r.counts, r.losses);
    MOK_HIP_TRY(hipGetLastError());
  }
  return hipSuccess;
}

hipError_t launch_router_bwd(const RouterBwdArgs& r, int cus, hipStream_t s) {
  if (r.T == 0) return hipSuccess;
  RouterBwd a{r.logits, r.T,   r.ld,        r.E,   r.k,      r.bias,     r.mask,    r.sigmoid,
              r.renorm, r.scale, r.d_weights, r.ids, r.counts, r.d_losses, r.d_logits};
  auto go = [&](auto tag) {
    using LT = decltype(tag);
    with_layout(r.E, [&](auto g, auto v) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value;
      const int64_t gpb = 256 / G;
      const int grid = (int)std::min<int64_t>((r.T + gpb - 1) / gpb, (int64_t)cus * 64);
      router_bwd_rows<LT, G, V, 256><<<grid, 256, 0, s>>>(a);
    });
  };
  r.logits_fp32 ? go(float{}) : go(uint16_t{});
  return hipGetLastError();
}

}  // namespace mok
