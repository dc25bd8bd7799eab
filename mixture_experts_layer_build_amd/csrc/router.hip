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
// once and every reduction over a token is four DPP instructions. The k
// choices are k rounds of (largest key, lowest id that has it, take it out).
// Bound by HBM for small k; the rounds cost about 5 instructions per expert
// held by a lane, so at 16 experts per lane and k = 8 they weigh as much as
// the loads.
#include <algorithm>
#include <type_traits>

#include "mok_internal.h"
#include "wave_ops.h"

namespace mok {
namespace {

// exp(x) for x <= 0 within 2 ulp: the rounding error of x * log2(e) is put
// back as a factor 1 + lo * ln 2 (the hardware exponential alone would lose
// |x| / 2 ulp). Below -150 the result is 0 in fp32.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
  x = __builtin_fmaxf(x, -150.0f);
  const float t = x * kLog2e;
  const float lo = __builtin_fmaf(x, kLog2e, -t);
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, lo * kLn2, e);
}

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

struct RouterFwd {
  const void* logits;
  int64_t T, ld;
  int E, k;
  const float* bias;      // null: none
  const uint8_t* mask;    // null: every token
  int sigmoid, renorm;
  float scale;
  float* weights;
  int64_t* ids;
  float* part;            // [workgroups][2 (E + 1)]: sums of p and of lse^2, then counts and live tokens
};

// A token's logits and whether it is live or without an order.
template <typename LT, int G, int VPL>
struct Row {
  float l[VPL];
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
      top = __builtin_fmaxf(top, l[i]);
    }
    top = grp_max<G>(top);
    mk = grp_max<G>(mk);
    broken = grp_min<G>(-bad) < 0;
    live = broken || mk > -kInf;
  }
};

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
    Row<LT, G, VPL> r;
    r.load(row, a.bias, E, gl, keep);
    float key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * G + gl;
      key[i] = r.broken ? -kInf : (a.bias && e < E) ? r.l[i] + a.bias[e] : r.l[i];
    }
    int pick[KQ];
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
    // weights of the choices: lane j of the group holds choice j, j + G, ...
    float w[KQ], ltop = -kInf;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      w[q] = pick[q] >= 0 ? load1(row + pick[q]) : -kInf;
      ltop = __builtin_fmaxf(ltop, w[q]);
    }
    ltop = grp_max<G>(ltop);
    // the scores over all experts, where anything needs them
    float den = 0.f, score[VPL];
    const float ptop = a.sigmoid ? __builtin_fminf(r.top, 0.f) : r.top;
    if (STATS || (!a.sigmoid && !a.renorm)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float l = r.l[i];
        // sigmoid(l) / e^ptop = e^(min(l, 0) - ptop) / (1 + e^-|l|): no 0 / 0 where every logit is far below 0
        score[i] = l == -kInf ? 0.f
                   : a.sigmoid ? exp_neg(__builtin_fminf(l, 0.f) - ptop) / (1.f + exp_neg(-__builtin_fabsf(l)))
                               : exp_neg(l - ptop);
        den += score[i];
      }
      den = grp_sum<G>(den);
    }
    const float wtop = a.sigmoid ? __builtin_fminf(ltop, 0.f) : ltop;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const float l = w[q];
      if (pick[q] < 0)
        w[q] = 0.f;
      else if (a.sigmoid)
        w[q] = exp_neg(__builtin_fminf(l, 0.f) - (a.renorm ? wtop : 0.f)) / (1.f + exp_neg(-__builtin_fabsf(l)));
      else
        w[q] = exp_neg(l - (a.renorm ? wtop : ptop));
      sum += w[q];
    }
    const float total = a.renorm ? grp_sum<G>(sum) : a.sigmoid ? 1.f : den;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const int j = q * G + gl;
      if (in && j < k) {
        const int64_t o = t * k + j;
        a.ids[o] = pick[q];
        a.weights[o] = r.broken ? __builtin_nanf("") : pick[q] >= 0 ? w[q] / total * a.scale : 0.f;
      }
      if (STATS && pick[q] >= 0) atomicAdd(cnt + pick[q], 1);  // integers: any order gives the same count
    }
    if constexpr (STATS) {
      if (r.live) {
        const float nan = r.broken ? __builtin_nanf("") : 0.f;
        const float inv = 1.f / den;
#pragma unroll
        for (int i = 0; i < VPL; ++i) psum[i] += score[i] * inv + nan;
        if (gl == 0) {
          const float lse = r.top + __logf(den) + nan;
          zsum += lse * lse;
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
    float* part = a.part + (int64_t)blockIdx.x * 2 * (E + 1);
    for (int i = threadIdx.x; i <= E; i += BLOCK) {
      float s = 0.f;
#pragma unroll
      for (int wv = 0; wv < WAVES; ++wv) s += sums[wv * (E + 1) + i];
      part[i] = s;
      ((int*)part)[E + 1 + i] = cnt[i];
    }
  }
}

// Adds the workgroups' partial rows in a fixed order and forms the losses.
// One workgroup; a column has 1024 / 64 = 16 adders.
__global__ void __launch_bounds__(1024) router_stats(const float* __restrict__ part, int nparts, int E, int k,
                                                     int sigmoid, int32_t* counts, float* losses) {
  __shared__ float fs[16][64];
  __shared__ int is[16][64];
  __shared__ float pc[1025];
  __shared__ int ic[1025];
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int W = 2 * (E + 1);
  for (int c0 = 0; c0 <= E; c0 += 64) {
    const int c = c0 + lane;
    float f = 0.f;
    int n = 0;
    if (c <= E)
#pragma unroll 4
      for (int r = g; r < nparts; r += 16) {
        f += part[(int64_t)r * W + c];
        n += ((const int*)part)[(int64_t)r * W + E + 1 + c];
      }
    fs[g][lane] = f;
    is[g][lane] = n;
    __syncthreads();
    if (g == 0 && c <= E) {
#pragma unroll
      for (int i = 1; i < 16; ++i) f += fs[i][lane], n += is[i][lane];
      pc[c] = f;
      ic[c] = n;
      counts[c] = n;
    }
    __syncthreads();
  }
  if (threadIdx.x >= 64) return;
  float s = 0.f;
  for (int c = lane; c < E; c += 64) s = __builtin_fmaf((float)ic[c], pc[c], s);
  s = wave_sum(s);
  if (lane == 0) {
    const float n = (float)max(ic[E], 1);
    losses[0] = s / n / n * ((float)E / (float)k);
    losses[1] = sigmoid ? 0.f : pc[E] / n;
  }
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
  const int base = (lane_id() / G) * G;  // the group's first lane in the wave
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
    Row<LT, G, VPL> r;
    r.load(row, a.bias, E, gl, keep);
    // the choices, one or more per lane; an id outside [0, E) has no gradient
    int id[KQ];
    float c[KQ], lc[KQ], ltop = -kInf;
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      const int j = q * G + gl;
      id[q] = -1;
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
    ltop = grp_max<G>(ltop);
    const float ptop = a.sigmoid ? __builtin_fminf(r.top, 0.f) : r.top;
    const float nan = r.broken ? __builtin_nanf("") : 0.f;
    float p[VPL], den = 0.f;
    const bool full = losses || (!a.sigmoid && !a.renorm);
    if (full) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float l = r.l[i];
        p[i] = l == -kInf ? 0.f
               : a.sigmoid ? exp_neg(__builtin_fminf(l, 0.f) - ptop) / (1.f + exp_neg(-__builtin_fabsf(l)))
                           : exp_neg(l - ptop);
        den += p[i];
      }
      den = grp_sum<G>(den);
      const float inv = 1.f / den;
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = p[i] * inv + nan;
    }
    // c becomes the gradient to the chosen logits
    float along = 0.f;  // softmax without renormalisation: sum_j p_cj dw_j
    {
      const float wtop = a.sigmoid ? __builtin_fminf(ltop, 0.f) : ltop;
      float sc[KQ], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        const float l = lc[q];
        sc[q] = id[q] < 0 ? 0.f
                : a.sigmoid ? exp_neg(__builtin_fminf(l, 0.f) - (a.renorm ? wtop : 0.f)) / (1.f + exp_neg(-__builtin_fabsf(l)))
                : a.renorm  ? exp_neg(l - wtop)
                            : exp_neg(l - ptop) / den;
        sum += sc[q];
        dot = __builtin_fmaf(sc[q], c[q], dot);
      }
      if (a.renorm) {
        sum = grp_sum<G>(sum);
        dot = sum > 0.f ? grp_sum<G>(dot) / sum : 0.f;
      } else if (!a.sigmoid) {
        along = grp_sum<G>(dot);
      }
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        if (id[q] < 0) continue;
        if (a.renorm) c[q] = sc[q] / sum * (c[q] - dot);
        else c[q] *= sc[q];
        if (a.sigmoid) {  // 1 - sigmoid(l) = e^(min(-l, 0)) / (1 + e^-|l|)
          const float l = lc[q];
          c[q] *= exp_neg(__builtin_fminf(-l, 0.f)) / (1.f + exp_neg(-__builtin_fabsf(l)));
        }
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
      const float zl = a.sigmoid ? 0.f : gz * (r.top + __logf(den));
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float l = r.l[i];
        float d = p[i] * (dl[i] - pa + zl);
        if (a.sigmoid && l > -kInf) d *= exp_neg(__builtin_fminf(-l, 0.f)) / (1.f + exp_neg(-__builtin_fabsf(l)));
        dl[i] = d - p[i] * along;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) dl[i] = full ? -p[i] * along : 0.f;
    }
    // each choice to the lane that owns its expert (a repeated id adds up)
#pragma unroll
    for (int q = 0; q < KQ; ++q)
      for (int j = 0; j < G; ++j) {
        if (q * G + j >= k) break;
        const int e = __shfl(id[q], base + j);
        const float v = __shfl(c[q], base + j);
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

constexpr int kStatsBlock = 512, kStatsParts = 256;

}  // namespace

// Workgroups of the forward with statistics, at most: a constant, so the
// order of the sums does not depend on the device.
int64_t router_parts(int64_t T, int64_t E) {
  const int64_t gpb = kStatsBlock / (E <= 256 ? 16 : 64);
  return std::min<int64_t>((std::max<int64_t>(T, 1) + gpb - 1) / gpb, kStatsParts);
}

hipError_t launch_router(const RouterArgs& r, int cus, hipStream_t s) {
  RouterFwd a{r.logits, r.T, r.ld, r.E, r.k, r.bias, r.mask, r.sigmoid, r.renorm, r.scale, r.weights, r.ids, r.part};
  const bool stats = r.counts != nullptr;
  if (r.T == 0 && !stats) return hipSuccess;
  const int parts = (int)router_parts(r.T, r.E);
  auto go = [&](auto tag) {
    using LT = decltype(tag);
    with_layout(r.E, [&](auto g, auto v) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value;
      if (stats) {
        const size_t lds = sizeof(float) * (size_t)(r.E + 1) * (1 + kStatsBlock / 64);
        router_rows<LT, G, V, kStatsBlock, true><<<parts, kStatsBlock, lds, s>>>(a);
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
    router_stats<<<1, 1024, 0, s>>>(r.part, parts, r.E, r.k, r.sigmoid, r.counts, r.losses);
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
