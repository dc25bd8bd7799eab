// Weights in 4 bits: quantized and read back, their product with few rows, and
// the layer's forward on 4-bit experts.
//
// The products are bound by reading the weights once, so every weight goes from
// memory straight into the registers of the one wave that multiplies it; LDS
// only joins the partial sums of the waves. They run on the 16 x 16 x 32 bf16
// matrix instruction with the rows of x (16 tokens) as its first operand and 16
// rows of the weight as its second: at up to 16 tokens most of its work is for
// rows that are not there, but it keeps far ahead of the memory, and one lane
// holds one weight row throughout (row lane % 16, its four-lane column kg =
// lane / 16), so scales and zero points are one load per lane.
//
// A wave works on chunks of 128 columns: 16 bytes of codes per lane, those of
// the 32 columns 32 kg .. 32 kg + 31.
//   int4: the dword exchange of the four lane rows gives every lane 8 columns of
//     each 32-column block, so that each matrix instruction stays within one
//     group, whatever its size. A code c becomes the bf16 128 + c by one OR (the
//     exact integer); the sum over a group is sum (128 + c) x, from which (128 +
//     zero) sum x is taken away in fp32 before the scale is applied. The sums of
//     x come from a matrix instruction with ones. The cancellation costs at most
//     5 of the 24 bits.
//   MXFP4: the scaled conversion of gfx950 turns two codes into two bf16 with
//     their block's scale, exactly: nothing is left to do but the product.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "mok_internal.h"

namespace mok {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32v4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32v2;

constexpr int kChunk = 128;  // columns of a wave's step

// One weight as a kernel sees it.
struct W4 {
  const uint8_t* codes;
  const void* scale;
  const uint8_t* zero;
};
W4 w4_of(const mok_w4& w) { return W4{w.codes, w.scale, w.zero}; }

// FMT: 0 int4 with the zero point 8, 1 int4 with zero points, 2 MXFP4.
constexpr int kSym = 0, kZero = 1, kMx = 2;

__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

#if defined(__HIP_DEVICE_COMPILE__)
// E8M0 byte as the fp32 that the scaled conversion takes.
__device__ __forceinline__ float e8m0(uint32_t b) { return b == 255 ? __builtin_nanf("") : u2f(b == 0 ? 0x00400000u : b << 23); }

// Eight MXFP4 codes of a dword as bf16, times scale.
__device__ __forceinline__ bf16x8 mx_values(uint32_t w, float scale) {
  typedef __attribute__((ext_vector_type(2))) __bf16 b2;
  const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const b2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const b2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Dword i of lane row kg becomes dword kg of lane row i (4 x 4 over the four
// rows of 16 lanes).
__device__ __forceinline__ void exchange(u32v4& w) {
  const u32v2 a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const u32v2 b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const u32v2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const u32v2 d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w = u32v4{c[0], c[1], d[0], d[1]};
}
#else
__device__ float e8m0(uint32_t b);
__device__ bf16x8 mx_values(uint32_t w, float scale);
__device__ void exchange(u32v4& w);
#endif

// Eight int4 codes of a dword as the bf16 integers 128 + c, in the order 0, 4,
// 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ bf16x8 int4_values(uint32_t w) {
  u32v4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, v);
}
// Eight bf16 in that order.
__device__ __forceinline__ bf16x8 int4_order(u32v4 x) {
  const u32v4 v{perm(x[2], x[0], 0x05040100u), perm(x[2], x[0], 0x07060302u), perm(x[3], x[1], 0x05040100u),
                perm(x[3], x[1], 0x07060302u)};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One lane's part of a chunk of 16 weight rows: codes, and the scales and zero
// points of the groups (MXFP4: of its own block).
template <int FMT, int G>
struct Chunk {
  static constexpr int NG = FMT == kMx ? 1 : kChunk / G;
  u32v4 codes;
  float scale[NG], zero[NG];

  // Row `row` of a weight of K columns at columns k0..; columns past K count as zeros (whatever the codes, x is 0).
  __device__ __forceinline__ void load(const W4& w, int64_t row, int k0, int K, int kg) {
    const int k = k0 + 32 * kg;
    const bool in = k < K;
    codes = u32v4{0, 0, 0, 0};
    if (in) codes = *reinterpret_cast<const u32v4*>(w.codes + row * (K / 2) + k / 2);
    if constexpr (FMT == kMx) {
      scale[0] = in ? e8m0(((const uint8_t*)w.scale)[row * (K / 32) + k / 32]) : 1.f;
    } else {
      const int groups = K / G;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int at = k0 / G + i;
        scale[i] = 0.f, zero[i] = 8.f;
        if (at < groups) {
          scale[i] = bf16_to_f32(((const uint16_t*)w.scale)[row * groups + at]);
          if (FMT == kZero) zero[i] = (float)w.zero[row * groups + at];
        }
      }
    }
  }
};

// One lane's x of a chunk: 16 tokens, four operands. In int4's order for int4,
// with the groups' sums of x; token `row` is null where there is none.
template <int FMT, int G>
struct Tokens {
  static constexpr int NG = FMT == kMx ? 1 : kChunk / G;
  bf16x8 v[4];
  f32x4 sum[NG];

  __device__ __forceinline__ void load(const uint16_t* row, int k0, int K, int kg) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + (FMT == kMx ? 32 * kg + 8 * j : 32 * j + 8 * kg);
      u32v4 x{0, 0, 0, 0};
      if (row && k < K) x = *reinterpret_cast<const u32v4*>(row + k);
      v[j] = FMT == kMx ? __builtin_bit_cast(bf16x8, x) : int4_order(x);
    }
    if constexpr (FMT != kMx) {
      const u32v4 ones{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4 / NG; ++j)
          sum[i] = mfma16(v[i * (4 / NG) + j], __builtin_bit_cast(bf16x8, ones), sum[i]);
      }
    }
  }
};

// The chunk's products out[t] = x_t . w for TT tiles of 16 tokens; tiles
// without their bit in `live` (the same in every lane) are left out.
template <int FMT, int G, int TT>
__device__ __forceinline__ void multiply(Chunk<FMT, G>& w, const Tokens<FMT, G> (&x)[TT], uint32_t live,
                                         f32x4 (&out)[TT]) {
#pragma unroll
  for (int t = 0; t < TT; ++t) out[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (FMT == kMx) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 b = mx_values(w.codes[j], w.scale[0]);
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (TT == 1 || (live >> t & 1)) out[t] = mfma16(x[t].v[j], b, out[t]);
    }
  } else {
    constexpr int NG = kChunk / G, PER = 4 / NG;
    exchange(w.codes);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      f32x4 acc[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const bf16x8 b = int4_values(w.codes[i * PER + j]);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (TT == 1 || (live >> t & 1)) acc[t] = mfma16(x[t].v[i * PER + j], b, acc[t]);
      }
      const float off = 128.f + w.zero[i];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) out[t][r] += w.scale[i] * (acc[t][r] - off * x[t].sum[i][r]);
    }
  }
}

// ---------------------------------------------------------------------------
// y = x W^T: a workgroup takes 16 rows of the weight and 16 TT tokens, its
// waves the chunks in turn.
// ---------------------------------------------------------------------------
template <int FMT, int G, int TT, int NW>
__global__ void __launch_bounds__(NW * 64)
w4_product(const uint16_t* x, int64_t ld_x, int T, int64_t n, int K, W4 w, uint16_t* y, int64_t ld_y) {
  __shared__ f32x4 part[NW][TT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kg = lane >> 4, li = lane & 15;
  const int64_t row = min((int64_t)blockIdx.x * 16 + li, n - 1);
  const int t0 = blockIdx.y * (16 * TT);
  f32x4 sum[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * kChunk; k0 < K; k0 += NW * kChunk) {
    Chunk<FMT, G> c;
    c.load(w, row, k0, K, kg);
    Tokens<FMT, G> xs[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int tok = t0 + 16 * t + li;
      xs[t].load(tok < T ? x + tok * ld_x : nullptr, k0, K, kg);
    }
    f32x4 v[TT];
    multiply<FMT, G, TT>(c, xs, ~0u, v);
#pragma unroll
    for (int t = 0; t < TT; ++t) sum[t] += v[t];
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) part[wave][t][lane] = sum[t];
  __syncthreads();
  for (int i = threadIdx.x; i < TT * 256; i += NW * 64) {  // token i / 16, weight row i % 16
    const int t = i >> 8, tok = (i >> 4) & 15, at = (tok >> 2) * 16 + (i & 15);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) v += part[q][t][at][tok & 3];
    const int64_t col = (int64_t)blockIdx.x * 16 + (i & 15);
    if (t0 + (i >> 4) < T && col < n) y[(t0 + (i >> 4)) * ld_y + col] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// The layer
// ---------------------------------------------------------------------------
struct Layer {
  int H, I, Is, E, k, T;
  float limit;
  W4 gate, up, down, sgate, sup, sdown;
  const uint16_t* x;
  const float* rw;
  const int64_t* ids;
  uint16_t* h;   // [T k, I], then [T, Is]
  uint16_t* out;
};

__device__ __forceinline__ int choice(const Layer& p, int pair) {
  const int64_t e = p.ids[pair];
  return e >= 0 && e < p.E ? (int)e : -1;
}

// h of one expert's rows: 16 columns of I per workgroup. blockIdx.y numbers the
// distinct experts among the ids (in order), the shared expert behind them.
template <int FMT, int G, int TT, int NW>
__global__ void __launch_bounds__(NW * 64) w4_gate_up(Layer p) {
  __shared__ f32x4 part[2][NW][TT][64];
  __shared__ uint32_t seen[32];
  __shared__ int count;
  extern __shared__ uint8_t dyn[];
  uint16_t* list = (uint16_t*)dyn;  // [T k] the expert's pairs
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, kg = lane >> 4, li = lane & 15;
  const int pairs = p.T * p.k;
  const int slots = min(p.E, pairs);
  const bool shared = (int)blockIdx.y == slots;
  int e = 0, rows = p.T;
  if (!shared) {
    if (tid < 32) seen[tid] = 0;
    if (tid == 0) count = 0;
    __syncthreads();
    for (int i = tid; i < pairs; i += NW * 64) {
      const int c = choice(p, i);
      if (c >= 0) atomicOr(&seen[c >> 5], 1u << (c & 31));
    }
    __syncthreads();
    // the blockIdx.y-th expert seen
    int left = blockIdx.y;
    e = -1;
    for (int q = 0; q < 32; ++q) {
      uint32_t bits = seen[q];
      const int c = __popc(bits);
      if (left < c) {
        for (; left > 0; --left) bits &= bits - 1;
        e = 32 * q + __ffs(bits) - 1;
        break;
      }
      left -= c;
    }
    if (e < 0) return;  // fewer experts than slots: the whole workgroup
    // its pairs, in any order: a row's h does not depend on its place
    for (int i = tid; i < pairs; i += NW * 64)
      if (choice(p, i) == e) list[atomicAdd(&count, 1)] = (uint16_t)i;
    __syncthreads();
    rows = count;
  }
  const int I = shared ? p.Is : p.I, K = p.H;
  const int n0 = blockIdx.x * 16;
  if (n0 >= I) return;
  const int64_t row = (shared ? 0 : (int64_t)e * I) + min(n0 + li, I - 1);
  const W4 wg = shared ? p.sgate : p.gate, wu = shared ? p.sup : p.up;
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    f32x4 g[TT], u[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) g[t] = u[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* xr[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int r = r0 + 16 * t + li;
      xr[t] = r < rows ? p.x + (int64_t)(shared ? r : list[r] / p.k) * K : nullptr;
    }
    for (int k0 = wave * kChunk; k0 < K; k0 += NW * kChunk) {
      Chunk<FMT, G> cg, cu;
      cg.load(wg, row, k0, K, kg);
      cu.load(wu, row, k0, K, kg);
      Tokens<FMT, G> xs[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) xs[t].load(xr[t], k0, K, kg);
      f32x4 v[TT];
      multiply<FMT, G, TT>(cg, xs, ~0u, v);
#pragma unroll
      for (int t = 0; t < TT; ++t) g[t] += v[t];
      multiply<FMT, G, TT>(cu, xs, ~0u, v);
#pragma unroll
      for (int t = 0; t < TT; ++t) u[t] += v[t];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) part[0][wave][t][lane] = g[t], part[1][wave][t][lane] = u[t];
    __syncthreads();
    for (int i = tid; i < TT * 256; i += NW * 64) {
      const int t = i >> 8, tok = (i >> 4) & 15, at = (tok >> 2) * 16 + (i & 15);
      float vg = 0.f, vu = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) vg += part[0][q][t][at][tok & 3], vu += part[1][q][t][at][tok & 3];
      const int r = r0 + (i >> 4), col = n0 + (i & 15);
      if (r < rows && col < I) {
        const float lg = fminf(vg, p.limit), lu = fminf(fmaxf(vu, -p.limit), p.limit);
        const float v = lg / (1.f + __expf(-lg)) * lu;
        uint16_t* h = shared ? p.h + (int64_t)pairs * p.I + (int64_t)r * I : p.h + (int64_t)list[r] * I;
        h[col] = f32_to_bf16(v);
      }
    }
    __syncthreads();
  }
}

// LDS of the output kernel besides its partial sums: weights and coefficients
// [NT][k] fp32, ids [NT][k], and a byte for every (distinct expert, token).
size_t down_lds(int nt, int k, int E) {
  return (size_t)nt * k * (4 + 4 + 2) + (size_t)std::min(E, nt * k) * nt;
}

// The output: 16 columns of H for 16 TT tokens per workgroup. Its work is every
// chunk of every distinct expert of these tokens, and of the shared expert,
// taken by the waves in turn. A token's row of h is that of its first choice of
// the expert (zeros if it has none), and the chunk's result goes to the token's
// sum times the router weight of its choices of the expert. So a token's sums
// are added in a fixed order, and no other launch joins them.
template <int FMT, int G, int TT, int NW>
__global__ void __launch_bounds__(NW * 64) w4_down(Layer p) {
  constexpr int NT = 16 * TT;
  __shared__ f32x4 part[NW][TT][64];
  __shared__ uint32_t seen[32];
  __shared__ int before[33];
  __shared__ int16_t expert[1024];
  extern __shared__ uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = lane >> 4,
            li = lane & 15;
  const int t0 = blockIdx.y * NT, nt = min(NT, p.T - t0), pairs = nt * p.k;
  float* given = (float*)dyn;
  float* coef = given + NT * p.k;
  int16_t* id = (int16_t*)(coef + NT * p.k);
  uint8_t* slot = (uint8_t*)(id + NT * p.k);  // 1 + the token's first choice of the expert, 0: none
  if (tid < 32) seen[tid] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += NW * 64) {
    const int c = choice(p, t0 * p.k + i);
    id[i] = (int16_t)c;
    given[i] = p.rw[t0 * p.k + i];
    if (c >= 0) atomicOr(&seen[c >> 5], 1u << (c & 31));
  }
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int q = 0; q < 32; ++q) before[q] = n, n += __popc(seen[q]);
    before[32] = n;
  }
  __syncthreads();
  const int distinct = before[32];
  auto place = [&](int e) { return before[e >> 5] + __popc(seen[e >> 5] & ((1u << (e & 31)) - 1)); };
  for (int i = tid; i < distinct * NT / 4; i += NW * 64) ((uint32_t*)slot)[i] = 0;
  for (int e = tid; e < p.E; e += NW * 64)
    if (seen[e >> 5] >> (e & 31) & 1) expert[place(e)] = (int16_t)e;
  __syncthreads();
  for (int i = tid; i < pairs; i += NW * 64) {
    const int e = id[i], t = i / p.k, b = t * p.k;
    if (e < 0) continue;
    float sum = 0.f;
    bool first = true;
    for (int j = b; j < b + p.k; ++j)
      if (id[j] == e) {
        sum += given[j];
        first = first && j >= i;
      }
    if (first) {
      coef[i] = sum;
      slot[place(e) * NT + t] = (uint8_t)(i - b + 1);
    }
  }
  __syncthreads();

  const int64_t col = min((int)blockIdx.x * 16 + li, p.H - 1);
  const int C = (p.I + kChunk - 1) / kChunk, routed = distinct * C;
  const int units = routed + (p.Is + kChunk - 1) / kChunk;
  f32x4 sum[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int q = wave; q < units; q += NW) {
    Chunk<FMT, G> c;
    Tokens<FMT, G> xs[TT];
    f32x4 v[TT];
    if (q < routed) {
      const int at = q / C, k0 = (q - at * C) * kChunk, e = expert[at];
      c.load(p.down, (int64_t)e * p.H + col, k0, p.I, kg);
      uint32_t live = 0;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int tok = 16 * t + li, s = slot[at * NT + tok];
        if (__ballot(s != 0) != 0) live |= 1u << t;
        const int64_t pair = (int64_t)(t0 + tok) * p.k + s - 1;
        xs[t].load(s ? p.h + pair * p.I : nullptr, k0, p.I, kg);
      }
      multiply<FMT, G, TT>(c, xs, live, v);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t s4 = *(const uint32_t*)(slot + at * NT + 16 * t + 4 * kg);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = s4 >> (8 * r) & 255;
          // (not 0 times v: another token's expert may hold what is not finite)
          if (s) sum[t][r] += coef[(16 * t + 4 * kg + r) * p.k + s - 1] * v[t][r];
        }
      }
    } else {
      const int k0 = (q - routed) * kChunk;
      c.load(p.sdown, col, k0, p.Is, kg);
      const uint16_t* hs = p.h + (int64_t)p.T * p.k * p.I;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int tok = 16 * t + li;
        xs[t].load(tok < nt ? hs + (int64_t)(t0 + tok) * p.Is : nullptr, k0, p.Is, kg);
      }
      multiply<FMT, G, TT>(c, xs, ~0u, v);
#pragma unroll
      for (int t = 0; t < TT; ++t) sum[t] += v[t];
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) part[wave][t][lane] = sum[t];
  __syncthreads();
  for (int i = tid; i < TT * 256; i += NW * 64) {
    const int t = i >> 8, tok = (i >> 4) & 15, at = (tok >> 2) * 16 + (i & 15);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += part[w][t][at][tok & 3];
    const int c = blockIdx.x * 16 + (i & 15);
    if ((i >> 4) < nt && c < p.H) p.out[(int64_t)(t0 + (i >> 4)) * p.H + c] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// Quantizing and reading back: eight elements per lane, a group's lanes side by
// side in one wave.
// ---------------------------------------------------------------------------
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

template <typename T, int FMT, int G>
__global__ void __launch_bounds__(256)
w4_quantize(const T* src, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, void* scale, uint8_t* zero) {
  constexpr int LANES = G / 8;
  const int64_t per = cols / 8, all = rows * per;
  // (whole waves go round together; lanes past the end hold zeros and store nothing)
  const int64_t step = (int64_t)gridDim.x * 256, end = (all + 63) / 64 * 64;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += step) {
    const bool in = i < all;
    const int64_t row = in ? i / per : 0, at = in ? i - row * per : 0;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (in) {
      const T* s = src + row * ld + at * 8;
      if constexpr (sizeof(T) == 4) {
        *(f32x4*)v = *(const f32x4*)s;
        *(f32x4*)(v + 4) = *(const f32x4*)(s + 4);
      } else {
        const u32v4 w = *(const u32v4*)s;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = u2f(w[j] << 16), v[2 * j + 1] = u2f(w[j] & 0xFFFF0000u);
      }
    }
    uint32_t out = 0;
    const int64_t group = row * (cols / G) + at * 8 / G;
    const bool first = in && threadIdx.x % LANES == 0;
    if constexpr (FMT == kMx) {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      amax = group_max<LANES>(amax);
      int x = -127;
      if (amax > 0.f) x = max(-127, floor_log2_bits(f2u(amax)) - 2);
      if (first) ((uint8_t*)scale)[group] = (uint8_t)(x + 127);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = __builtin_ldexpf(fabsf(v[j]), -x);
        // halves below 2, whole numbers below 4, even ones above, 6 at most
        const float q = a < 2.f ? rintf(a * 2.f) : a < 4.f ? rintf(a) + 2.f : fminf(rintf(a * 0.5f) + 4.f, 7.f);
        out |= ((uint32_t)q | (f2u(v[j]) >> 28 & 8u)) << (4 * j);
      }
    } else {
      float sc, z = 8.f, lowest = 0.f;
      if constexpr (FMT == kZero) {
        float hi = 0.f, lo = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) hi = fmaxf(hi, v[j]), lo = fmaxf(lo, -v[j]);
        hi = group_max<LANES>(hi), lo = group_max<LANES>(lo);
        sc = bf16_to_f32(f32_to_bf16((hi + lo) / 15.f));
        z = sc > 0.f ? fminf(rintf(lo / sc), 15.f) : 0.f;
        if (first) zero[group] = (uint8_t)z;
      } else {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
        sc = bf16_to_f32(f32_to_bf16(group_max<LANES>(amax) / 7.f));
      }
      if (first) ((uint16_t*)scale)[group] = (uint16_t)(f2u(sc) >> 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = sc > 0.f ? fminf(fmaxf(rintf(v[j] / sc) + z, lowest), 15.f) : z;
        out |= (uint32_t)q << (4 * j);
      }
    }
    if (in) *(uint32_t*)(codes + i * 4) = out;
  }
}

template <int FMT>
__global__ void __launch_bounds__(256)
w4_dequantize(W4 w, int64_t elements, int G, uint16_t* dst) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < elements / 8; i += (int64_t)gridDim.x * 256) {
    const uint32_t c = *(const uint32_t*)(w.codes + i * 4);
    const int64_t group = i * 8 / G;
    if constexpr (FMT == kMx) {
      *(bf16x8*)(dst + i * 8) = mx_values(c, e8m0(((const uint8_t*)w.scale)[group]));
    } else {
      const float sc = bf16_to_f32(((const uint16_t*)w.scale)[group]);
      const float z = FMT == kZero ? (float)w.zero[group] : 8.f;
      u32v4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(((float)(c >> (8 * j) & 15) - z) * sc, ((float)(c >> (8 * j + 4) & 15) - z) * sc);
      *(u32v4*)(dst + i * 8) = o;
    }
  }
}

// f(format, group) as constants.
template <typename F>
void with_format(int format, int group, bool zero, F&& f) {
  using std::integral_constant;
  auto grouped = [&](auto fmt) {
    if (group == 32)
      f(fmt, integral_constant<int, 32>{});
    else if (group == 64)
      f(fmt, integral_constant<int, 64>{});
    else
      f(fmt, integral_constant<int, 128>{});
  };
  if (format == MOK_W4_MXFP4)
    f(integral_constant<int, kMx>{}, integral_constant<int, 32>{});
  else if (zero)
    grouped(integral_constant<int, kZero>{});
  else
    grouped(integral_constant<int, kSym>{});
}

}  // namespace

hipError_t launch_w4_quantize(const void* src, int src_fp32, int64_t rows, int64_t cols, int64_t ld, int format,
                              int group, uint8_t* codes, void* scale, uint8_t* zero, hipStream_t s) {
  const int grid = (int)std::min<int64_t>((rows * cols / 8 + 255) / 256, 1 << 20);
  with_format(format, group, zero != nullptr, [&](auto fmt, auto g) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    if (src_fp32)
      w4_quantize<float, FMT, G><<<grid, 256, 0, s>>>((const float*)src, rows, cols, ld, codes, scale, zero);
    else
      w4_quantize<uint16_t, FMT, G><<<grid, 256, 0, s>>>((const uint16_t*)src, rows, cols, ld, codes, scale, zero);
  });
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(const mok_w4& w, int64_t rows, int64_t cols, int format, int group, void* dst,
                                hipStream_t s) {
  const int64_t n = rows * cols;
  const int grid = (int)std::min<int64_t>((n / 8 + 255) / 256, 1 << 20);
  uint16_t* d = (uint16_t*)dst;
  if (format == MOK_W4_MXFP4)
    w4_dequantize<kMx><<<grid, 256, 0, s>>>(w4_of(w), n, group, d);
  else if (w.zero)
    w4_dequantize<kZero><<<grid, 256, 0, s>>>(w4_of(w), n, group, d);
  else
    w4_dequantize<kSym><<<grid, 256, 0, s>>>(w4_of(w), n, group, d);
  return hipGetLastError();
}

hipError_t launch_w4_matmul(const void* x, int64_t ld_x, int64_t T, int64_t n, int64_t k, int format, int group,
                            const mok_w4& w, void* y, int64_t ld_y, hipStream_t s) {
  const int slabs = (int)((n + 15) / 16);
  with_format(format, group, w.zero != nullptr, [&](auto fmt, auto g) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    if (T <= 16)
      w4_product<FMT, G, 1, 8><<<dim3(slabs, 1), 512, 0, s>>>((const uint16_t*)x, ld_x, (int)T, n, (int)k, w4_of(w),
                                                            (uint16_t*)y, ld_y);
    else
      w4_product<FMT, G, 4, 8><<<dim3(slabs, (T + 63) / 64), 512, 0, s>>>((const uint16_t*)x, ld_x, (int)T, n, (int)k,
                                                                        w4_of(w), (uint16_t*)y, ld_y);
  });
  return hipGetLastError();
}

size_t w4_layer_scratch(const mok_w4_layer& l, int64_t T) {
  return (size_t)std::max<int64_t>(1, T * ((int64_t)l.topk * l.intermediate + l.shared_intermediate)) * 2;
}

hipError_t launch_w4_layer(const mok_w4_layer& l, const void* x, const float* router_w, const int64_t* ids, int64_t T,
                           void* out, void* scratch, hipStream_t s) {
  Layer p{};
  p.H = l.hidden, p.I = l.intermediate, p.Is = l.shared_intermediate, p.E = l.num_experts, p.k = l.topk, p.T = (int)T;
  p.limit = l.swiglu_limit > 0.f ? l.swiglu_limit : __builtin_inff();
  p.gate = w4_of(l.routed_gate), p.up = w4_of(l.routed_up), p.down = w4_of(l.routed_down);
  p.sgate = w4_of(l.shared_gate), p.sup = w4_of(l.shared_up), p.sdown = w4_of(l.shared_down);
  p.x = (const uint16_t*)x, p.rw = router_w, p.ids = ids, p.h = (uint16_t*)scratch, p.out = (uint16_t*)out;
  const int pairs = p.T * p.k, slots = std::min(p.E, pairs);
  const dim3 up((std::max(p.I, p.Is) + 15) / 16, slots + (p.Is > 0 ? 1 : 0));
  const int slabs = (p.H + 15) / 16;
  with_format(l.format, l.group, l.routed_gate.zero != nullptr, [&](auto fmt, auto g) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    w4_gate_up<FMT, G, 1, 8><<<up, 512, (size_t)pairs * 2, s>>>(p);
    if (p.T <= 16 || p.E > 256)
      w4_down<FMT, G, 1, 8><<<dim3(slabs, (p.T + 15) / 16), 512, down_lds(16, p.k, p.E), s>>>(p);
    else
      w4_down<FMT, G, 4, 8><<<dim3(slabs, (p.T + 63) / 64), 512, down_lds(64, p.k, p.E), s>>>(p);
  });
  return hipGetLastError();
}

}  // namespace mok
