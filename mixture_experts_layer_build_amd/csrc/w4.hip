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

// One lane's part of a chunk of 16 weight rows, as loaded: codes, and the scales
// and zero points of the chunk's groups (MXFP4: the scale of its own block).
template <int FMT, int G>
struct Chunk {
  static constexpr int NG = FMT == kMx ? 1 : kChunk / G;
  u32v4 codes;
  uint32_t sc[(NG + 1) / 2], z;

  // Row `row` of a weight of K columns at columns k0..; `whole`: K is a multiple of the chunk and the scales and zero
  // points are aligned to a chunk's. Columns past K stand for zeros.
  __device__ __forceinline__ void load(const W4& w, int64_t row, int k0, int K, int kg, bool whole) {
    const int k = k0 + 32 * kg;
    const bool in = k < K;
    codes = u32v4{0, 0, 0, 0};
    if (in) codes = *reinterpret_cast<const u32v4*>(w.codes + row * (K / 2) + k / 2);
    z = 0;
    if constexpr (FMT == kMx) {
      sc[0] = in ? ((const uint8_t*)w.scale)[row * (K / 32) + k / 32] : 127;
    } else {
      const int groups = K / G, at = k0 / G;
      const uint16_t* s = (const uint16_t*)w.scale + row * groups + at;
      const uint8_t* zp = FMT == kZero ? w.zero + row * groups + at : nullptr;
      if (NG > 1 && whole) {
        if constexpr (NG == 4) {
          const u32v2 v = *reinterpret_cast<const u32v2*>(s);
          sc[0] = v[0], sc[1] = v[1];
          if (FMT == kZero) z = *reinterpret_cast<const uint32_t*>(zp);
        } else if constexpr (NG == 2) {
          sc[0] = *reinterpret_cast<const uint32_t*>(s);
          if (FMT == kZero) z = *reinterpret_cast<const uint16_t*>(zp);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if (i % 2 == 0) sc[i / 2] = 0;
          if (at + i < groups) {
            sc[i / 2] |= (uint32_t)s[i] << (16 * (i % 2));
            if (FMT == kZero) z |= (uint32_t)zp[i] << (8 * i);
          }
        }
      }
    }
  }
  __device__ __forceinline__ float scale(int i) const {
    return i % 2 ? u2f(sc[i / 2] & 0xFFFF0000u) : u2f(sc[i / 2] << 16);
  }
  // 128 + the zero point of group i
  __device__ __forceinline__ float offset(int i) const {
    return FMT == kZero ? 128.f + (float)(z >> (8 * i) & 255) : 136.f;
  }
};

// One lane's x of a chunk, as loaded: four operands of a row (null: zeros).
// ORDERED: the row is stored in the order of int4_values.
struct TokenChunk {
  u32v4 v[4];
  template <int FMT>
  __device__ __forceinline__ void load(const uint16_t* row, int k0, int K, int kg) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + (FMT == kMx ? 32 * kg + 8 * j : 32 * j + 8 * kg);
      v[j] = u32v4{0, 0, 0, 0};
      if (row && k < K) v[j] = *reinterpret_cast<const u32v4*>(row + k);
    }
  }
};

// x of a chunk as the products take it: the operands in int4's order, and for
// int4 the groups' sums of x.
template <int FMT, int G>
struct Tokens {
  static constexpr int NG = FMT == kMx ? 1 : kChunk / G;
  bf16x8 v[4];
  f32x4 sum[NG];

  template <bool ORDERED>
  __device__ __forceinline__ void set(const TokenChunk& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = FMT == kMx || ORDERED ? __builtin_bit_cast(bf16x8, x.v[j]) : int4_order(x.v[j]);
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

// The chunk's products x_t . w for TT tiles of 16 rows of x in P parts each
// (whose sum x is), added to out.
template <int FMT, int G, int TT, int P>
__device__ __forceinline__ void multiply(Chunk<FMT, G> w, const Tokens<FMT, G> (&x)[TT][P], f32x4 (&out)[TT]) {
  if constexpr (FMT == kMx) {
    const float scale = e8m0(w.sc[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 b = mx_values(w.codes[j], scale);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int q = 0; q < P; ++q) out[t] = mfma16(x[t][q].v[j], b, out[t]);
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
#pragma unroll
          for (int q = 0; q < P; ++q) acc[t] = mfma16(x[t][q].v[i * PER + j], b, acc[t]);
      }
      const float scale = w.scale(i), off = w.offset(i);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float sum = x[t][0].sum[i][r];
#pragma unroll
          for (int q = 1; q < P; ++q) sum += x[t][q].sum[i][r];
          out[t][r] += scale * (acc[t][r] - off * sum);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// y = x W^T: a workgroup takes 16 NS rows of the weight and 16 TT rows of x,
// its waves the chunks in turn; the next chunk's weights are loaded before a
// chunk is multiplied.
// ---------------------------------------------------------------------------
template <int FMT, int G, int TT, int NS, int NW>
__global__ void __launch_bounds__(NW * 64)
w4_product(const uint16_t* x, int64_t ld_x, int T, int64_t n, int K, W4 w, bool whole, uint16_t* y, int64_t ld_y) {
  __shared__ f32x4 part[NW][NS][TT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kg = lane >> 4, li = lane & 15;
  const int t0 = blockIdx.y * (16 * TT);
  int64_t row[NS];
  const uint16_t* xr[TT];
#pragma unroll
  for (int s = 0; s < NS; ++s) row[s] = min((int64_t)blockIdx.x * (16 * NS) + 16 * s + li, n - 1);
#pragma unroll
  for (int t = 0; t < TT; ++t) xr[t] = t0 + 16 * t + li < T ? x + (t0 + 16 * t + li) * ld_x : nullptr;
  f32x4 sum[NS][TT];
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int t = 0; t < TT; ++t) sum[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  int k0 = wave * kChunk;
  Chunk<FMT, G> c[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) c[s].load(w, row[s], k0, K, kg, whole && k0 < K);
  for (; k0 < K; k0 += NW * kChunk) {
    TokenChunk xc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xc[t].template load<FMT>(xr[t], k0, K, kg);
    Chunk<FMT, G> next[NS];
    const int k1 = k0 + NW * kChunk;
#pragma unroll
    for (int s = 0; s < NS; ++s) next[s].load(w, row[s], k1, K, kg, whole && k1 < K);
    Tokens<FMT, G> xs[TT][1];
#pragma unroll
    for (int t = 0; t < TT; ++t) xs[t][0].template set<false>(xc[t]);
#pragma unroll
    for (int s = 0; s < NS; ++s) multiply<FMT, G, TT, 1>(c[s], xs, sum[s]);
#pragma unroll
    for (int s = 0; s < NS; ++s) c[s] = next[s];
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave][s][t][lane] = sum[s][t];
  __syncthreads();
  for (int i = threadIdx.x; i < NS * TT * 256; i += NW * 64) {  // weight row i % 16 of its sixteen, row of x i / 16
    const int s = i / (TT * 256), at16 = i % (TT * 256), t = at16 >> 8, tok = (at16 >> 4) & 15;
    const int at = (tok >> 2) * 16 + (i & 15);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) v += part[q][s][t][at][tok & 3];
    const int64_t col = (int64_t)blockIdx.x * (16 * NS) + 16 * s + (i & 15);
    if (t0 + (at16 >> 4) < T && col < n) y[(t0 + (at16 >> 4)) * ld_y + col] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// The layer: h of every choice, then the output. h is kept as two bf16 that add
// up to it (16 bits of it): the matrix instructions take bf16, and one alone
// would double the output's error. It is stored in the order of int4_values.
// ---------------------------------------------------------------------------
struct Layer {
  int H, I, Is, E, k, T;
  float limit;
  W4 gate, up, down, sgate, sup, sdown;
  bool whole_h, whole_i, whole_s;  // whole chunks along hidden, intermediate, shared intermediate
  const uint16_t* x;
  const float* rw;
  const int64_t* ids;
  uint16_t* h;  // [T k][2][I], then [T][2][Is]
  float* y;     // [T k + T][H]
  uint16_t* out;
};

__device__ __forceinline__ int choice(const Layer& p, int pair) {
  const int64_t e = p.ids[pair];
  return e >= 0 && e < p.E ? (int)e : -1;
}

// LDS of the choices sorted by expert, in row tiles of 16.
size_t plan_lds(const Layer& p) {
  const size_t pairs = (size_t)p.T * p.k, tiles = std::min<size_t>(p.E, pairs) + pairs / 16;
  return (p.E + tiles) * 4 + pairs * 4;
}

struct Plan {
  int routed, tiles;   // row tiles of the routed experts; with the shared expert's behind them
  const int* tile;     // expert << 18 | (rows - 1) << 14 | first choice in the list
  const uint16_t* list;

  // The same list in every workgroup: an expert's choices in their own order, since which of them share a row tile
  // must not depend on who asks.
  template <int NTHR>
  __device__ __forceinline__ void build(const Layer& p, uint8_t* lds, int (&part)[NTHR / 64 + 1]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, pairs = p.T * p.k;
    int* cursor = (int*)lds;  // [E]: count, then where the expert's next choice goes, then its end
    int* to = cursor + p.E;
    uint16_t* any = (uint16_t*)(to + min(p.E, pairs) + pairs / 16);
    uint16_t* out = any + pairs;
    for (int e = tid; e < p.E; e += NTHR) cursor[e] = 0;
    __syncthreads();
    for (int i = tid; i < pairs; i += NTHR) {
      const int e = choice(p, i);
      if (e >= 0) atomicAdd(&cursor[e], 1);
    }
    int base = 0;  // rows | tiles << 16 of the experts before
    for (int e0 = 0; e0 < p.E; e0 += NTHR) {
      __syncthreads();
      const int e = e0 + tid, rows = e < p.E ? cursor[e] : 0, tiles_e = (rows + 15) / 16;
      const int mine = rows | tiles_e << 16;
      int s = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(s, d);
        if (lane >= d) s += v;
      }
      if (lane == 63) part[wave] = s;
      __syncthreads();
      int before = base, all = base;
      for (int w = 0; w < NTHR / 64; ++w) {
        if (w < wave) before += part[w];
        all += part[w];
      }
      before += s - mine;
      const int r0 = before & 0xFFFF, t0 = before >> 16;
      if (e < p.E) cursor[e] = r0;
      for (int q = 0; q < tiles_e; ++q) to[t0 + q] = e << 18 | (min(16, rows - 16 * q) - 1) << 14 | (r0 + 16 * q);
      base = all;
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += NTHR) {
      const int e = choice(p, i);
      if (e >= 0) any[atomicAdd(&cursor[e], 1)] = (uint16_t)i;
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += NTHR) {
      const int e = choice(p, i);
      if (e < 0) continue;
      const int first = e > 0 ? cursor[e - 1] : 0, end = cursor[e];
      int at = first;
      for (int q = first; q < end; ++q) at += any[q] < i;
      out[at] = (uint16_t)i;
    }
    __syncthreads();
    routed = base >> 16;
    tiles = routed + (p.Is > 0 ? (p.T + 15) / 16 : 0);
    tile = to, list = out;
  }
};

// A row tile: its expert (-1: the shared one) and this lane's choice (T k + the
// token for the shared expert), -1 past its rows.
struct RowTile {
  int e, rows, first;
  bool shared;
  __device__ __forceinline__ void get(const Plan& l, int i, int T) {
    shared = i >= l.routed;
    if (shared) {
      e = 0, first = 16 * (i - l.routed), rows = min(16, T - first);
    } else {
      const int v = __builtin_amdgcn_readfirstlane(l.tile[i]);
      e = v >> 18, rows = (v >> 14 & 15) + 1, first = v & 0x3FFF;
    }
  }
  __device__ __forceinline__ int pair(const Plan& l, int r, int pairs) const {
    return r >= rows ? -1 : shared ? pairs + first + r : l.list[first + r];
  }
};

// The element of int4_values' order that element i of eight goes to.
__device__ __forceinline__ int ordered(int i) { return (i & 3) * 2 + (i >> 2); }

// h: items of one row tile and 16 columns of I, taken in turn by the
// workgroups; a workgroup's waves take the item's chunks in turn, the next
// step's weights and x on their way while one is multiplied.
template <int FMT, int G, int NW>
__global__ void __launch_bounds__(NW * 64) w4_gate_up(Layer p) {
  __shared__ f32x4 part[2][NW][64];
  __shared__ int scan[NW + 1];
  extern __shared__ uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = lane >> 4,
            li = lane & 15;
  Plan l;
  l.build<NW * 64>(p, dyn, scan);
  const int pairs = p.T * p.k, K = p.H;
  const int slabs_r = (p.I + 15) / 16, slabs_s = (p.Is + 15) / 16;
  const int items_r = l.routed * slabs_r, items = items_r + (l.tiles - l.routed) * slabs_s;
  const int steps = (K + NW * kChunk - 1) / (NW * kChunk);  // of an item, for each wave

  struct Step {
    Chunk<FMT, G> g, u;
    TokenChunk x;
  };
  RowTile t;
  int n0 = 0;
  auto item = [&](int i) {
    const bool sh = i >= items_r;
    const int v = sh ? i - items_r : i, slabs = sh ? slabs_s : slabs_r;
    t.get(l, (sh ? l.routed : 0) + v / slabs, p.T);
    n0 = v % slabs * 16;
  };
  const uint16_t* xr = nullptr;
  int64_t row = 0;
  auto begin = [&] {
    const int pr = t.pair(l, li, pairs), wide = t.shared ? p.Is : p.I;
    xr = pr < 0 ? nullptr : p.x + (int64_t)(t.shared ? pr - pairs : pr / p.k) * K;
    row = (int64_t)t.e * wide + min(n0 + li, wide - 1);
  };
  auto load = [&](Step& s, int st) {
    const int k0 = (st * NW + wave) * kChunk;
    const bool whole = p.whole_h && k0 < K;
    const W4 wg = t.shared ? p.sgate : p.gate, wu = t.shared ? p.sup : p.up;
    s.g.load(wg, row, k0, K, kg, whole);
    s.u.load(wu, row, k0, K, kg, whole);
    s.x.template load<FMT>(xr, k0, K, kg);
  };
  int i = blockIdx.x;
  if (i >= items) return;
  Step cur;
  item(i);
  begin();
  load(cur, 0);
  while (true) {
    f32x4 g[1]{f32x4{0.f, 0.f, 0.f, 0.f}}, u[1]{f32x4{0.f, 0.f, 0.f, 0.f}};
    const RowTile done = t;
    const int col0 = n0, following = i + gridDim.x;
    for (int st = 0; st < steps; ++st) {
      Step next;
      if (st + 1 < steps) {
        load(next, st + 1);
      } else if (following < items) {
        item(following);
        begin();
        load(next, 0);
      }
      Tokens<FMT, G> xs[1][1];
      xs[0][0].template set<false>(cur.x);
      multiply<FMT, G, 1, 1>(cur.g, xs, g);
      multiply<FMT, G, 1, 1>(cur.u, xs, u);
      cur = next;
    }
    part[0][wave][lane] = g[0], part[1][wave][lane] = u[0];
    __syncthreads();
    if (tid < 256) {  // row tid / 16, column tid % 16
      const int r = tid >> 4, c = tid & 15, at = (r >> 2) * 16 + c;
      float vg = 0.f, vu = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) vg += part[0][q][at][r & 3], vu += part[1][q][at][r & 3];
      const int pr = done.pair(l, r, pairs), wide = done.shared ? p.Is : p.I, col = col0 + c;
      if (pr >= 0 && col < wide) {
        const float lg = fminf(vg, p.limit), lu = fminf(fmaxf(vu, -p.limit), p.limit);
        const float v = lg / (1.f + __expf(-lg)) * lu;
        const uint16_t hi = f32_to_bf16(v), lo = f32_to_bf16(v - bf16_to_f32(hi));
        uint16_t* h = p.h + (done.shared ? (int64_t)pairs * 2 * p.I + (int64_t)(pr - pairs) * 2 * p.Is
                                         : (int64_t)pr * 2 * p.I);
        const int to = FMT == kMx ? col : (col & ~7) + ordered(col & 7);
        h[to] = hi, h[wide + to] = lo;
      }
    }
    if (following >= items) break;
    i = following;
    __syncthreads();
  }
}

// y of every choice and of the shared expert: items as above, of 16 columns of H.
template <int FMT, int G, int NW>
__global__ void __launch_bounds__(NW * 64) w4_down(Layer p) {
  __shared__ f32x4 part[NW][64];
  __shared__ int scan[NW + 1];
  extern __shared__ uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = lane >> 4,
            li = lane & 15;
  Plan l;
  l.build<NW * 64>(p, dyn, scan);
  const int pairs = p.T * p.k, slabs = (p.H + 15) / 16, items = l.tiles * slabs;
  struct Step {
    Chunk<FMT, G> w;
    TokenChunk x[2];
  };
  RowTile t;
  int n0 = 0, K = 0;
  const uint16_t* hr = nullptr;
  int64_t row = 0;
  auto begin = [&](int i) {
    t.get(l, i / slabs, p.T);
    n0 = i % slabs * 16;
    K = t.shared ? p.Is : p.I;
    const int pr = t.pair(l, li, pairs);
    hr = pr < 0 ? nullptr
         : t.shared ? p.h + (int64_t)pairs * 2 * p.I + (int64_t)(pr - pairs) * 2 * p.Is
                    : p.h + (int64_t)pr * 2 * p.I;
    row = (int64_t)t.e * p.H + min(n0 + li, p.H - 1);
  };
  auto steps = [&] { return (K + NW * kChunk - 1) / (NW * kChunk); };
  auto load = [&](Step& s, int st) {
    const int k0 = (st * NW + wave) * kChunk;
    s.w.load(t.shared ? p.sdown : p.down, row, k0, K, kg, (t.shared ? p.whole_s : p.whole_i) && k0 < K);
#pragma unroll
    for (int q = 0; q < 2; ++q) s.x[q].template load<FMT>(hr ? hr + q * K : nullptr, k0, K, kg);
  };
  int i = blockIdx.x;
  if (i >= items) return;
  Step cur;
  begin(i);
  load(cur, 0);
  while (true) {
    f32x4 y[1]{f32x4{0.f, 0.f, 0.f, 0.f}};
    const RowTile done = t;
    const int col0 = n0, following = i + gridDim.x, n = steps();
    for (int st = 0; st < n; ++st) {
      Step next;
      if (st + 1 < n) {
        load(next, st + 1);
      } else if (following < items) {
        begin(following);
        load(next, 0);
      }
      Tokens<FMT, G> xs[1][2];
      xs[0][0].template set<true>(cur.x[0]);
      xs[0][1].template set<true>(cur.x[1]);
      multiply<FMT, G, 1, 2>(cur.w, xs, y);
      cur = next;
    }
    part[wave][lane] = y[0];
    __syncthreads();
    for (int j = tid; j < 256; j += NW * 64) {
      const int r = j >> 4, c = j & 15, at = (r >> 2) * 16 + c;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) v += part[q][at][r & 3];
      const int pr = done.pair(l, r, pairs);
      if (pr >= 0 && col0 + c < p.H) p.y[(int64_t)pr * p.H + col0 + c] = v;
    }
    if (following >= items) break;
    i = following;
    __syncthreads();
  }
}

// The output: a token's choices in their order, then the shared expert's.
__global__ void __launch_bounds__(256) w4_combine(Layer p) {
  const int t = blockIdx.y;
  const float* y = p.y + (int64_t)t * p.k * p.H;
  for (int c = blockIdx.x * 256 + threadIdx.x; c < p.H; c += gridDim.x * 256) {
    float v = 0.f;
    for (int j = 0; j < p.k; ++j)
      if (choice(p, t * p.k + j) >= 0) v += p.rw[t * p.k + j] * y[(int64_t)j * p.H + c];
    if (p.Is > 0) v += p.y[((int64_t)p.T * p.k + t) * p.H + c];
    p.out[(int64_t)t * p.H + c] = f32_to_bf16(v);
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

// Whether rows of `k` elements are whole chunks whose scales and zero points can be loaded at once.
static bool whole_chunks(const mok_w4& w, int64_t k, int group) {
  const uintptr_t most = 2 * (kChunk / group);
  return k % kChunk == 0 && (uintptr_t)w.scale % most == 0 && (uintptr_t)w.zero % (most / 2) == 0;
}

hipError_t launch_w4_matmul(const void* x, int64_t ld_x, int64_t T, int64_t n, int64_t k, int format, int group,
                            const mok_w4& w, void* y, int64_t ld_y, hipStream_t s) {
  const bool whole = whole_chunks(w, k, group);
  with_format(format, group, w.zero != nullptr, [&](auto fmt, auto g) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    if (T <= 16)
      w4_product<FMT, G, 1, 1, 8><<<dim3((unsigned)((n + 15) / 16), 1), 512, 0, s>>>(
          (const uint16_t*)x, ld_x, (int)T, n, (int)k, w4_of(w), whole, (uint16_t*)y, ld_y);
    else
      w4_product<FMT, G, 4, 2, 8><<<dim3((unsigned)((n + 31) / 32), (unsigned)((T + 63) / 64)), 512, 0, s>>>(
          (const uint16_t*)x, ld_x, (int)T, n, (int)k, w4_of(w), whole, (uint16_t*)y, ld_y);
  });
  return hipGetLastError();
}

static size_t h_elements(const mok_w4_layer& l, int64_t T) {
  const size_t n = (size_t)T * 2 * ((size_t)l.topk * l.intermediate + l.shared_intermediate);
  return (n + 7) / 8 * 8;
}
size_t w4_layer_scratch(const mok_w4_layer& l, int64_t T) {
  return std::max<size_t>(16, h_elements(l, T) * 2 + (size_t)T * (l.topk + 1) * l.hidden * 4);
}

hipError_t launch_w4_layer(const mok_w4_layer& l, const void* x, const float* router_w, const int64_t* ids, int64_t T,
                           void* out, void* scratch, int cus, hipStream_t s) {
  Layer p{};
  p.H = l.hidden, p.I = l.intermediate, p.Is = l.shared_intermediate, p.E = l.num_experts, p.k = l.topk, p.T = (int)T;
  p.limit = l.swiglu_limit > 0.f ? l.swiglu_limit : __builtin_inff();
  p.gate = w4_of(l.routed_gate), p.up = w4_of(l.routed_up), p.down = w4_of(l.routed_down);
  p.sgate = w4_of(l.shared_gate), p.sup = w4_of(l.shared_up), p.sdown = w4_of(l.shared_down);
  const bool sh = p.Is > 0;
  auto whole = [&](const mok_w4& w, int k) { return whole_chunks(w, k, l.group); };
  p.whole_h = whole(l.routed_gate, p.H) && whole(l.routed_up, p.H) &&
              (!sh || (whole(l.shared_gate, p.H) && whole(l.shared_up, p.H)));
  p.whole_i = whole(l.routed_down, p.I), p.whole_s = sh && whole(l.shared_down, p.Is);
  p.x = (const uint16_t*)x, p.rw = router_w, p.ids = ids, p.h = (uint16_t*)scratch, p.out = (uint16_t*)out;
  p.y = (float*)((uint16_t*)scratch + h_elements(l, T));
  const int pairs = p.T * p.k, tiles = std::min(p.E, pairs) + pairs / 16, shared = sh ? (p.T + 15) / 16 : 0;
  const int64_t up = (int64_t)tiles * ((p.I + 15) / 16) + (int64_t)shared * ((p.Is + 15) / 16);
  const int64_t down = (int64_t)(tiles + shared) * ((p.H + 15) / 16);
  const size_t lds = plan_lds(p);
  with_format(l.format, l.group, l.routed_gate.zero != nullptr, [&](auto fmt, auto g) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    w4_gate_up<FMT, G, 8><<<(unsigned)std::min<int64_t>(up, 2 * cus), 512, lds, s>>>(p);
    w4_down<FMT, G, 4><<<(unsigned)std::min<int64_t>(down, 4 * cus), 256, lds, s>>>(p);
  });
  w4_combine<<<dim3((p.H + 255) / 256, p.T), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace mok
