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
// lane / 16), so scales and zero points are one value per lane.
//
// A wave works on chunks of 128 columns: 16 bytes of codes per lane. Loads are
// made with four neighbouring lanes side by side in one row (row lane / 4), and
// the registers are then moved to the lanes of the matrix instruction
// (ds_bpermute): with neighbouring lanes in different rows the address unit,
// which takes four lanes of 16 bytes at a time, was busy four times as long and
// bound the layer (64 tokens, 128 experts of 768 x 2048: 130 us).
//   A lane then has the codes of the 32 columns 32 kg .. 32 kg + 31; an exchange
//     between the four lane rows gives it 8 columns of each 32-column block, so
//     that each matrix instruction stays within one group, whatever its size.
//   int4: a code c becomes the bf16 16 + c by a shift and an AND with OR (the
//     exact integer: 16 is the smallest base whose significand has c's four bits
//     free); the sum over a group is sum (16 + c) x, from which (16 + zero) sum x
//     is taken away in fp32 before the scale is applied. The sums of x come from
//     a matrix instruction with ones. The sums round at (16 + c) |x| where the
//     result's terms are |c - zero| |x|: 12 times as much for normally
//     distributed weights in groups of 128 (3.6 of the 24 bits; 8 bits where one
//     outlier sets a group's scale), without bound where most codes are the zero
//     point's.
//   MXFP4: the scaled conversion of gfx950 turns two codes into two bf16 with
//     their block's scale, exactly: nothing is left to do but the product.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "mok_internal.h"
#include "wave_ops.h"

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

// Eight int4 codes of a dword as the bf16 integers 16 + c, in the order 0, 4, 1,
// 5, 2, 6, 3, 7.
__device__ __forceinline__ bf16x8 int4_values(uint32_t w) {
  u32v4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ((i == 0 ? w << 3 : w >> (4 * i - 3)) & 0x00780078u) | 0x41804180u;
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

// The lane (as a byte address) that loads what this lane multiplies.
__device__ __forceinline__ int source_lane(int lane) { return ((lane & 15) * 4 + (lane >> 4)) * 4; }
__device__ __forceinline__ uint32_t from_lane(int src, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute(src, (int)v);
}

// One lane's part of a chunk of 16 weight rows, as loaded: codes, and the scales
// and zero points of the chunk's groups.
// WHOLE: rows are whole chunks, and their scales and zero points aligned to a
// chunk's (one load). Nothing in a load branches or looks at what it gets: with a
// fixed number of loads the compiler waits for a chunk's own ones, not for those
// of the next chunk.
// Columns past the row's end stand for zeros: the last ones are read again, with
// a scale of 0 (MXFP4: codes of 0).
template <int FMT, int G, bool WHOLE>
struct Chunk {
  static constexpr int NG = kChunk / G;  // groups
  static constexpr int NS = WHOLE ? (FMT != kMx && NG == 4 ? 2 : 1) : NG, NZ = FMT == kZero ? (WHOLE ? 1 : NG) : 0;
  u32v4 codes;
  uint32_t s[NS], z[NZ > 0 ? NZ : 1];

  // Row `row` of a weight of K columns at columns k0 and on; kq: this lane's quarter of them.
  __device__ __forceinline__ void load(const W4& w, int64_t row, int k0, int K, int kq) {
    const int k = min(k0 + 32 * kq, K - 32), groups = K / G;
    codes = *reinterpret_cast<const u32v4*>(w.codes + row * (K / 2) + k / 2);
    const int at = min(k0, K - (WHOLE ? kChunk : G)) / G;
    if constexpr (FMT == kMx) {
      const uint8_t* p = (const uint8_t*)w.scale + row * groups;
      if constexpr (WHOLE) {
        s[0] = *reinterpret_cast<const uint32_t*>(p + at);
      } else {
#pragma unroll
        for (int i = 0; i < NG; ++i) s[i] = p[min(at + i, groups - 1)];
      }
    } else {
      const uint16_t* p = (const uint16_t*)w.scale + row * groups;
      if constexpr (!WHOLE) {
#pragma unroll
        for (int i = 0; i < NG; ++i) s[i] = p[min(at + i, groups - 1)];
      } else if constexpr (NG == 4) {
        const u32v2 v = *reinterpret_cast<const u32v2*>(p + at);
        s[0] = v[0], s[1] = v[1];
      } else if constexpr (NG == 2) {
        s[0] = *reinterpret_cast<const uint32_t*>(p + at);
      } else {
        s[0] = p[at];
      }
      if constexpr (FMT == kZero) {
        const uint8_t* q = w.zero + row * groups;
        if constexpr (!WHOLE) {
#pragma unroll
          for (int i = 0; i < NG; ++i) z[i] = q[min(at + i, groups - 1)];
        } else if constexpr (NG == 4) {
          z[0] = *reinterpret_cast<const uint32_t*>(q + at);
        } else if constexpr (NG == 2) {
          z[0] = *reinterpret_cast<const uint16_t*>(q + at);
        } else {
          z[0] = q[at];
        }
      }
    }
  }
  // Moves it to the lanes that multiply it.
  __device__ __forceinline__ void arrange(int src, int k0, int K) {
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[i] = from_lane(src, codes[i]);
    exchange(codes);
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = from_lane(src, s[i]);
#pragma unroll
    for (int i = 0; i < NZ; ++i) z[i] = from_lane(src, z[i]);
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (k0 + i * G < K) continue;
        if (FMT == kMx)
          codes[i] = 0;
        else
          s[i] = 0;
      }
    }
  }
  // (arranged) of group i: the scale, and 16 + the zero point
  __device__ __forceinline__ float scale(int i) const {
    if (FMT == kMx) return e8m0(WHOLE ? s[0] >> (8 * i) & 255 : s[i]);
    if (!WHOLE) return u2f(s[i] << 16);
    return i % 2 ? u2f(s[i / 2] & 0xFFFF0000u) : u2f(s[i / 2] << 16);
  }
  __device__ __forceinline__ float offset(int i) const {
    return FMT == kZero ? 16.f + (float)(WHOLE ? z[0] >> (8 * i) & 255 : z[i]) : 24.f;
  }
};

// One lane's x of a chunk: four operands of a row, 8 columns of each block of
// 32. Columns past the row's end repeat its last block (the weight's are zeros
// there).
struct TokenChunk {
  u32v4 v[4];
  __device__ __forceinline__ void load(const uint16_t* row, int k0, int K, int kq) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const u32v4*>(row + min(k0 + 32 * j, K - 32) + 8 * kq);
  }
  // From h, which lies as it is multiplied (a block after the other). Rows past the tile's repeat its last one, which
  // costs no traffic.
  __device__ __forceinline__ void load_blocks(const uint16_t* tile, int k0, int K, int lane, int rows) {
    const int at = (lane & 48) + min(lane & 15, rows - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<const u32v4*>(tile + (int64_t)(min(k0 / 32 + j, K / 32 - 1) * 64 + at) * 8);
  }
  __device__ __forceinline__ void arrange(int src) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = from_lane(src, v[j][i]);
  }
};

// x of a chunk in P parts (whose sum x is) as the products take it: the operands
// in int4's order (ORDERED: they are in it), and for int4 the groups' sums of x.
template <int FMT, int G, int P>
struct Tokens {
  static constexpr int NG = FMT == kMx ? 1 : kChunk / G;
  bf16x8 v[P][4];
  f32x4 sum[NG];

  template <bool ORDERED>
  __device__ __forceinline__ void set(int q, const TokenChunk& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[q][j] = FMT == kMx || ORDERED ? __builtin_bit_cast(bf16x8, x.v[j]) : int4_order(x.v[j]);
  }
  __device__ __forceinline__ void add_up() {
    if constexpr (FMT != kMx) {
      const u32v4 ones{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4 / NG; ++j)
#pragma unroll
          for (int q = 0; q < P; ++q)
            sum[i] = mfma16(v[q][i * (4 / NG) + j], __builtin_bit_cast(bf16x8, ones), sum[i]);
      }
    }
  }
};

// The products x_t . w of an arranged chunk for TT tiles of 16 rows of x, added to
// out.
template <int FMT, int G, bool WHOLE, int TT, int P>
__device__ __forceinline__ void multiply(const Chunk<FMT, G, WHOLE>& w, const Tokens<FMT, G, P> (&x)[TT],
                                         f32x4 (&out)[TT]) {
  if constexpr (FMT == kMx) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 b = mx_values(w.codes[j], w.scale(j));
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int q = 0; q < P; ++q) out[t] = mfma16(x[t].v[q][j], b, out[t]);
    }
  } else {
    constexpr int NG = kChunk / G, PER = 4 / NG;
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
          for (int q = 0; q < P; ++q) acc[t] = mfma16(x[t].v[q][i * PER + j], b, acc[t]);
      }
      const float scale = w.scale(i), off = w.offset(i);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) out[t][r] += scale * (acc[t][r] - off * x[t].sum[i][r]);
    }
  }
}

// ---------------------------------------------------------------------------
// y = x W^T: a workgroup takes 16 NS rows of the weight and 16 TT rows of x,
// its waves the chunks in turn; the next chunk's weights are loaded before a
// chunk is multiplied.
// ---------------------------------------------------------------------------
template <int FMT, int G, bool WHOLE, int TT, int NS, int NW>
__global__ void __launch_bounds__(NW * 64)
w4_product(const uint16_t* x, int64_t ld_x, int T, int64_t n, int K, W4 w, uint16_t* y, int64_t ld_y) {
  __shared__ f32x4 part[NW][NS][TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lrow = lane >> 2,
            kq = lane & 3, src = source_lane(lane);
  const int t0 = blockIdx.y * (16 * TT);
  // (rows past the ends repeat the last ones: their results are not stored)
  int64_t row[NS];
  const uint16_t* xr[TT];
#pragma unroll
  for (int s = 0; s < NS; ++s) row[s] = min((int64_t)blockIdx.x * (16 * NS) + 16 * s + lrow, n - 1);
#pragma unroll
  for (int t = 0; t < TT; ++t) xr[t] = x + min(t0 + 16 * t + lrow, T - 1) * ld_x;
  f32x4 sum[NS][TT];
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int t = 0; t < TT; ++t) sum[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Step {
    Chunk<FMT, G, WHOLE> w[NS];
    TokenChunk x[TT];
  };
  auto load = [&](Step& to, int k0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) to.w[s].load(w, row[s], k0, K, kq);
#pragma unroll
    for (int t = 0; t < TT; ++t) to.x[t].load(xr[t], k0, K, kq);
  };
  int k0 = wave * kChunk;
  auto turn = [&](Step& cur, Step& next) {
    load(next, k0 + NW * kChunk);
    Tokens<FMT, G, 1> xs[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) cur.x[t].arrange(src), xs[t].template set<false>(0, cur.x[t]), xs[t].add_up();
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      cur.w[s].arrange(src, k0, K);
      multiply<FMT, G, WHOLE, TT, 1>(cur.w[s], xs, sum[s]);
    }
    k0 += NW * kChunk;
    return k0 < K;
  };
  // (two buffers in turn: a copy from one to the other would wait for the loads)
  Step a, b;
  if (k0 < K) {
    load(a, k0);
    while (turn(a, b) && turn(b, a)) {
    }
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
// The layer: h of every choice, then the output. h is kept as three bf16 that add
// up to its fp32 value (the matrix instructions take bf16): with one the output
// is off by 0.0025 of its norm, with two by 1.2e-4 (64 tokens, MXFP4, both
// against the elementary operations in fp32), with three by 0.3e-4. It is stored
// as it is multiplied: per row tile and part its blocks of 32 columns, each as the
// lanes take it, eight columns of a row per lane (in the order of int4_values).
// ---------------------------------------------------------------------------
constexpr int kParts = 3;           // of h
constexpr int kTile = 16 * kParts;  // elements of a row tile's h per column

struct Layer {
  int H, I, Is, E, k, T;
  float limit;
  W4 gate, up, down, sgate, sup, sdown;
  const uint16_t* x;
  const float* rw;
  const int64_t* ids;
  uint16_t* h;  // [max_tiles][kParts][16 I], then [shared tiles][kParts][16 Is]
  int max_tiles;
  bool by_token;  // a row tile has all tokens, and all parts of their h (part q of token t in row q T + t); one launch
                  // makes the output
  float* y;     // [T k + T][H]
  uint16_t* out;
};

__device__ __forceinline__ int choice(const Layer& p, int pair) {
  const int64_t e = p.ids[pair];
  return e >= 0 && e < p.E ? (int)e : -1;
}

// A batch with at most as many choices, and with at most 16 rows of h's parts,
// needs no lists of an expert's tokens: a row tile holds every token, in its own
// row (the same matrix instructions). More tokens with a tile for each part took
// 36.7 us for 16 tokens, 1 of 128 experts of 768 x 2048 and a shared one; with
// lists 30.2.
constexpr int kFewPairs = 16;
bool by_token(int T, int k) { return T * k <= kFewPairs && T * kParts <= 16; }

// Runs that the choices are counted and sorted in, one wave each.
constexpr int kRuns = 4;

// LDS of the choices sorted by expert, in row tiles of 16.
size_t plan_lds(const Layer& p) {
  return (size_t)(kRuns * p.E + p.max_tiles) * 4 + (size_t)p.T * p.k * 2;
}

struct Plan {
  int routed, tiles;   // row tiles of the routed experts; with the shared expert's behind them
  const int* tile;     // expert << 18 | (rows - 1) << 14 | first choice in the list
  const uint16_t* list;

  // The same list in every workgroup: an expert's choices in their own order, since which of them share a row tile
  // must not depend on who asks. The choices are cut into runs; what each run has of each expert is counted, and then
  // a wave goes through its run, 64 choices at a time, each placed behind those of its expert before it. (Ranking every
  // choice among all of its expert took 19.0 ms for 8192 choices of one expert of 768 x 2048; so 0.53.)
  template <int NTHR>
  __device__ __forceinline__ void build(const Layer& p, uint8_t* lds, int (&part)[NTHR / 64 + 1]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, pairs = p.T * p.k;
    if (pairs <= 64) {
      // one wave, a lane for every choice, and one barrier (1 token, 8 of 128 experts: the layer 20.3 -> 18.8 us, with
      // the output in one launch)
      int* to = (int*)lds;
      uint16_t* out = (uint16_t*)(to + p.max_tiles);
      if (wave == 0) {
        const int e = lane < pairs ? choice(p, lane) : -1;
        int n = 0, at = 0;
        for (uint64_t rest = __ballot(e >= 0); rest != 0;) {
          const int x = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)rest) - 1);
          const uint64_t m = __ballot(e == x);
          const int rows = p.by_token ? p.T : __popcll(m);
          if (e == x) out[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)lane;
          for (int q = 0; q < (rows + 15) / 16; ++q, ++n)
            if (lane == 0) to[n] = x << 18 | (min(16, rows - 16 * q) - 1) << 14 | (at + 16 * q);
          at += __popcll(m);
          rest &= ~m;
        }
        if (lane == 0) part[0] = n;
      }
      __syncthreads();
      routed = part[0];
      tiles = routed + (p.Is > 0 ? (p.T + 15) / 16 : 0);
      tile = to, list = out;
      return;
    }
    static_assert(NTHR / 64 >= kRuns, "a wave for each run");
    int* cursor = (int*)lds;  // [kRuns][E]: a run's count of an expert, then where its next choice of it goes
    int* to = cursor + kRuns * p.E;
    uint16_t* out = (uint16_t*)(to + p.max_tiles);
    const int run = (pairs + kRuns * 64 - 1) / (kRuns * 64) * 64;
    for (int e = tid; e < kRuns * p.E; e += NTHR) cursor[e] = 0;
    __syncthreads();
    for (int i = tid; i < pairs; i += NTHR) {
      const int e = choice(p, i);
      if (e >= 0) atomicAdd(&cursor[i / run * p.E + e], 1);
    }
    int base = 0;  // rows | tiles << 16 of the experts before
    for (int e0 = 0; e0 < p.E; e0 += NTHR) {
      __syncthreads();
      const int e = e0 + tid;
      int rows = 0;
      if (e < p.E)
#pragma unroll
        for (int q = 0; q < kRuns; ++q) rows += cursor[q * p.E + e];
      const int tiles_e = (rows + 15) / 16, mine = rows | tiles_e << 16;
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
      if (e < p.E)
        for (int q = 0, at = r0; q < kRuns; ++q) {
          const int n = cursor[q * p.E + e];
          cursor[q * p.E + e] = at;
          at += n;
        }
      for (int q = 0; q < tiles_e; ++q) to[t0 + q] = e << 18 | (min(16, rows - 16 * q) - 1) << 14 | (r0 + 16 * q);
      base = all;
    }
    __syncthreads();
    if (wave < kRuns) {
      volatile int* mine = cursor + wave * p.E;  // (no other wave's; LDS takes a wave's accesses in order)
      const int bits = 32 - __builtin_clz(p.E);
      for (int i0 = wave * run; i0 < min(pairs, (wave + 1) * run); i0 += 64) {
        const int i = i0 + lane, e = i < pairs ? choice(p, i) : -1;
        uint64_t same = __ballot(e >= 0);  // lanes with this lane's expert
        for (int b = 0; b < bits; ++b) {
          const uint64_t m = __ballot(e >> b & 1);
          same &= e >> b & 1 ? m : ~m;
        }
        if (e >= 0) {
          const int at = mine[e], rank = __popcll(same & ((1ull << lane) - 1));
          out[at + rank] = (uint16_t)i;
          if (rank == 0) mine[e] = at + __popcll(same);
        }
      }
    }
    __syncthreads();
    routed = base >> 16;
    tiles = routed + (p.Is > 0 ? (p.T + 15) / 16 : 0);
    tile = to, list = out;
  }
};

// A row tile: an expert (0 for the shared one) and its choices (T k + the token
// for the shared expert).
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
  // The choice of its r-th row (a row past them: of the last one).
  __device__ __forceinline__ int pair(const Plan& l, int r, int pairs) const {
    r = first + min(r, rows - 1);
    return shared ? pairs + r : l.list[r];
  }
  __device__ __forceinline__ int token(const Plan& l, int r, const Layer& p) const {
    r = min(r, rows - 1);
    return p.by_token ? r : shared ? first + r : l.list[first + r] / p.k;
  }
};

// The element of int4_values' order that element i of eight goes to.
__device__ __forceinline__ int ordered(int i) { return (i & 3) * 2 + (i >> 2); }

// h: items of one row tile and 16 columns of I, taken in turn by the
// workgroups; a workgroup's waves take the item's chunks in turn. The loop runs
// over the items' steps, with the next step's weights and x on their way.
template <int FMT, int G, bool WHOLE, int NW>
__global__ void __launch_bounds__(NW * 64) w4_gate_up(Layer p) {
  __shared__ f32x4 part[2][NW][64];
  __shared__ int scan[NW + 1];
  extern __shared__ uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6),
            lrow = lane >> 2, kq = lane & 3, src = source_lane(lane);
  Plan l;
  l.build<NW * 64>(p, dyn, scan);
  const int K = p.H;
  const int slabs_r = (p.I + 15) / 16, slabs_s = (p.Is + 15) / 16;
  const int items_r = l.routed * slabs_r, items = items_r + (l.tiles - l.routed) * slabs_s;
  const int steps = (K + NW * kChunk - 1) / (NW * kChunk);  // of an item, for each wave
  int i = blockIdx.x;
  if (i >= items) return;

  struct Step {
    Chunk<FMT, G, WHOLE> g, u;
    TokenChunk x;
  };
  struct Item {
    RowTile t;
    int tile, n0;
  } now, ahead;
  const uint16_t* xr = nullptr;
  int64_t row = 0;
  auto begin = [&](int at) {
    const bool sh = at >= items_r;
    const int v = sh ? at - items_r : at, slabs = sh ? slabs_s : slabs_r, wide = sh ? p.Is : p.I;
    ahead.tile = v / slabs;
    ahead.t.get(l, (sh ? l.routed : 0) + ahead.tile, p.T);
    ahead.n0 = v % slabs * 16;
    xr = p.x + (int64_t)ahead.t.token(l, lrow, p) * K;
    row = (int64_t)ahead.t.e * wide + min(ahead.n0 + lrow, wide - 1);
  };
  auto load = [&](Step& s, int st) {
    const int k0 = (st * NW + wave) * kChunk;
    const W4 wg = ahead.t.shared ? p.sgate : p.gate, wu = ahead.t.shared ? p.sup : p.up;
    s.g.load(wg, row, k0, K, kq);
    s.u.load(wu, row, k0, K, kq);
    s.x.load(xr, k0, K, kq);
  };
  f32x4 g[1], u[1];
  int st = 0;
  auto turn = [&](Step& cur, Step& next) {
    if (st == 0) g[0] = u[0] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool last = st == steps - 1;
    if (last && i + (int)gridDim.x < items) begin(i + gridDim.x);
    load(next, last ? 0 : st + 1);  // (behind the last item: the same one's first step again, for nothing)
    // a wave whose chunk lies behind the row's end has no part in it
    const int k0 = (st * NW + wave) * kChunk;
    if (k0 < K) {
      Tokens<FMT, G, 1> xs[1];
      cur.x.arrange(src);
      xs[0].template set<false>(0, cur.x);
      xs[0].add_up();
      cur.g.arrange(src, k0, K);
      cur.u.arrange(src, k0, K);
      multiply<FMT, G, WHOLE, 1, 1>(cur.g, xs, g);
      multiply<FMT, G, WHOLE, 1, 1>(cur.u, xs, u);
    }
    ++st;
    if (!last) return true;
    part[0][wave][lane] = g[0], part[1][wave][lane] = u[0];
    __syncthreads();
    for (int j = tid; j < 256; j += NW * 64) {  // row j / 16, column j % 16
      const int r = j >> 4, c = j & 15, at = (r >> 2) * 16 + c;
      float vg = 0.f, vu = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) vg += part[0][q][at][r & 3], vu += part[1][q][at][r & 3];
      const int wide = now.t.shared ? p.Is : p.I, col = now.n0 + c;
      if (r < now.t.rows && col < wide) {
        // (comparisons, which leave a NaN what it is: fminf and fmaxf would give the limit)
        const float lg = vg > p.limit ? p.limit : vg;
        const float lu = vu > p.limit ? p.limit : vu < -p.limit ? -p.limit : vu;
        const float v = lg / (1.f + __expf(-lg)) * lu;
        uint16_t* h = p.h + (now.t.shared ? (int64_t)p.max_tiles * kTile * p.I : 0) + (int64_t)now.tile * kTile * wide;
        h += (col / 32 * 64 + col / 8 % 4 * 16 + r) * 8 + (FMT == kMx ? col & 7 : ordered(col & 7));
        float rest = v;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          uint16_t part = f32_to_bf16(rest);
          // (what is finite in fp32 and rounds to an infinity: the largest bf16, and the rest)
          if ((part & 0x7FFFu) == 0x7F80u && __builtin_isfinite(rest)) --part;
          h[q * (p.by_token ? 8 * p.T : 16 * wide)] = part;
          const float of = bf16_to_f32(part);
          rest = rest == of ? 0.f : rest - of;  // (an infinity leaves nothing)
        }
      }
    }
    i += gridDim.x;
    if (i >= items) return false;
    now = ahead;
    st = 0;
    __syncthreads();
    return true;
  };
  // (two buffers in turn: a copy from one to the other would wait for the loads)
  Step a, b;
  begin(i);
  load(a, 0);
  now = ahead;
  while (turn(a, b) && turn(b, a)) {
  }
}

// y of every choice and of the shared expert: items as above, of 16 NS columns of
// H (which divides the reading of h by NS). The weights of the next step are on
// their way; h is loaded behind the products into the registers of the step
// before: two sets of them cost a wave per SIMD, or spills.
// Workgroups of it (of four waves) that a compute unit holds: what its registers allow without spills, two where a
// lane has the scales of four groups in two sets, else three (64 tokens, 128 experts of 768 x 2048, int4 with zero
// points: groups of 32 124 us with two, 142 with three; 17 tokens, 32 experts of 2048 x 7168, groups of 64 223 with
// three, 228 with two; MXFP4, which has its four in one register, 95 with three, 97 with two).
template <int FMT, int G, bool WHOLE>
constexpr int kDownPerCu = !WHOLE || (FMT != kMx && G == 32) ? 2 : 3;

template <int FMT, int G, bool WHOLE, int NW, int NS>
__global__ void __launch_bounds__(NW * 64, (kDownPerCu<FMT, G, WHOLE>)) w4_down(Layer p) {
  __shared__ f32x4 part[NS][NW][64];
  __shared__ int scan[NW + 1];
  extern __shared__ uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6),
            lrow = lane >> 2, kq = lane & 3, src = source_lane(lane);
  Plan l;
  l.build<NW * 64>(p, dyn, scan);
  const int pairs = p.T * p.k, slabs = (p.H + 16 * NS - 1) / (16 * NS), items = l.tiles * slabs;
  int i = blockIdx.x;
  if (i >= items) return;
  struct Step {
    Chunk<FMT, G, WHOLE> w[NS];
  };
  struct Item {
    RowTile t;
    int n0, K;
  } now, ahead;
  const uint16_t* hr = nullptr;
  int64_t row[NS] = {};
  auto begin = [&](int at) {
    const int tile = at / slabs;
    ahead.t.get(l, tile, p.T);
    ahead.n0 = at % slabs * (16 * NS);
    ahead.K = ahead.t.shared ? p.Is : p.I;
    hr = p.h + (ahead.t.shared ? (int64_t)p.max_tiles * kTile * p.I + (int64_t)(tile - l.routed) * kTile * p.Is
                               : (int64_t)tile * kTile * p.I);
#pragma unroll
    for (int s = 0; s < NS; ++s) row[s] = (int64_t)ahead.t.e * p.H + min(ahead.n0 + 16 * s + lrow, p.H - 1);
  };
  auto load = [&](Step& s, int st) {
    const int k0 = (st * NW + wave) * kChunk;
#pragma unroll
    for (int q = 0; q < NS; ++q) s.w[q].load(ahead.t.shared ? p.sdown : p.down, row[q], k0, ahead.K, kq);
  };
  TokenChunk x[kParts];
  auto load_h = [&](int st) {
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      x[q].load_blocks(hr + q * 16 * ahead.K, (st * NW + wave) * kChunk, ahead.K, lane, ahead.t.rows);
  };
  f32x4 y[NS][1];
  int st = 0;
  auto turn = [&](Step& cur, Step& next) {
    if (st == 0)
#pragma unroll
      for (int s = 0; s < NS; ++s) y[s][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool last = (st + 1) * NW * kChunk >= now.K;
    if (last && i + (int)gridDim.x < items) begin(i + gridDim.x);
    load(next, last ? 0 : st + 1);  // (behind the last item: the same one's first step again, for nothing)
    const int k0 = (st * NW + wave) * kChunk;
    if (k0 < now.K) {
      Tokens<FMT, G, kParts> xs[1];
#pragma unroll
      for (int q = 0; q < kParts; ++q) xs[0].template set<true>(q, x[q]);
      xs[0].add_up();
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        cur.w[s].arrange(src, k0, now.K);
        multiply<FMT, G, WHOLE, 1, kParts>(cur.w[s], xs, y[s]);
      }
    }
    load_h(last ? 0 : st + 1);
    ++st;
    if (!last) return true;
#pragma unroll
    for (int s = 0; s < NS; ++s) part[s][wave][lane] = y[s][0];
    __syncthreads();
    for (int j = tid; j < 256 * NS; j += NW * 64) {  // row j / (16 NS), column j % (16 NS)
      const int r = j / (16 * NS), c = j % (16 * NS), s = c >> 4, at = (r >> 2) * 16 + (c & 15), col = now.n0 + c;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) v += part[s][q][at][r & 3];
      if (r < now.t.rows && col < p.H) p.y[(int64_t)now.t.pair(l, r, pairs) * p.H + col] = v;
    }
    i += gridDim.x;
    if (i >= items) return false;
    now = ahead;
    st = 0;
    __syncthreads();
    return true;
  };
  // (two buffers in turn: a copy from one to the other would wait for the loads)
  Step a, b;
  begin(i);
  load(a, 0);
  load_h(0);
  now = ahead;
  while (turn(a, b) && turn(b, a)) {
  }
}

// The output of a batch of few choices: 16 columns of H per workgroup, its work
// every chunk of every expert chosen and of the shared one, taken by the waves in
// turn. A chunk's results go to the tokens' sums times their router weights of
// the expert (tokens that did not choose it are left out: it may hold what is not
// finite), so there is nothing for another launch to join.
// The parts of h are rows of one tile, summed at the end: a third of the loads and
// products (1 token, 8 of 128 experts of 768 x 2048 and a shared one: 19.7 us,
// 21.8 with a tile for each).
template <int FMT, int G, bool WHOLE, int NW>
__global__ void __launch_bounds__(NW * 64) w4_down_few(Layer p) {
  __shared__ f32x4 part[NW][64];
  __shared__ f32x4 coef[kFewPairs][4];      // of an expert, [16 rows]
  __shared__ int expert[kFewPairs], chosen[kFewPairs], count;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = lane >> 4,
            lrow = lane >> 2, kq = lane & 3, src = source_lane(lane);
  const int pairs = p.T * p.k;
  if (wave == 0) {  // the experts in the order of Plan's row tiles
    const int e = lane < pairs ? choice(p, lane) : -1;
    const float w = lane < pairs ? p.rw[lane] : 0.f;
    const int t = lane / p.k;
    float sum = 0.f;  // of the token's weights of this expert (it may have been chosen twice)
    for (int j = t * p.k; j < (t + 1) * p.k; ++j) {
      const float v = __shfl(w, j & 63);
      if (__shfl(e, j & 63) == e) sum += v;
    }
    if (lane < kFewPairs) chosen[lane] = 0;
    int n = 0;
    for (uint64_t rest = __ballot(e >= 0); rest != 0; ++n) {
      const int x = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)rest) - 1);
      if (e == x) {
        for (int q = 0; q < kParts; ++q) {
          ((float*)coef[n])[q * p.T + t] = sum;
          atomicOr(&chosen[n], 1 << (q * p.T + t));
        }
        expert[n] = x;
      }
      rest &= ~__ballot(e == x);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int C = (p.I + kChunk - 1) / kChunk, routed = count * C, units = routed + (p.Is + kChunk - 1) / kChunk;
  const int64_t col = min((int)blockIdx.x * 16 + lrow, p.H - 1);
  struct Step {
    Chunk<FMT, G, WHOLE> w;
    TokenChunk x;
  };
  // Unit u (behind the last one: that again, for nothing): the shared expert's, the expert's place, its K and column.
  struct Unit {
    bool sh;
    int i, K, k0;
  };
  auto unit = [&](int u) {
    u = min(u, units - 1);
    const bool sh = u >= routed;
    const int i = sh ? 0 : u / C;
    return Unit{sh, i, sh ? p.Is : p.I, (sh ? u - routed : u - i * C) * kChunk};
  };
  auto load = [&](Step& s, const Unit& t) {
    const int e = t.sh ? 0 : __builtin_amdgcn_readfirstlane(expert[t.i]);
    s.w.load(t.sh ? p.sdown : p.down, (int64_t)e * p.H + col, t.k0, t.K, kq);
    const uint16_t* h = p.h + (t.sh ? (int64_t)p.max_tiles * kTile * p.I : (int64_t)t.i * kTile * p.I);
    s.x.load_blocks(h, t.k0, t.K, lane, kParts * p.T);
  };
  f32x4 sum{0.f, 0.f, 0.f, 0.f};
  int u = wave;
  auto turn = [&](Step& cur, Step& next) {
    load(next, unit(u + NW));
    const Unit t = unit(u);
    Tokens<FMT, G, 1> xs[1];
    xs[0].template set<true>(0, cur.x);
    xs[0].add_up();
    cur.w.arrange(src, t.k0, t.K);
    f32x4 v[1]{f32x4{0.f, 0.f, 0.f, 0.f}};
    multiply<FMT, G, WHOLE, 1, 1>(cur.w, xs, v);
    const f32x4 c = coef[t.i][kg];
    const int who = t.sh ? 0xFFFF : chosen[t.i];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (who >> (4 * kg + r) & 1) sum[r] += (t.sh ? 1.f : c[r]) * v[0][r];
    u += NW;
    return u < units;
  };
  Step a, b;
  if (u < units) {
    load(a, unit(u));
    while (turn(a, b) && turn(b, a)) {
    }
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (tid < 256) {
    const int t = tid >> 4, c = blockIdx.x * 16 + (tid & 15);
    float v = 0.f;
    for (int row = min(t, p.T - 1), n = 0; n < kParts; ++n, row += p.T) {
      const int at = (row >> 2) * 16 + (tid & 15);
#pragma unroll
      for (int q = 0; q < NW; ++q) v += part[q][at][row & 3];
    }
    if (t < p.T && c < p.H) p.out[(int64_t)t * p.H + c] = f32_to_bf16(v);
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
  v = fmaxf(v, dpp_movf<kQuadXor1>(v));
  v = fmaxf(v, dpp_movf<kQuadXor2>(v));
  if (LANES > 4) v = fmaxf(v, dpp_movf<kHalfMirror>(v));
  if (LANES > 8) v = fmaxf(v, dpp_movf<kMirror>(v));
  return v;
}

// v / d for each of eight, d > 0, as IEEE has it where it is a whole number or
// half of one, and on the same side of every such number elsewhere: what rint
// asks. bf16 values (8 bits each): the quotient lies on a half number or 2^-9 of
// itself from it, so one correction of v times the reciprocal (off by 2^-22) is
// enough: four instructions a value instead of eleven. Divisors outside the range
// where the reciprocal is exact to its last bit, and fp32 values, are divided.
template <bool BF16>
__device__ __forceinline__ void divide8(const float (&v)[8], float d, float (&q)[8]) {
  if (BF16 && d > 0x1p-100f && d < 0x1p100f) {
    const float r = __builtin_amdgcn_rcpf(d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = v[j] * r;
      q[j] = __builtin_fmaf(__builtin_fmaf(-a, d, v[j]), r, a);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = v[j] / d;
  }
}

template <typename T, int FMT, int G, int TURNS>
__global__ void __launch_bounds__(256)
w4_quantize(const T* src, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, void* scale, uint8_t* zero) {
  constexpr int LANES = G / 8;
  const int64_t per = cols / 8, all = rows * per;
  const int64_t start = (int64_t)blockIdx.x * (256 * TURNS) + threadIdx.x;
  // what the lane takes in all its turns is on its way before the first (lanes past the end: zeros, and no stores)
  uint4 raw[TURNS][sizeof(T) / 2];
  int64_t rowt[TURNS];
#pragma unroll
  for (int n = 0; n < TURNS; ++n) {
    const int64_t i = start + 256 * n;
    rowt[n] = rows > 1 ? i / per : 0;
    const uint4* s = (const uint4*)(src + rowt[n] * ld + (i - rowt[n] * per) * 8);
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) raw[n][j] = i < all ? s[j] : uint4{0, 0, 0, 0};
  }
#pragma unroll
  for (int n = 0; n < TURNS; ++n) {
    const int64_t i = start + 256 * n, row = rowt[n], at = i - row * per;
    const bool in = i < all;
    float v[8];
    if constexpr (sizeof(T) == 4) {
      __builtin_memcpy(v, raw[n], 32);
    } else {
      const u32v4 w = __builtin_bit_cast(u32v4, raw[n][0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = u2f(w[j] << 16), v[2 * j + 1] = u2f(w[j] & 0xFFFF0000u);
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
      float sc, z = 8.f;
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
      float q[8];
      divide8<sizeof(T) == 2>(v, sc > 0.f ? sc : 1.f, q);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        out |= (uint32_t)(sc > 0.f ? fminf(fmaxf(rintf(q[j]) + z, 0.f), 15.f) : z) << (4 * j);
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

// f(format, group, whole chunks) as constants.
template <typename F>
void with_format(int format, int group, bool zero, bool whole, F&& f) {
  using std::integral_constant;
  using std::true_type;
  using std::false_type;
  auto grouped = [&](auto fmt, auto wh) {
    if (group == 32)
      f(fmt, integral_constant<int, 32>{}, wh);
    else if (group == 64)
      f(fmt, integral_constant<int, 64>{}, wh);
    else
      f(fmt, integral_constant<int, 128>{}, true_type{});  // a row is whole chunks
  };
  auto either = [&](auto wh) {
    if (format == MOK_W4_MXFP4)
      f(integral_constant<int, kMx>{}, integral_constant<int, 32>{}, wh);
    else if (zero)
      grouped(integral_constant<int, kZero>{}, wh);
    else
      grouped(integral_constant<int, kSym>{}, wh);
  };
  whole ? either(true_type{}) : either(false_type{});
}

}  // namespace

hipError_t launch_w4_quantize(const void* src, int src_fp32, int64_t rows, int64_t cols, int64_t ld, int format,
                              int group, uint8_t* codes, void* scale, uint8_t* zero, hipStream_t s) {
  const int64_t units = rows * cols / 8;
  if (ld == cols) cols *= rows, ld = cols, rows = 1;  // dense: one row (finding the row is a 64-bit division per lane)
  with_format(format, group, zero != nullptr, true, [&](auto fmt, auto g, auto) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    auto go = [&](auto src_type, auto turns) {
      using T = decltype(src_type);
      constexpr int TURNS = decltype(turns)::value;
      w4_quantize<T, FMT, G, TURNS><<<(unsigned)((units + 256 * TURNS - 1) / (256 * TURNS)), 256, 0, s>>>(
          (const T*)src, rows, cols, ld, codes, scale, zero);
    };
    // four turns of a lane where there is work for them (201 M elements 131 -> 122 us; 1.6 M 4.0 -> 6.2)
    auto sized = [&](auto src_type) {
      units >= 1 << 20 ? go(src_type, std::integral_constant<int, 4>{}) : go(src_type, std::integral_constant<int, 1>{});
    };
    src_fp32 ? sized(float{}) : sized(uint16_t{});
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
static bool whole_chunks(const mok_w4& w, int64_t k, int format, int group) {
  if (k % kChunk != 0) return false;
  const uintptr_t most = 2 * (kChunk / group);
  if (format == MOK_W4_MXFP4) return (uintptr_t)w.scale % 4 == 0;
  return (uintptr_t)w.scale % most == 0 && (uintptr_t)w.zero % (most / 2) == 0;
}

hipError_t launch_w4_matmul(const void* x, int64_t ld_x, int64_t T, int64_t n, int64_t k, int format, int group,
                            const mok_w4& w, void* y, int64_t ld_y, hipStream_t s) {
  using std::integral_constant;
  with_format(format, group, w.zero != nullptr, whole_chunks(w, k, format, group), [&](auto fmt, auto g, auto wh) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    constexpr bool WHOLE = decltype(wh)::value;
    auto go = [&](auto tt, auto ns, auto nw) {
      constexpr int TT = decltype(tt)::value, NS = decltype(ns)::value, NW = decltype(nw)::value;
      const dim3 grid((unsigned)((n + 16 * NS - 1) / (16 * NS)), (unsigned)((T + 16 * TT - 1) / (16 * TT)));
      w4_product<FMT, G, WHOLE, TT, NS, NW><<<grid, NW * 64, 0, s>>>((const uint16_t*)x, ld_x, (int)T, n, (int)k, w4_of(w),
                                                                     (uint16_t*)y, ld_y);
    };
    // As few weight rows per workgroup as leave one workgroup for each of 256 compute units, at 16 waves; with more
    // workgroups than that, fewer waves of more rows each, which reuse x. (A constant, so that the order of the sums
    // does not depend on the device.) K 4096, 1 row, int4: 4096 rows of weight 4.6 us (with 32 per workgroup 5.6),
    // 5120 6.1 (5.6); 20 rows: 4096 6.5 (32: 7.3, 64: 11), 8192 11.1 (8.0, 11.6), 10240 15.8 (13.4, 11.8).
    constexpr int64_t kOnce = 256;
    const int64_t tokens = (T + 31) / 32;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 4> four;
    const integral_constant<int, 16> waves;
    if (T <= 16 && n <= 16 * kOnce)
      go(one, one, waves);
    else if (T <= 16)
      go(one, two, waves);
    else if ((n + 15) / 16 * tokens <= kOnce)
      go(two, one, waves);
    else if ((n + 31) / 32 * tokens <= kOnce)
      go(two, two, waves);
    else
      go(two, four, integral_constant<int, 8>{});
  });
  return hipGetLastError();
}

// Row tiles of the routed experts, at most, and of the shared one.
static int64_t max_tiles(const mok_w4_layer& l, int64_t T) {
  const int64_t pairs = T * l.topk;
  return std::min<int64_t>(l.num_experts, pairs) + pairs / 16;
}
static int64_t shared_tiles(const mok_w4_layer& l, int64_t T) { return l.shared_intermediate > 0 ? (T + 15) / 16 : 0; }
static int64_t h_elements(const mok_w4_layer& l, int64_t T) {
  return kTile * (max_tiles(l, T) * l.intermediate + shared_tiles(l, T) * l.shared_intermediate);
}
size_t w4_layer_scratch(const mok_w4_layer& l, int64_t T) {
  return std::max<size_t>(16, (size_t)h_elements(l, T) * 2 + (size_t)T * (l.topk + 1) * l.hidden * 4);
}

hipError_t launch_w4_layer(const mok_w4_layer& l, const void* x, const float* router_w, const int64_t* ids, int64_t T,
                           void* out, void* scratch, int cus, hipStream_t s) {
  Layer p{};
  p.H = l.hidden, p.I = l.intermediate, p.Is = l.shared_intermediate, p.E = l.num_experts, p.k = l.topk, p.T = (int)T;
  p.limit = l.swiglu_limit > 0.f ? l.swiglu_limit : __builtin_inff();
  p.gate = w4_of(l.routed_gate), p.up = w4_of(l.routed_up), p.down = w4_of(l.routed_down);
  p.sgate = w4_of(l.shared_gate), p.sup = w4_of(l.shared_up), p.sdown = w4_of(l.shared_down);
  const bool sh = p.Is > 0;
  auto whole = [&](const mok_w4& w, int k) { return whole_chunks(w, k, l.format, l.group); };
  const bool all_whole = whole(l.routed_gate, p.H) && whole(l.routed_up, p.H) && whole(l.routed_down, p.I) &&
                         (!sh || (whole(l.shared_gate, p.H) && whole(l.shared_up, p.H) && whole(l.shared_down, p.Is)));
  p.x = (const uint16_t*)x, p.rw = router_w, p.ids = ids, p.h = (uint16_t*)scratch, p.out = (uint16_t*)out;
  p.y = (float*)((uint16_t*)scratch + h_elements(l, T));
  p.max_tiles = (int)max_tiles(l, T);
  p.by_token = by_token(p.T, p.k);
  const int64_t shared = shared_tiles(l, T);
  const int64_t up = (int64_t)p.max_tiles * ((p.I + 15) / 16) + shared * ((p.Is + 15) / 16);
  // weight rows of an item of w4_down, in sixteens: h is read once for them (64 tokens, 128 experts of 768 x 2048,
  // MXFP4: 103 us with 2, 99 with 3, 95 with 4)
  constexpr int kDownSlabs = 4;
  const int64_t down = (p.max_tiles + shared) * ((p.H + 16 * kDownSlabs - 1) / (16 * kDownSlabs));
  const size_t lds = plan_lds(p);
  with_format(l.format, l.group, l.routed_gate.zero != nullptr, all_whole, [&](auto fmt, auto g, auto wh) {
    constexpr int FMT = decltype(fmt)::value, G = decltype(g)::value;
    constexpr bool WHOLE = decltype(wh)::value;
    // as many workgroups as stay on the card together (gate_up: 16 waves per compute unit)
    w4_gate_up<FMT, G, WHOLE, 8><<<(unsigned)std::min<int64_t>(up, 2 * cus), 512, lds, s>>>(p);
    if (p.by_token)
      w4_down_few<FMT, G, WHOLE, 16><<<(p.H + 15) / 16, 1024, 0, s>>>(p);
    else
      w4_down<FMT, G, WHOLE, 4, kDownSlabs>
          <<<(unsigned)std::min<int64_t>(down, kDownPerCu<FMT, G, WHOLE> * cus), 256, lds, s>>>(p);
  });
  if (!p.by_token) w4_combine<<<dim3((p.H + 255) / 256, p.T), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace mok
