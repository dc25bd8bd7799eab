// Matrix products grouped by expert, rows given by offsets: y = x W_e^T per
// expert, and its gradients dx = dy W_e and dW_e = dy^T x.
//
// All three are C[m, n] = sum over k of A(m, k) B(n, k), with other roles:
//         m                n             contraction     A          B
//   y     e's rows         W's rows      W's columns     x          W_e
//   dx    e's rows         W's columns   W's rows        dy         W_e^T
//   dW    W's rows         W's columns   e's rows        dy^T       x^T
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "gemm_common.h"
#include "mok_internal.h"

namespace mok {
namespace {

// Elements of the output, dense.
__host__ __device__ __forceinline__ int64_t out_elements(int op, const GroupedArgs& g) {
  return op == GROUPED_Y ? g.rows * g.n : op == GROUPED_DX ? g.rows * g.k : g.E * g.n * g.k;
}

// Bounds of expert e's rows, whatever the offsets hold.
__device__ __forceinline__ void segment(const GroupedArgs& g, int e, int& lo, int& hi) {
  int64_t a, b;
  if (g.offsets64) {
    a = ((const int64_t*)g.offsets)[e];
    b = ((const int64_t*)g.offsets)[e + 1];
  } else {
    a = ((const int32_t*)g.offsets)[e];
    b = ((const int32_t*)g.offsets)[e + 1];
  }
  lo = (int)min(max(a, (int64_t)0), g.rows);
  hi = (int)min(max(b, (int64_t)lo), g.rows);
}

// Exclusive prefix sums of the experts' M tiles of `bm` rows in tiles[0..E],
// by the whole workgroup. `part`: one int per wave. Sums end at what offsets that
// do not decrease can give, rows / bm + E: decreasing ones may name all rows for
// every other expert, 2^31 tiles at 2^29 rows, which neither an int nor the time
// of a call holds. (With every wave's sum cut off there too, no sum passes 2^30.)
template <int NTHR>
__device__ __forceinline__ void scan_tiles(const GroupedArgs& g, int bm, int32_t* tiles, int32_t* part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int most = (int)(g.rows / bm) + g.E;
  int base = 0;
  for (int e0 = 0; e0 < g.E; e0 += NTHR) {
    const int e = e0 + tid;
    int cnt = 0;
    if (e < g.E) {
      int lo, hi;
      segment(g, e, lo, hi);
      cnt = (hi - lo + bm - 1) / bm;
    }
    int s = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(s, d);
      if (lane >= d) s += v;
    }
    if (lane == 63) part[wave] = min(s, most);
    __syncthreads();
    int before = base, all = base;
    for (int w = 0; w < NTHR / 64; ++w) {
      if (w < wave) before += part[w];
      all += part[w];
    }
    if (e < g.E) tiles[e] = min(before + s - cnt, most);
    base = min(all, most);
    __syncthreads();
  }
  if (tid == 0) tiles[g.E] = base;
  __syncthreads();
}

// The expert of M tile mt: the largest e with tiles[e] <= mt.
__device__ __forceinline__ int expert_of(const int32_t* tiles, int E, int mt) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tiles[mid] <= mt)
      lo = mid;
    else
      hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Zeros in the rows of no expert, cols elements of each, by the whole grid.
__device__ __forceinline__ void zero_rest(const GroupedArgs& g, int cols) {
  int first, end, x;
  segment(g, 0, first, x);
  segment(g, g.E - 1, x, end);
  end = max(end, first);
  const int64_t n = (int64_t)first + (g.rows - end);
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    uint16_t* row = (uint16_t*)g.out + (i < first ? i : end + (i - first)) * g.ld_out;
    for (int c = threadIdx.x; c < cols; c += blockDim.x) row[c] = 0;
  }
}

// ---------------------------------------------------------------------------
// 256 x 256 output tiles, eight waves of 128 x 64 (4 x 2 MFMA tiles of 32 x
// 32), operands in a ring of four LDS stages of 32 contraction steps.
//
// A stage holds an operand either as 256 rows of 32 dense contraction elements
// ("rows", 64 bytes each; x, dy, W of y) or as 32 contraction rows of 256 dense
// elements ("columns", 512 bytes each; W of dx, both operands of dW), as it lies
// in memory; columns are turned on the way to the registers by the transposing
// LDS read. 16-byte chunks are swizzled so that the reads of a wave's quarter
// hit every bank once: rows by (row / 4) % 4 within 64 bytes, columns by
// 4 (row % 4) within 512.
//
// One barrier per stage, in the middle of its products: the fragments of the
// second half are in registers by then, so the products go on while the waves
// meet, and the loads issued behind it have two stages' time to land.
//
// DMA: widths and strides that are multiples of 8 elements in 16-byte aligned
// tensors are loaded straight to LDS, three stages ahead. Others go through
// registers, one or two stages ahead: 16-byte loads at the elements' own
// alignment (which the memory takes), where a chunk of 8 ends behind its row
// the 8 that end with the row's last one. That costs a third: 4099 rows, 37
// experts of 1001 x 1037 36 us, of 1000 x 1040 27; dx and dW of 12327 rows, 18
// experts of 2176 x 4690 812 us, of 2176 x 4688 587.
// ---------------------------------------------------------------------------
constexpr int kStep = 32, kRing = 4;
constexpr int kNumXcd = 8;
constexpr int kGroupM = 4;               // M tiles that run together with all N tiles
constexpr uint32_t kOff = 0x80000000u;   // past every resource: loads return 0

// S: rows and columns of a tile.
template <int S>
struct Shape {
  static constexpr int kThreads = S == 256 ? 512 : 256, kWaves = kThreads / 64;
  static constexpr int kWaveRows = S / 2, kWavesN = S / 64;  // a wave has S / 2 rows and 64 columns
  static constexpr int kBlocks = kWaveRows / 32;             // its MFMA tiles along the rows
  static constexpr int kOperandBytes = S * kStep * 2, kStageBytes = 2 * kOperandBytes;
  static_assert(kOperandBytes == kWaves * 2 * 1024, "two loads of a wave per operand and stage");
};

template <int S>
struct alignas(16) TileLds {
  uint8_t ring[kRing][Shape<S>::kStageBytes];
  int32_t tiles[kGroupedMaxExperts + 1];
  int32_t part[Shape<S>::kWaves];
};

// 16 bytes at an element's alignment.
struct __attribute__((packed, aligned(2))) Unaligned16 {
  u32x4 v;
};

// How the operands come to LDS: by DMA, through registers, or (rows of fewer
// than eight elements) through registers one by one.
constexpr int kDma = 0, kRegisters = 1, kSingles = 2;

// Eight elements as load_eight read them, the last of its row first shifted
// down: the n of the row (0 for n < 0), zeros behind them.
__device__ __forceinline__ u32x4 settle(u32x4 v, int n) {
  typedef __attribute__((ext_vector_type(2))) uint64_t u64x2;
  const u64x2 w = __builtin_bit_cast(u64x2, v);
  const int s = 16 * (8 - min(max(n, 1), 8));  // 0 to 112
  const uint64_t over = s == 0 ? 0 : w[1] << ((64 - s) & 63);
  const uint64_t low = s >= 64 ? w[1] >> (s - 64) : (w[0] >> (s & 63)) | over;
  return __builtin_bit_cast(u32x4, n > 0 ? u64x2{low, s >= 64 ? 0 : w[1] >> (s & 63)} : u64x2{0, 0});
}

// An operand of the current tile.
template <bool COLUMNS, int S>
struct Operand {
  static constexpr int kRowChunks = S / 8, kLoadRows = 64 / kRowChunks;  // columns: chunks of a row, rows of a load

  const uint8_t* base;  // its first row (rows) or its first contraction row (columns) at the tile
  int64_t ld;           // bytes from row to row
  uint32_t off[2];      // this lane's two loads of a stage, kOff if outside
  int chunk[2];         // rows: the contraction chunk of each; columns: its contraction row
  int width[2];         // columns: elements from its first one to the row's end (not for DMA)
  int front;            // columns: elements of a row in front of the tile
  bool ragged;          // columns: the row ends inside the tile

  // `have`: rows (columns: elements) from the tile's first one on that exist.
  __device__ __forceinline__ void init(const void* p, int64_t ld_elements, int have, int front_, int wave, int lane) {
    base = (const uint8_t*)p;
    ld = ld_elements * 2;
    front = front_, ragged = COLUMNS && have < S;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (COLUMNS) {
        const int row = (2 * wave + i) * kLoadRows + lane / kRowChunks, c = lane % kRowChunks ^ (4 * (row & 3));
        chunk[i] = row;
        width[i] = have - c * 8;
        off[i] = c * 8 < have ? (uint32_t)(row * ld) + 16u * c : kOff;
      } else {
        const int row = (2 * wave + i) * 16 + (lane >> 2), c = (lane & 3) ^ ((row >> 2) & 3);
        chunk[i] = c;
        off[i] = row < have ? (uint32_t)(row * ld) + 16u * c : kOff;
      }
    }
  }
  // Load i of the two for contraction elements k0 .. k0 + 31 of K, to LDS at `to`.
  __device__ __forceinline__ void load(int k0, int K, uint32_t to, int wave, int i) const {
    to += (uint32_t)(2 * wave + i) * 1024u;
    if (COLUMNS)  // rows past K lie behind the resource's end
      lds_dma16(rsrc(base + (int64_t)k0 * ld, (uint32_t)(min(K - k0, kStep) * ld)), off[i], 0, to);
    else
      lds_dma16(rsrc(base + (int64_t)k0 * 2, 0x7FFFFFFFu), k0 + 8 * chunk[i] < K ? off[i] : kOff, 0, to);
  }
  // The same through registers: from memory, and to LDS.
  __device__ __forceinline__ int count(int k0, int K, int i) const {
    if (COLUMNS) return k0 + chunk[i] < K ? width[i] : 0;
    return off[i] != kOff ? K - k0 - 8 * chunk[i] : 0;
  }
  // Where a chunk ends behind its row, the eight elements that end with the
  // row's last one are read; where it has none, the first eight of the first
  // row. So a load needs no branch, and those behind it can be counted.
  template <int MODE>
  __device__ __forceinline__ u32x4 fetch(int k0, int K, int i) const {
    const uint8_t* p = base + (COLUMNS ? (int64_t)k0 * ld : (int64_t)k0 * 2) + off[i];
    const int n = count(k0, K, i);
    if constexpr (MODE == kRegisters) {
      return ((const Unaligned16*)(n > 0 ? p - 2 * (8 - min(n, 8)) : base - 2 * front))->v;
    } else {
      u32x4 v{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) v[j / 2] |= (uint32_t)((const uint16_t*)p)[j] << (16 * (j % 2));
      return v;
    }
  }
  // (What lies in rows or columns outside the output is not looked at.)
  template <int MODE>
  __device__ __forceinline__ void put(u32x4 v, int k0, int K, uint8_t* to, int wave, int lane, int i) const {
    if (MODE == kRegisters && (ragged || K - k0 < kStep)) v = settle(v, count(k0, K, i));
    *reinterpret_cast<u32x4*>(to + (2 * wave + i) * 1024 + lane * 16) = v;
  }
  // The fragment of 32 rows from `row0`, contraction elements 16 ks + 8 lh + 0..7 of row row0 + lr.
  static __device__ __forceinline__ bf16x8 fragment(const uint8_t* st, int row0, int ks, int lane) {
    const int lr = lane & 31, lh = lane >> 5;
    if (COLUMNS) {
      typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
      typedef __attribute__((address_space(3))) bf16x4 lds4;
      const int i = lane & 15, m = row0 + (lr & 16) + 4 * (i & 3), k = 16 * ks + 8 * lh + (i >> 2);
      // (k % 4 is i / 4 in both reads)
      const uint8_t* at = st + k * (S * 2) + ((m >> 3) ^ (4 * (i >> 2))) * 16 + (m & 7) * 2;
#if defined(__HIP_DEVICE_COMPILE__)
      const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)at);
      const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(at + 4 * S * 2));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
#else
      return bf16x8{};
#endif
    } else {
      const int row = row0 + lr;
      return *reinterpret_cast<const bf16x8*>(st + row * 64 + (((2 * ks + lh) ^ (lr >> 2)) & 3) * 16);
    }
  }
};

// Writes a wave's results (BLOCKS x 32 rows of 64) through its 4 KiB of LDS, 32 rows of 128
// bytes at a time, whole lines of a row per store.
// PAST: past the caches (not the parts, which the next launch reads: 64 rows, y of 256 over 8192: 12.0 us instead of
// 11.2).
template <typename T, bool DMA, bool PAST, int BLOCKS>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[BLOCKS][2], uint8_t* lds, T* out, int64_t ld, int rows,
                                           int cols, int lane) {
  constexpr int PART = sizeof(T) == 4 ? 2 : 1;  // passes over the 64 columns
  const int lr = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
    for (int h = 0; h < PART; ++h) {
#pragma unroll
      for (int j = 0; j < 2 / PART; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& a = acc[i][h + j];
          uint8_t* row = lds + lr * 128;
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(row + ((j * 4 + q) ^ (lr & 7)) * 16 + lh * 8) =
                make_uint2(pack_bf16x2(a[4 * q], a[4 * q + 1]), pack_bf16x2(a[4 * q + 2], a[4 * q + 3]));
          else
            *reinterpret_cast<f32x4*>(row + ((2 * q + lh) ^ (lr & 7)) * 16) =
                f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
        }
      const int c = lane & 7, col = (h * 8 + c) * (int)(16 / sizeof(T));
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 8) {
        const int r = r0 + (lane >> 3);
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + r * 128 + (c ^ (r & 7)) * 16);
        T* to = out + (int64_t)(i * 32 + r) * ld + col;
        constexpr int PER = 16 / sizeof(T);
        if (i * 32 + r >= rows) continue;
        if constexpr (DMA) {
          if (col < cols) {
            if constexpr (PAST)
              __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(to));
            else
              *reinterpret_cast<u32x4*>(to) = v;
          }
        } else if (col + PER <= cols) {
          ((Unaligned16*)to)->v = v;
        } else {
#pragma unroll
          for (int j = 0; j < PER - 1; ++j) {
            if (col + j >= cols) break;
            if constexpr (sizeof(T) == 4)
              to[j] = u2f(v[j]);
            else
              to[j] = (T)(v[j / 2] >> (16 * (j % 2)));
          }
        }
      }
    }
}

// A tile of the output, or (PARTS) of a part of its contraction: its operands,
// and where a wave's results go.
template <int OP, bool PARTS, int S>
struct Tile {
  using OpA = Operand<OP == GROUPED_DW, S>;
  using OpB = Operand<OP != GROUPED_Y, S>;
  static constexpr int kOperandBytes = Shape<S>::kOperandBytes, kStageBytes = Shape<S>::kStageBytes;
  OpA A;
  OpB B;
  int K, rows, cols;  // contraction length; rows and columns of the output from the tile's corner on
  int64_t out;        // element of its corner
  int turn;           // the stage that its contraction begins with
  int split, first_stage, end_stage;  // PARTS: which of them it is

  // Item `id` of `all` tiles times the parts of the contraction.
  __device__ __forceinline__ void init(const GroupedArgs& g, const int32_t* tiles, int64_t id, int64_t all, int wave,
                                       int lane) {
    if (PARTS) {
      split = (int)(id / all);
      id -= split * all;
    }
    const int N = (int)(OP == GROUPED_Y ? g.n : g.k), nt = (N + S - 1) / S;
    int e, local, nm;
    if (OP == GROUPED_DW) {
      nm = (int)((g.n + S - 1) / S);
      e = (int)(id / (nm * nt));
      local = (int)(id - (int64_t)e * nm * nt);
    } else {
      e = expert_of(tiles, g.E, (int)(id / nt));
      local = (int)(id - (int64_t)tiles[e] * nt);
      nm = tiles[e + 1] - tiles[e];
    }
    const int first = local / (kGroupM * nt) * kGroupM, gm = min(kGroupM, nm - first), r = local - first * nt;
    const int m0 = __builtin_amdgcn_readfirstlane((first + r % gm) * S);
    const int n0 = __builtin_amdgcn_readfirstlane(r / gm * S);
    int lo, hi;
    segment(g, e, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo), hi = __builtin_amdgcn_readfirstlane(hi);
    rows = (OP == GROUPED_DW ? (int)g.n : hi - lo) - m0, cols = N - n0;
    K = (int)(OP == GROUPED_Y ? g.k : OP == GROUPED_DX ? g.n : hi - lo);
    // Rows that lie a multiple of 4 KiB apart have the same columns in the same
    // memory channels: tiles start at different columns, spread over the range
    // between the XCDs and the experts, and by a few stages between tiles that
    // share operands (which stay near each other for the cache's sake).
    if (PARTS) {
      const int every = (K + kStep - 1) / kStep;
      first_stage = (int)((int64_t)every * split / g.splits);
      end_stage = (int)((int64_t)every * (split + 1) / g.splits);
    }
    const int n = steps();
    turn = 0;
    if (OP != GROUPED_DW && n > 0) {
      const int apart = OP == GROUPED_Y ? 2 * ((m0 / S + n0 / S) % 4) : 0;
      turn = ((int)(blockIdx.x % kNumXcd) * n / kNumXcd + 3 * e + apart) % n;
    }
    const uint16_t* a = (const uint16_t*)g.a;
    const uint16_t* b = (const uint16_t*)g.b;
    if (OP == GROUPED_DW) {
      A.init(a + lo * g.ld_a + m0, g.ld_a, rows, m0, wave, lane);
      B.init(b + lo * g.ld_b + n0, g.ld_b, cols, n0, wave, lane);
      out = ((int64_t)e * g.n + m0) * g.k + n0;
    } else {
      A.init(a + (lo + m0) * g.ld_a, g.ld_a, rows, 0, wave, lane);
      B.init(b + (int64_t)e * g.n * g.k + (OP == GROUPED_Y ? n0 * g.k : n0), g.k, cols, n0, wave, lane);
      out = (lo + m0) * (PARTS ? N : g.ld_out) + n0;
    }
  }
  __device__ __forceinline__ int steps() const { return PARTS ? end_stage - first_stage : (K + kStep - 1) / kStep; }
  // First contraction element of the kt-th stage.
  __device__ __forceinline__ int at(int kt) const {
    const int n = steps(), k = kt + turn;
    return ((PARTS ? first_stage : 0) + (k < n ? k : k - n)) * kStep;
  }
  // Loads stage kt.
  __device__ __forceinline__ void issue(int kt, uint32_t ring, int wave) const {
    const uint32_t to = ring + (uint32_t)(kt % kRing) * kStageBytes;
    A.load(at(kt), K, to, wave, 0), A.load(at(kt), K, to, wave, 1);
    B.load(at(kt), K, to + kOperandBytes, wave, 0), B.load(at(kt), K, to + kOperandBytes, wave, 1);
  }
  // The four loads of a wave for stage kt, and their way to LDS (without DMA).
  template <int MODE>
  __device__ __forceinline__ void fetch(int kt, u32x4 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = A.template fetch<MODE>(at(kt), K, i), v[2 + i] = B.template fetch<MODE>(at(kt), K, i);
  }
  template <int MODE>
  __device__ __forceinline__ void put(int kt, const u32x4 (&v)[4], uint8_t* ring, int wave, int lane) const {
    uint8_t* to = ring + kt % kRing * kStageBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      A.template put<MODE>(v[i], at(kt), K, to, wave, lane, i);
      B.template put<MODE>(v[2 + i], at(kt), K, to + kOperandBytes, wave, lane, i);
    }
  }
  // One of the four loads of a wave for stage kt.
  __device__ __forceinline__ void issue_part(int kt, int part, uint32_t ring, int wave) const {
    const uint32_t to = ring + (uint32_t)(kt % kRing) * kStageBytes;
    if (part < 2)
      A.load(at(kt), K, to, wave, part);
    else
      B.load(at(kt), K, to + kOperandBytes, wave, part - 2);
  }
};

// OUT: where the results go.
constexpr int kBf16 = 0, kF32 = 1, kParts = 2;  // kParts: fp32 sums of a part of the contraction

template <int OP, int OUT, int MODE, int S>
__global__ void __launch_bounds__(Shape<S>::kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
grouped_tiles(GroupedArgs g) {
  using H = Shape<S>;
  constexpr bool PARTS = OUT == kParts, DMA = MODE == kDma;
  using T = Tile<OP, PARTS, S>;
  __shared__ TileLds<S> L;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / H::kWavesN, wn = wave % H::kWavesN;
  const int N = (int)(OP == GROUPED_Y ? g.n : g.k), nt = (N + S - 1) / S;
  if (OP != GROUPED_DW) scan_tiles<H::kThreads>(g, S, L.tiles, L.part);
  const int64_t all =
      OP == GROUPED_DW ? (int64_t)g.E * ((g.n + S - 1) / S) * nt : (int64_t)L.tiles[g.E] * nt;
  const int64_t items = PARTS ? all * g.splits : all;
  // Workgroup b runs on XCD b % 8. Runs of neighbouring tiles, which share
  // operands, go to the XCDs in turn: as many as an XCD has workgroups, but in
  // the last round the XCDs share what is left evenly.
  const int nq = gridDim.x % kNumXcd == 0 ? kNumXcd : 1, slots = gridDim.x / nq;
  const int xcd = blockIdx.x % nq, slot = blockIdx.x / nq;
  const int64_t full = items - items % gridDim.x;
  const int last = (int)(items - full + nq - 1) / nq;
  // the tile behind `at`, this workgroup's first one of a round
  auto tile_of = [&](int64_t at) {
    if (at + gridDim.x <= items) return at + (int64_t)xcd * slots + slot;
    return slot < last ? at + (int64_t)xcd * last + slot : items;
  };
  int64_t round = 0, id = tile_of(0);
  const uint32_t ring = lds_addr(&L.ring[0][0]);
  T t;
  // The first stages of the tile `id`.
  auto begin = [&] {
    t.init(g, L.tiles, id, all, wave, lane);
    if (DMA)
      for (int kt = 0; kt < min(t.steps(), kRing - 1); ++kt) t.issue(kt, ring, wave);
  };
  if (id < items) begin();
  while (id < items) {
    f32x16 acc[H::kBlocks][2];
#pragma unroll
    for (int i = 0; i < H::kBlocks; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    const int nk = t.steps();
    // NI: 32-row blocks of this wave that hold rows, rounded up to 0, 1, 2 or all (at compile time, so that a ragged
    // tile leaves out reads and products without branches between them)
    auto run = [&](auto ni_c) {
      constexpr int NI = decltype(ni_c)::value;
      bf16x8 fa[2][NI > 0 ? NI : 1], fb[2][2];
      // without DMA: stages on their way. (Two for the smaller tile: a load takes longer than a stage's products, 193 x
      // 75 over 16384 rows 431 us against 476; the larger one has no registers left.)
      constexpr int SETS = S == 128 && MODE == kRegisters ? 2 : 1;
      u32x4 v[SETS][4];
      // read(st, ks, r): the r-th of the fragments of half ks, in the order of their use
      auto read = [&](const uint8_t* st, int ks, int r) {
        if (NI > 0 && r < NI + 2) {
          if (r == 0 || r == 2)
            fb[ks][r / 2] = T::OpB::fragment(st + T::kOperandBytes, wn * 64 + r / 2 * 32, ks, lane);
          else if (const int i = r == 1 ? 0 : r - 2; i < NI)
            fa[ks][i] = T::OpA::fragment(st, wm * H::kWaveRows + i * 32, ks, lane);
        }
      };
      auto stage = [&](int kt) { return (const uint8_t*)&L.ring[kt % kRing][0]; };
      // The products of half ks, between them the reads of the other half's
      // fragments and a stage's loads: while a product occupies the matrix
      // pipe, the wave's next instructions go to the other units, so none of
      // them may queue up in front of the products.
      constexpr int kMost = 2 * H::kBlocks;
      auto half = [&](int ks, auto read_next, auto&& load) {
#pragma unroll
        for (int m = 0; m < kMost; ++m) {
          if constexpr (NI > 0) if (m / 2 < NI) {
            __builtin_amdgcn_sched_barrier(0);
            acc[m / 2][m % 2] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[ks][m % 2], fa[ks][m / 2], acc[m / 2][m % 2], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
          }
          read_next(m);
          load(m);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      // One stage; AFTER: how many of this wave's loads behind stage kt + 1's may be in flight (-1: there is no such
      // stage). Kept free of branches: where paths meet, the compiler waits for the reads of either.
      auto step = [&](int kt, auto after, auto more, auto set) {
        constexpr int AFTER = decltype(after)::value;
        constexpr bool MORE = decltype(more)::value;
        half(0, [&](int m) { read(stage(kt), 1, m); }, [](int) {});
        if constexpr (AFTER >= 0) {
          if (DMA) {
            wait_vmcnt<(AFTER < 0 ? 0 : AFTER)>();
          } else {
            constexpr int SET = decltype(set)::value;
            t.template put<MODE>(kt + 1, v[SET], &L.ring[0][0], wave, lane);
            // (no stage behind the last one: that again, so that the loads in flight can be counted)
            t.template fetch<MODE>(min(kt + 1 + SETS, nk - 1), v[SET]);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          }
          // stage kt + 1 has landed, and nobody reads stage kt - 1 any more (its last fragments went into products
          // that this wave has issued; the reads in flight are of stage kt)
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          half(1, [&](int m) { read(stage(kt + 1), 0, m); }, [&](int m) {
            constexpr int EVERY = kMost / 4;
            if (DMA && MORE && m % EVERY == EVERY - 1) t.issue_part(kt + kRing - 1, m / EVERY, ring, wave);
          });
        } else {
          half(1, [](int) {}, [](int) {});
        }
      };
      using std::integral_constant;
      if (!DMA) {
        t.template fetch<MODE>(0, v[0]);
        if (SETS > 1) t.template fetch<MODE>(min(1, nk - 1), v[SETS - 1]);
        t.template put<MODE>(0, v[0], &L.ring[0][0], wave, lane);
        t.template fetch<MODE>(min(SETS, nk - 1), v[0]);
      } else if (nk > kRing - 2) {
        wait_vmcnt<4 * (kRing - 2)>();  // (the stores of the tile before are younger than the first stages' loads)
      } else {
        wait_vmcnt<0>();
      }
      __syncthreads();  // stage 0 has landed for every wave
      for (int r = 0; r < NI + 2; ++r) read(stage(0), 0, r);
      int kt = 0;
      const integral_constant<int, 0> set0;
      const integral_constant<int, 4 * (kRing - 3)> full;
      if constexpr (DMA) {
        constexpr int AHEAD = kRing - 1;  // stages from a load to its use
        for (; kt < nk - AHEAD; ++kt) step(kt, full, std::true_type{}, set0);
        // the last stages: one fewer in flight from step to step
        auto drain = [&](auto self, auto left) {
          constexpr int LEFT = decltype(left)::value;
          if constexpr (LEFT > 1) {
            if (nk >= LEFT) step(kt++, integral_constant<int, 4 * (LEFT - 2)>{}, std::false_type{}, set0);
            self(self, integral_constant<int, LEFT - 1>{});
          }
        };
        drain(drain, integral_constant<int, AHEAD>{});
      } else if constexpr (SETS == 2) {
        for (; kt < nk - 2; kt += 2) {
          step(kt, full, std::true_type{}, integral_constant<int, 1>{});
          step(kt + 1, full, std::true_type{}, set0);
        }
        if (kt < nk - 1) step(kt++, full, std::true_type{}, integral_constant<int, 1>{});
      } else {
        for (; kt < nk - 1; ++kt) step(kt, full, std::true_type{}, set0);
      }
      step(kt, integral_constant<int, -1>{}, std::false_type{}, set0);
    };
    const int live = min(H::kBlocks, max(0, (t.rows - wm * H::kWaveRows + 31) / 32));
    if (nk > 0) {
      if (live > 2)
        run(std::integral_constant<int, H::kBlocks>{});
      else if (live == 2)
        run(std::integral_constant<int, 2>{});
      else if (live == 1)
        run(std::integral_constant<int, 1>{});
      else
        run(std::integral_constant<int, 0>{});
    }
    // ---- results, while the next tile's first stages are loaded ----
    __syncthreads();  // nobody reads the ring any more
    const int64_t out = t.out;
    const int split = PARTS ? t.split : 0;
    const int rows = t.rows - wm * H::kWaveRows, cols = t.cols - wn * 64;
    round += gridDim.x;
    id = tile_of(round);
    if (id < items) begin();
    // the last stage is not in use before every wave has passed the next tile's first barrier
    static_assert(H::kWaves * 4096 == H::kStageBytes, "4 KiB for each wave");
    uint8_t* part = &L.ring[kRing - 1][0] + wave * 4096;
    const int64_t ld = OP == GROUPED_DW ? g.k : OUT == kParts ? N : g.ld_out;
    const int64_t at = out + (int64_t)(wm * H::kWaveRows) * ld + wn * 64;
    if constexpr (OUT == kBf16)
      store_tile<uint16_t, DMA, true, H::kBlocks>(acc, part, (uint16_t*)g.out + at, ld, rows, cols, lane);
    else if constexpr (OUT == kF32)
      store_tile<float, DMA, true, H::kBlocks>(acc, part, (float*)g.out + at, ld, rows, cols, lane);
    else
      store_tile<float, DMA, false, H::kBlocks>(acc, part, g.part + split * out_elements(OP, g) + at, ld, rows, cols, lane);
  }
  if (OP != GROUPED_DW && OUT != kParts && g.zero_rest) zero_rest(g, N);
}

// The sum of the parts, in their order, eight loads at a time: one by one they
// take the latency each (64 rows, y of 256 over 2048: 12.4 us instead of 9.7).
template <int OP>
__global__ void __launch_bounds__(256) grouped_join(GroupedArgs g) {
  const int64_t n = out_elements(OP, g);
  const int N = (int)(OP == GROUPED_Y ? g.n : g.k);
  int first = 0, end = 0, x;
  if (OP != GROUPED_DW) segment(g, 0, first, x), segment(g, g.E - 1, x, end);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = OP == GROUPED_DW ? 0 : i / N, to = OP == GROUPED_DW ? i : row * g.ld_out + (i - row * N);
    const bool mine = OP == GROUPED_DW || (row >= first && row < end);
    if (!mine && !g.zero_rest) continue;
    float v = 0.f;
    if (mine)
#pragma unroll 8
      for (int s = 0; s < g.splits; ++s) v += g.part[s * n + i];
    if (OP == GROUPED_DW && g.out_fp32)
      ((float*)g.out)[to] = v;
    else
      ((uint16_t*)g.out)[to] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// y for few rows per expert (decoding, small batches): bound by reading the
// weights of the experts that have rows. A workgroup takes 16 rows of one
// expert's weight and all its rows of x, 16 at a time; its waves take
// chunks of 128 columns in turn and their sums are joined through LDS. Weights
// and x go from memory straight into the operands of the 16 x 16 x 32 matrix
// instruction (lane % 16 is the row of x, or of the weight, lane / 16 the
// eighth of 32 columns).
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8, kFewChunk = 128;

__global__ void __launch_bounds__(kFewWaves * 64) grouped_few(GroupedArgs g) {
  __shared__ f32x4 part[kFewWaves][64];
  __shared__ uint64_t busy[kGroupedMaxExperts / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = lane >> 4, li = lane & 15;
  if (g.zero_rest && blockIdx.y == 0) zero_rest(g, (int)g.n);
  // the blockIdx.y-th expert with rows
  for (int e0 = 0; e0 < g.E; e0 += kFewWaves * 64) {
    int lo = 0, hi = 0;
    if (e0 + tid < g.E) segment(g, e0 + tid, lo, hi);
    const uint64_t m = __ballot(hi > lo);
    if (lane == 0 && e0 + wave * 64 < g.E) busy[e0 / 64 + wave] = m;
  }
  __syncthreads();
  int e = -1, left = blockIdx.y;
  for (int q = 0; q * 64 < g.E; ++q) {
    uint64_t m = busy[q];
    const int c = __popcll(m);
    if (left < c) {
      for (; left > 0; --left) m &= m - 1;
      e = 64 * q + __ffsll((unsigned long long)m) - 1;
      break;
    }
    left -= c;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  if (e < 0) return;  // fewer experts than workgroups: all of it
  int lo, hi;
  segment(g, e, lo, hi);
  const int K = (int)g.k, n0 = blockIdx.x * 16;
  const uint16_t* w = (const uint16_t*)g.b + ((int64_t)e * g.n + min(n0 + li, (int)g.n - 1)) * K;
  for (int r0 = lo; r0 < hi; r0 += 16) {
    f32x4 sum{0.f, 0.f, 0.f, 0.f};
    // (rows past the end repeat the last one: their results are not stored)
    const uint16_t* x = (const uint16_t*)g.a + (int64_t)min(r0 + li, hi - 1) * g.ld_a;
    for (int k0 = wave * kFewChunk; k0 < K; k0 += kFewWaves * kFewChunk) {
      bf16x8 a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 32 * j + 8 * kg;
        const bf16x8 none{};
        b[j] = k < K ? *(const bf16x8*)(w + k) : none;
        a[j] = k < K ? *(const bf16x8*)(x + k) : none;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], b[j], sum, 0, 0, 0);
    }
    part[wave][lane] = sum;
    __syncthreads();
    if (tid < 256) {  // row tid / 16, column tid % 16
      const int r = tid >> 4, at = (r >> 2) * 16 + (tid & 15);
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kFewWaves; ++q) v += part[q][at][r & 3];
      const int row = r0 + r, col = n0 + (tid & 15);
      if (row < hi && col < g.n) ((uint16_t*)g.out)[(int64_t)row * g.ld_out + col] = f32_to_bf16(v);
    }
    __syncthreads();
  }
}

bool by_eight(const GroupedArgs& g) {
  return ((g.n | g.k | g.ld_a | g.ld_b | g.ld_out) & 7) == 0 &&
         (((uintptr_t)g.a | (uintptr_t)g.b | (uintptr_t)g.out) & 15) == 0;
}

}  // namespace

template <int OP, int OUT, int MODE>
static void launch_tiles(const GroupedArgs& g, bool small, int cus, hipStream_t s) {
  // (two waves per SIMD)
  if constexpr (OUT != kParts && MODE != kSingles) {
    if (!small) {
      grouped_tiles<OP, OUT, MODE, 256><<<cus, Shape<256>::kThreads, 0, s>>>(g);
      return;
    }
  }
  grouped_tiles<OP, OUT, MODE, 128><<<2 * cus, Shape<128>::kThreads, 0, s>>>(g);
}
template <int OP, int OUT>
static void launch_tiles(const GroupedArgs& g, bool small, int cus, hipStream_t s) {
  if (by_eight(g))
    launch_tiles<OP, OUT, kDma>(g, small, cus, s);
  else if (std::min(g.n, g.k) >= 8)
    launch_tiles<OP, OUT, kRegisters>(g, small, cus, s);
  else
    launch_tiles<OP, OUT, kSingles>(g, small, cus, s);
}

static int64_t tiles(int64_t n, int64_t s) { return (n + s - 1) / s; }

// Whether 128 x 128 tiles are faster than 256 x 256. They read each operand
// twice as often (65536 rows, 32 experts of 2048 x 7168: 2536 us against
// 1731), but there are four times as many of them, and a batch wastes less of
// them at the experts' ends. So: few rows per expert, where reading the weights
// is the work (4096 rows, 128 experts of 768 x 2048: 87 us against 101; 1024
// rows, 32 experts of 2048 x 7168: 192 against 185), or fewer tiles than would
// occupy the card (2048 rows, 8 experts of 2048 x 2048: 34 us against 42; 8192
// rows: 96 against 92).
static bool small_tiles(GroupedOp op, const GroupedArgs& g, int cus) {
  if (g.splits > 1 || g.rows <= 32 * (int64_t)g.E || std::min(g.n, g.k) < 8) return true;
  if (op == GROUPED_DW) return g.E * tiles(g.n, 256) * tiles(g.k, 256) < cus;
  // half a tile per expert is lost at its end, about
  const int64_t n = op == GROUPED_Y ? g.n : g.k;
  return (std::min<int64_t>(g.E, g.rows) + tiles(g.rows, 64)) * tiles(n, 128) <= cus * 7 / 2;
}

// Parts that the contraction is cut into where the tiles are far fewer than
// compute units and each would work through a long one alone (a stage of 32
// takes 0.25 us, whoever waits for it): as many as bring 256 items, of eight
// stages at least. 16384 rows, dW of 256 x 256: 119 us whole, 18 in parts; 64
// rows, y of 256 over 8192: 66 and 11; over 1024: 12.5 and 10.2. Below that the
// second launch costs what the parts gain; 512 items are no faster (16384 rows,
// dW of 1024 x 512: 32 us against 29). Constants, so that the order of the sums
// does not depend on the device.
int grouped_splits(GroupedOp op, int64_t rows, int E, int64_t n, int64_t k) {
  constexpr int64_t kItems = 256, kStages = 8, kMost = 64;
  if (rows == 0) return 1;
  const int64_t of_rows = std::min<int64_t>(E, rows) + rows / 128;
  const int64_t count = op == GROUPED_DW  ? E * tiles(n, 128) * tiles(k, 128)
                        : op == GROUPED_Y ? of_rows * tiles(n, 128)
                                          : of_rows * tiles(k, 128);
  const int64_t stages = tiles(op == GROUPED_DW ? rows / E : op == GROUPED_Y ? k : n, kStep);
  if (stages < 32) return 1;
  return (int)std::max<int64_t>(1, std::min({kItems / count, stages / kStages, kMost}));
}
size_t grouped_scratch(GroupedOp op, int64_t rows, int E, int64_t n, int64_t k) {
  const int parts = grouped_splits(op, rows, E, n, k);
  GroupedArgs g{};
  g.rows = rows, g.E = E, g.n = n, g.k = k;
  return parts > 1 ? (size_t)parts * out_elements(op, g) * 4 : 0;
}

template <int OP>
static void launch_op(const GroupedArgs& g, bool small, int cus, hipStream_t s) {
  if (g.splits > 1) {
    launch_tiles<OP, kParts>(g, true, cus, s);
    const int64_t blocks = tiles(out_elements(OP, g), 256);
    grouped_join<OP><<<(unsigned)std::min<int64_t>(blocks, 8 * cus), 256, 0, s>>>(g);
  } else if (OP == GROUPED_DW && g.out_fp32) {
    launch_tiles<OP, OP == GROUPED_DW ? kF32 : kBf16>(g, small, cus, s);
  } else {
    launch_tiles<OP, kBf16>(g, small, cus, s);
  }
}

hipError_t launch_grouped(GroupedOp op, const GroupedArgs& args, int cus, hipStream_t s) {
  GroupedArgs g = args;
  // A few rows per expert: every weight is used for 16 rows at most (8 rows,
  // 128 experts of 768 x 2048: 9 us against 28 with tiles; 256 rows 67 against 69,
  // 1024 rows 96 against 79). The host knows the average alone: where all of 256
  // rows chose one expert, its rows run 16 at a time on a few workgroups, 64 us
  // (83 spread evenly), and tiles would take 23.
  if (op == GROUPED_Y && by_eight(g) && g.rows <= 2 * (int64_t)g.E) {
    const dim3 grid((unsigned)((g.n + 15) / 16), (unsigned)std::min<int64_t>(g.E, g.rows));
    grouped_few<<<grid, kFewWaves * 64, 0, s>>>(g);
    return hipGetLastError();
  }
  g.splits = g.part ? grouped_splits(op, g.rows, g.E, g.n, g.k) : 1;
  const bool small = small_tiles(op, g, cus);
  switch (op) {
    case GROUPED_Y: launch_op<GROUPED_Y>(g, small, cus, s); break;
    case GROUPED_DX: launch_op<GROUPED_DX>(g, small, cus, s); break;
    default: launch_op<GROUPED_DW>(g, small, cus, s);
  }
  return hipGetLastError();
}

}  // namespace mok
