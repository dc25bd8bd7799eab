// Matrix products grouped by expert, rows given by offsets: y = x W_e^T per
// expert, and its gradients dx = dy W_e and dW_e = dy^T x.
//
// All three are C[m, n] = sum over k of A(m, k) B(n, k), with other roles:
//         m                n             contraction     A          B
//   y     e's rows         W's rows      W's columns     x          W_e
//   dx    e's rows         W's columns   W's rows        dy         W_e^T
//   dW    W's rows         W's columns   e's rows        dy^T       x^T
#include <algorithm>

#include "device_common.h"
#include "mok_internal.h"

namespace mok {
namespace {

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
// by the whole workgroup. `part`: one int per wave.
template <int NTHR>
__device__ __forceinline__ void scan_tiles(const GroupedArgs& g, int bm, int32_t* tiles, int32_t* part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
    if (lane == 63) part[wave] = s;
    __syncthreads();
    int before = base, all = base;
    for (int w = 0; w < NTHR / 64; ++w) {
      if (w < wave) before += part[w];
      all += part[w];
    }
    if (e < g.E) tiles[e] = before + s - cnt;
    base = all;
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
// Every width, stride and alignment: 64 x 64 output tiles, operands loaded
// element by element along whichever index is dense, four waves of one 32 x 32
// MFMA tile each.
// ---------------------------------------------------------------------------
constexpr int kAnyTile = 64, kAnyK = 32, kAnyThreads = 256;

template <int OP>
__global__ void __launch_bounds__(kAnyThreads) grouped_any(GroupedArgs g) {
  constexpr int LD = kAnyK + 8;  // 80-byte rows: 16-byte reads of 32 rows without bank conflicts
  __shared__ alignas(16) uint16_t As[kAnyTile * LD], Bs[kAnyTile * LD];
  __shared__ int32_t tiles[kGroupedMaxExperts + 1], part[kAnyThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lh = lane >> 5, wm = wave >> 1, wn = wave & 1;
  const int M = OP == GROUPED_DW ? (int)g.n : 0;
  const int N = (int)(OP == GROUPED_Y ? g.n : g.k);
  const int nt = (N + kAnyTile - 1) / kAnyTile;
  int64_t all;
  if (OP == GROUPED_DW) {
    all = (int64_t)g.E * ((M + kAnyTile - 1) / kAnyTile) * nt;
  } else {
    scan_tiles<kAnyThreads>(g, kAnyTile, tiles, part);
    all = (int64_t)tiles[g.E] * nt;
  }
  for (int64_t t = blockIdx.x; t < all; t += gridDim.x) {
    const int ni = (int)(t % nt), mt = (int)(t / nt);
    const int mts = (M + kAnyTile - 1) / kAnyTile;
    const int e = OP == GROUPED_DW ? mt / mts : expert_of(tiles, g.E, mt);
    int lo, hi;
    segment(g, e, lo, hi);
    const int m0 = (OP == GROUPED_DW ? mt - e * mts : mt - tiles[e]) * kAnyTile, n0 = ni * kAnyTile;
    const int mrows = OP == GROUPED_DW ? M : hi - lo;
    const int K = (int)(OP == GROUPED_Y ? g.k : OP == GROUPED_DX ? g.n : hi - lo);
    const uint16_t* A = (const uint16_t*)g.a + (int64_t)lo * g.ld_a;
    const uint16_t* B = (const uint16_t*)g.b + (OP == GROUPED_DW ? (int64_t)lo * g.ld_b : (int64_t)e * g.n * g.k);
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    for (int k0 = 0; k0 < K; k0 += kAnyK) {
#pragma unroll
      for (int i = 0; i < kAnyTile * kAnyK / kAnyThreads; ++i) {
        const int at = i * kAnyThreads + tid;
        {  // A
          const int m = OP == GROUPED_DW ? at % kAnyTile : at / kAnyK;
          const int k = OP == GROUPED_DW ? at / kAnyTile : at % kAnyK;
          uint16_t v = 0;
          if (m0 + m < mrows && k0 + k < K)
            v = OP == GROUPED_DW ? A[(int64_t)(k0 + k) * g.ld_a + m0 + m] : A[(int64_t)(m0 + m) * g.ld_a + k0 + k];
          As[m * LD + k] = v;
        }
        {  // B
          const int n = OP == GROUPED_Y ? at / kAnyK : at % kAnyTile;
          const int k = OP == GROUPED_Y ? at % kAnyK : at / kAnyTile;
          uint16_t v = 0;
          if (n0 + n < N && k0 + k < K)
            v = OP == GROUPED_Y    ? B[(int64_t)(n0 + n) * g.k + k0 + k]
                : OP == GROUPED_DX ? B[(int64_t)(k0 + k) * g.k + n0 + n]
                                   : B[(int64_t)(k0 + k) * g.ld_b + n0 + n];
          Bs[n * LD + k] = v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < kAnyK / 16; ++ks) {
        const bf16x8 fa = *reinterpret_cast<const bf16x8*>(As + (wm * 32 + lr) * LD + ks * 16 + lh * 8);
        const bf16x8 fb = *reinterpret_cast<const bf16x8*>(Bs + (wn * 32 + lr) * LD + ks * 16 + lh * 8);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb, fa, acc, 0, 0, 0);
      }
      __syncthreads();
    }
    // accumulator r of a lane: row lr, column 8 (r / 4) + 4 lh + r % 4 of its 32 x 32 tile
    const int m = m0 + wm * 32 + lr;
    if (m < mrows) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int n = n0 + wn * 32 + 8 * (r / 4) + 4 * lh + r % 4;
        if (n >= N) continue;
        if (OP == GROUPED_DW) {
          const int64_t at = ((int64_t)e * g.n + m) * g.k + n;
          if (g.out_fp32)
            ((float*)g.out)[at] = acc[r];
          else
            ((uint16_t*)g.out)[at] = f32_to_bf16(acc[r]);
        } else {
          ((uint16_t*)g.out)[(int64_t)(lo + m) * g.ld_out + n] = f32_to_bf16(acc[r]);
        }
      }
    }
  }
  if (OP != GROUPED_DW && g.zero_rest) zero_rest(g, N);
}

}  // namespace

hipError_t launch_grouped(GroupedOp op, const GroupedArgs& g, int cus, hipStream_t s) {
  const int grid = cus * 4;
  switch (op) {
    case GROUPED_Y: grouped_any<GROUPED_Y><<<grid, kAnyThreads, 0, s>>>(g); break;
    case GROUPED_DX: grouped_any<GROUPED_DX><<<grid, kAnyThreads, 0, s>>>(g); break;
    default: grouped_any<GROUPED_DW><<<grid, kAnyThreads, 0, s>>>(g); break;
  }
  return hipGetLastError();
}

}  // namespace mok
