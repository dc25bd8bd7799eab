// RMS norm with the residual's addition, forward and backward.
//
//   forward   s = x + residual;  rstd = (mean(s^2) + eps)^-1/2;  y = s * rstd * w
//   backward  xh = s * rstd, g = dy * w:  ds = rstd * (g - xh * mean(g * xh)) + dsum,
//             dw = sum over rows of dy * xh
//
// Everything between a load and a store is fp32, but for the row's statistics:
// the threads' sums of squares are added, and rstd is found, in fp64 (a few
// instructions a row, no slower). The sum is stored in the residual's type,
// and y is computed from the fp32 sum before that rounding, so each output is
// rounded once. The backward starts from the stored sum.
//
// Both directions are bound by HBM: an element costs a few flops and 4 to 14
// bytes. A row is held in registers between its statistics and its output,
// so each byte is moved once. 8 elements (16 bytes of bf16) per lane and
// load, lanes on consecutive chunks; a row belongs to one wave up to 2048
// columns, whose reduction needs no barrier, and to 256 or 512 threads
// above (a wave would need more registers than keep enough loads in
// flight). The backward holds three streams and dw, so a lane takes at most
// two such chunks of a row (with four it needed 166 registers or spilled: 246 us
// against 176 at 16384 x 7168). The grid is persistent: the weights stay in
// registers from row to row, and the backward adds dw up in registers over a
// workgroup's rows, writes one partial row per workgroup, and a second launch
// adds the partials in a fixed order (no atomics: the same bits on every
// run).
//
// Measured: forward 8192 x 2048 bf16 with residual 23.4 us (5.7 TB/s), 16384 x
// 7168 160 us, to MXFP8 134 us (6.2 TB/s); backward 16384 x 7168 with d_sum
// 162 us (5.8 TB/s), of fp32 rows 285 us, 8192 x 2048 27 us. A copy of 4 GiB
// runs at 4.6 TB/s.
#include <algorithm>
#include <type_traits>

#include "mok_internal.h"
#include "wave_ops.h"

namespace mok {
namespace {

// E4M3 codes and E8M0 scale of a lane's W elements of a 32-element block (32
// / W consecutive lanes), by the block rule of the quantizer (X = clamp(floor(
// log2 amax) - 8, -127, 127)). A block that holds an infinity or a NaN gets
// the NaN scale 0xFF, and the layer's products with it are NaN.
template <int W>
__device__ __forceinline__ void store_mxfp8(const float (&y)[W], uint8_t* codes, uint8_t* scale, bool first) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) amax = max(amax, f2u(y[i]) & 0x7FFFFFFFu);
  amax = W == 8 ? quad_max(amax) : octet_max(amax);
  const int X = mx_block_exponent(amax);
  const uint32_t lo = e4m3x4_encode_scaled(y[0], y[1], y[2], y[3], X);
  if constexpr (W == 8)
    *reinterpret_cast<uint2*>(codes) = make_uint2(lo, e4m3x4_encode_scaled(y[4], y[5], y[6], y[7], X));
  else
    *reinterpret_cast<uint32_t*>(codes) = lo;
  if (first) *scale = amax >= 0x7F800000u ? 0xFFu : (uint8_t)(X + 127);
}

// Sum over the TPR threads of a row. Waves join through LDS, in two sets of
// slots used in turn, so that one barrier per row is enough: a set is
// written again only after the barrier that follows its last read.
template <int TPR, typename T>
__device__ __forceinline__ T row_threads_sum(T x, T* slots, int group, int parity) {
  x = wave_sum(x);
  if constexpr (TPR == 64) return x;
  constexpr int W = TPR / 64;
  T* mine = slots + (parity * (int)(blockDim.x / TPR) + group) * W;
  const int wave = (int)(threadIdx.x % TPR) / 64;
  if (lane_id() == 0) mine[wave] = x;
  __syncthreads();
  T s = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) s += mine[i];
  return s;
}

#if defined(__HIP_DEVICE_COMPILE__)
// (sum of squares / cols + eps)^-1/2 to fp64's precision or nearly: the
// hardware's estimate and one Newton step.
__device__ __forceinline__ double row_rstd(double ss, int cols, float eps) {
  const double x = ss / (double)cols + (double)eps;
  const double r = __builtin_amdgcn_rsq(x);
  return x > 0.0 && x < __builtin_inf() ? r * (1.5 - 0.5 * x * r * r) : r;
}
#else
__device__ double row_rstd(double ss, int cols, float eps);  // device only
#endif

struct NormFwd {
  const void *x, *residual, *w;
  int w_fp32;
  int64_t rows, ld_x, ld_res;
  int cols;
  float eps;
  void* sum;        // residual's type; null without a residual
  uint16_t* y;      // null: not written
  uint8_t* codes;   // null: not written
  uint8_t* scale;
  float* rstd;      // null: not written
};

template <typename XT, typename RT>
constexpr int lane_width = std::is_same<RT, float>::value ? 4 : 8;

// RT: the residual's type, void for none. A lane takes 8 elements per load (16
// bytes of bf16), or 4 where the residual and the sum are fp32 (16 bytes of
// them): at 32 bytes a lane an instruction touches every line and fills none
// (bf16 x, fp32 residual, 16384 x 7168 to MXFP8 250 -> 221 us, 4096 x 2048 22
// -> 17; fp32 x without a residual only reads fp32, 18 us against 21).
template <typename XT, typename RT, bool STREAM, int BLOCK, int TPR, int NV>
__global__ void __launch_bounds__(BLOCK) rms_norm_rows(NormFwd a) {
  constexpr bool kRes = !std::is_void<RT>::value;
  using R = typename std::conditional<kRes, RT, float>::type;
  constexpr int W = lane_width<XT, RT>;
  constexpr int RPB = BLOCK / TPR;
  __shared__ double slots[2 * RPB * (TPR / 64)];
  // (a row's waves are whole waves, so its number and addresses are scalars)
  const uint32_t t = threadIdx.x % TPR;
  const int group = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const uint32_t nchunk = (uint32_t)a.cols / W;
  float w[NV][W];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = t + i * TPR;
#pragma unroll
    for (int q = 0; q < W; ++q) w[i][q] = 0.f;
    if (c < nchunk) {
      if (a.w_fp32)
        load_lane<false>((const float*)a.w + c * W, w[i]);
      else
        load_lane<false>((const uint16_t*)a.w + c * W, w[i]);
    }
  }
  int parity = 0;
  // every thread of the workgroup makes the same number of turns (barrier inside)
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB, parity ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < a.rows;
    const XT* x = (const XT*)a.x + row * a.ld_x;
    const R* res = (const R*)a.residual + row * a.ld_res;
    float v[NV][W];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = t + i * TPR;
      if (live && c < nchunk) {
        load_lane<STREAM>(x + c * W, v[i]);
        if constexpr (kRes) {
          float r[W];
          load_lane<STREAM>(res + c * W, r);
#pragma unroll
          for (int q = 0; q < W; ++q) v[i][q] += r[q];
        }
      } else {
#pragma unroll
        for (int q = 0; q < W; ++q) v[i][q] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < W; ++q) ss = __builtin_fmaf(v[i][q], v[i][q], ss);
    const double exact = row_rstd(row_threads_sum<TPR>((double)ss, slots, group, parity), a.cols, a.eps);
    const float rstd = (float)exact, rest = (float)(exact - (double)rstd);
    if (!live) continue;
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    const int64_t out = row * a.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = t + i * TPR;
      if (c >= nchunk) continue;
      if constexpr (kRes) store_once((R*)a.sum + out + c * W, v[i]);
      float y[W];
      if (a.codes) {
        // y rounded once to fp32, so that as few codes as can be fall on the
        // wrong side of a boundary: rstd and rstd * w in two parts each
#pragma unroll
        for (int q = 0; q < W; ++q) {
          const float hi = w[i][q] * rstd;
          const float lo = __builtin_fmaf(w[i][q], rstd, -hi) + w[i][q] * rest;
          y[q] = __builtin_fmaf(v[i][q], hi, v[i][q] * lo);
        }
      } else {
#pragma unroll
        for (int q = 0; q < W; ++q) y[q] = v[i][q] * rstd * w[i][q];
      }
      if (a.y) store_once(a.y + out + c * W, y);
      if (a.codes) store_mxfp8(y, a.codes + out + c * W, a.scale + (out >> 5) + c / (32 / W), t % (32 / W) == 0);
    }
  }
}

// Any width, stride and alignment: one workgroup per row, one element per
// lane and load, the row read twice (the second time from cache). Two-byte
// loads and the second pass are what it costs: 4096 x 5003 bf16 with residual 63
// us, 4096 x 20480 287 (floors 35 and 145); the backward, which also adds dw up
// in memory, 188 and 1250. Widths of models take the other kernel.
template <typename XT, typename RT>
__global__ void __launch_bounds__(256) rms_norm_any(NormFwd a) {
  constexpr bool kRes = !std::is_void<RT>::value;
  using R = typename std::conditional<kRes, RT, float>::type;
  __shared__ double slots[2 * 4];
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const XT* x = (const XT*)a.x + row * a.ld_x;
    const R* res = (const R*)a.residual + row * a.ld_res;
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      float v = load1(x + c);
      if constexpr (kRes) v += load1(res + c);
      ss = __builtin_fmaf(v, v, ss);
    }
    const float rstd = (float)row_rstd(row_threads_sum<256>((double)ss, slots, 0, parity), a.cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      float v = load1(x + c);
      if constexpr (kRes) {
        v += load1(res + c);
        store1((R*)a.sum + row * a.cols + c, v);
      }
      const float w = a.w_fp32 ? ((const float*)a.w)[c] : load1((const uint16_t*)a.w + c);
      if (a.y) store1(a.y + row * a.cols + c, v * rstd * w);
    }
  }
}

struct NormBwd {
  const uint16_t* dy;
  const void *s, *dsum, *w;
  const float* rstd;
  int w_fp32;
  int64_t rows, ld_dy, ld_s, ld_dsum;
  int cols;
  void* ds;         // s's type
  uint16_t* dx;     // bf16 copy of ds; null: not written
  float* dw_part;   // [workgroups, cols]
};

// A row's dy, s and d_sum stay as they were loaded and are converted twice,
// in the pass before the row's sum and in the one behind it: in fp32 they
// would take twice the registers, and half the waves would hide the loads.
// fp32 rows take 4 elements per lane, as in the forward, and go past the caches
// where the launch exceeds them (16384 x 7168 with d_sum 305 -> 285 us, without
// 216 -> 204; 8192 x 4096 90 -> 84; 4096 x 512, which the cache holds, 9.8 ->
// 10.1).
template <typename ST>
constexpr int bwd_width = std::is_same<ST, float>::value ? 4 : 8;
__device__ __forceinline__ void store_floats(float* p, const float (&v)[8]) { store8(p, v); }
__device__ __forceinline__ void store_floats(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <typename ST, typename WT, bool DSUM, bool STREAM, int BLOCK, int TPR, int NV>
__global__ void __launch_bounds__(BLOCK) __attribute__((amdgpu_waves_per_eu(4)))
rms_norm_bwd_rows(NormBwd a) {
  constexpr int W = bwd_width<ST>;
  constexpr int RPB = BLOCK / TPR;
  static_assert(BLOCK % TPR == 0, "whole rows");
  __shared__ float slots[2 * RPB * (TPR / 64)];
  __shared__ float dw_lds[RPB > 1 ? TPR * NV * W : 1];
  // (a row's waves are whole waves, so its number and addresses are scalars)
  const uint32_t t = threadIdx.x % TPR;
  const int group = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const uint32_t nchunk = (uint32_t)a.cols / W;
  Raw<WT, W> w[NV];
  float dw[NV][W];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = t + i * TPR;
#pragma unroll
    for (int q = 0; q < W; ++q) dw[i][q] = 0.f;
    if (c < nchunk) w[i].template load<false>((const WT*)a.w + c * W);
  }
  const float inv_cols = 1.0f / (float)a.cols;
  int parity = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB, parity ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < a.rows;
    const float rstd = live ? a.rstd[row] : 0.f;
    const uint16_t* pdy = a.dy + row * a.ld_dy;
    const ST* ps = (const ST*)a.s + row * a.ld_s;
    const ST* pd = (const ST*)a.dsum + row * a.ld_dsum;
    ST* pds = (ST*)a.ds + row * a.cols;
    uint16_t* pdx = a.dx + row * a.cols;
    Raw<uint16_t, W> dy[NV];
    Raw<ST, W> s[NV], dsum[DSUM ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = t + i * TPR;
      if (live && c < nchunk) {
        dy[i].template load<STREAM>(pdy + c * W);
        s[i].template load<STREAM>(ps + c * W);
        if constexpr (DSUM) dsum[i].template load<STREAM>(pd + c * W);
      }
    }
    float along = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      w[i].fresh();
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        float d[2], x[2], wv[2];
        dy[i].pair(j, d[0], d[1]);
        s[i].pair(j, x[0], x[1]);
        w[i].pair(j, wv[0], wv[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float xh = x[q] * rstd;
          dw[i][2 * j + q] = __builtin_fmaf(d[q], xh, dw[i][2 * j + q]);
          along = __builtin_fmaf(d[q] * wv[q], xh, along);
        }
      }
    }
    along = row_threads_sum<TPR>(along, slots, group, parity) * inv_cols;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = t + i * TPR;
      if (c >= nchunk) continue;
      w[i].fresh();
      dy[i].fresh();
      s[i].fresh();
      Raw<ST, W> ds;
      Raw<uint16_t, W> narrow;
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        float d[2], x[2], wv[2], more[2] = {0.f, 0.f};
        dy[i].pair(j, d[0], d[1]);
        s[i].pair(j, x[0], x[1]);
        w[i].pair(j, wv[0], wv[1]);
        if constexpr (DSUM) dsum[i].pair(j, more[0], more[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) d[q] = rstd * (d[q] * wv[q] - x[q] * rstd * along) + more[q];
        ds.set(j, d[0], d[1]);
        narrow.set(j, d[0], d[1]);
      }
      ds.template store<STREAM>(pds + c * W);
      if (a.dx) narrow.template store<STREAM>(pdx + c * W);
    }
  }
  // the workgroup's partial row: its row groups one after the other
  for (int g = 0; g < RPB; ++g) {
    if (RPB > 1) __syncthreads();
    if (group != g) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = t + i * TPR;
      if (c >= nchunk) continue;
      if constexpr (RPB > 1) {
        if (g > 0) {
          float have[W];
          load_lane<false>(dw_lds + c * W, have);
#pragma unroll
          for (int q = 0; q < W; ++q) dw[i][q] += have[q];
        }
        if (g < RPB - 1) store_floats(dw_lds + c * W, dw[i]);
      }
      if (g == RPB - 1) store_floats(a.dw_part + (int64_t)blockIdx.x * a.cols + c * W, dw[i]);
    }
  }
}

// dw_part is added to by the thread that owns a column of the workgroup
// (global memory, one workgroup's own row).
template <typename ST>
__global__ void __launch_bounds__(256) rms_norm_bwd_any(NormBwd a) {
  __shared__ float slots[2 * 4];
  const float inv_cols = 1.0f / (float)a.cols;
  float* part = a.dw_part + (int64_t)blockIdx.x * a.cols;
  for (int c = threadIdx.x; c < a.cols; c += 256) part[c] = 0.f;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const uint16_t* dy = a.dy + row * a.ld_dy;
    const ST* s = (const ST*)a.s + row * a.ld_s;
    const ST* dsum = (const ST*)a.dsum + row * a.ld_dsum;
    const float rstd = a.rstd[row];
    float along = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float w = a.w_fp32 ? ((const float*)a.w)[c] : load1((const uint16_t*)a.w + c);
      const float d = load1(dy + c), xh = load1(s + c) * rstd;
      part[c] += d * xh;
      along = __builtin_fmaf(d * w, xh, along);
    }
    along = row_threads_sum<256>(along, slots, 0, parity) * inv_cols;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float w = a.w_fp32 ? ((const float*)a.w)[c] : load1((const uint16_t*)a.w + c);
      float ds = rstd * (load1(dy + c) * w - load1(s + c) * rstd * along);
      if (a.dsum) ds += load1(dsum + c);
      store1((ST*)a.ds + row * a.cols + c, ds);
      if (a.dx) store1(a.dx + row * a.cols + c, ds);
    }
  }
}

// dw[c] = sum over the partial rows, in a fixed order: 16 threads per column
// take every 16th row, then their sums are added in order.
__global__ void __launch_bounds__(1024) reduce_dw_part(const float* __restrict__ part, int nparts, int cols,
                                                       void* dw, int w_fp32) {
  __shared__ float acc[16][64];
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int c = (int)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < cols)
#pragma unroll 4
    for (int r = g; r < nparts; r += 16) s += part[(int64_t)r * cols + c];
  acc[g][lane] = s;
  __syncthreads();
  if (g != 0 || c >= cols) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += acc[i][lane];
  if (w_fp32)
    ((float*)dw)[c] = s;
  else
    ((uint16_t*)dw)[c] = f32_to_bf16(s);
}

__global__ void zero_dw(void* dw, int cols, int w_fp32) {
  const int c = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  if (c >= cols) return;
  if (w_fp32)
    ((float*)dw)[c] = 0.f;
  else
    ((uint16_t*)dw)[c] = 0;
}

bool aligned16(const void* p) { return (((uintptr_t)p) & 15) == 0; }

// Inputs larger than the last-level cache (kCacheBytes) are loaded past it:
// what wrote them left nothing of them there that the first rows would still
// find. (16384 x 7168 bf16 with residual: 172 -> 166 us, to MXFP8 155 -> 139.
// Below, inputs that the cache still holds are worth more than that costs:
// 5003 x 7168 with an fp32 residual, 215 MB, past it 79 us for 64 if they are
// there, 80 for 82 if not. bf16 stores always go past it: 26 -> 24 us at 8192
// x 2048, 183 -> 172 at 16384 x 7168.)
template <typename XT, typename RT, int BLOCK, int TPR, int NV>
void run_fwd(const NormFwd& a, int cus, hipStream_t s) {
  const int64_t need = (a.rows + BLOCK / TPR - 1) / (BLOCK / TPR);
  const int grid = (int)std::min<int64_t>(need, (int64_t)cus * (2048 / BLOCK));
  constexpr int64_t kBytes = sizeof(XT) + (std::is_void<RT>::value ? 0 : std::is_same<RT, float>::value ? 4 : 2);
  if (a.rows * a.cols * kBytes > kCacheBytes)
    rms_norm_rows<XT, RT, true, BLOCK, TPR, NV><<<grid, BLOCK, 0, s>>>(a);
  else
    rms_norm_rows<XT, RT, false, BLOCK, TPR, NV><<<grid, BLOCK, 0, s>>>(a);
}

template <typename XT, typename RT>
void pick_fwd(const NormFwd& a, bool vec, int cus, hipStream_t s) {
  if (!vec) {
    rms_norm_any<XT, RT><<<(int)std::min<int64_t>(a.rows, (int64_t)cus * 8), 256, 0, s>>>(a);
    return;
  }
  const int c = a.cols;
  constexpr int M = 8 / lane_width<XT, RT>;  // twice the loads where a lane takes half
  if (c <= 512)
    run_fwd<XT, RT, 256, 64, 1 * M>(a, cus, s);
  else if (c <= 1024)
    run_fwd<XT, RT, 256, 64, 2 * M>(a, cus, s);
  else if (c <= 2048)
    run_fwd<XT, RT, 256, 64, 4 * M>(a, cus, s);
  else if (c <= 4096)
    run_fwd<XT, RT, 256, 256, 2 * M>(a, cus, s);
  else if (c <= 8192)
    run_fwd<XT, RT, 256, 256, 4 * M>(a, cus, s);
  else
    run_fwd<XT, RT, 512, 512, 4 * M>(a, cus, s);
}

// Workgroups of the backward, at most: two per compute unit, enough to fill
// the chip, few enough that the partial rows of dw stay a small share of the
// traffic. A constant, so the order of dw's sums does not depend on the
// device.
constexpr int kNormBwdParts = 512;

template <typename ST, typename WT, bool DSUM>
int run_bwd(const NormBwd& a, bool vec, hipStream_t s) {
  const int c = a.cols;
  auto grid = [&](int rows_per_block) {
    return (int)std::min<int64_t>((a.rows + rows_per_block - 1) / rows_per_block, kNormBwdParts);
  };
  const bool stream = a.rows * a.cols * (int64_t)(2 + (DSUM ? 2 : 1) * sizeof(ST)) > kCacheBytes;
  auto go = [&](auto block, auto tpr, auto nv) {
    constexpr int BLOCK = decltype(block)::value, TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    const int g = grid(BLOCK / TPR);
    if (stream)
      rms_norm_bwd_rows<ST, WT, DSUM, true, BLOCK, TPR, NV><<<g, BLOCK, 0, s>>>(a);
    else
      rms_norm_bwd_rows<ST, WT, DSUM, false, BLOCK, TPR, NV><<<g, BLOCK, 0, s>>>(a);
    return g;
  };
  using std::integral_constant;
  if (!vec) {
    rms_norm_bwd_any<ST><<<grid(1), 256, 0, s>>>(a);
    return grid(1);
  }
  constexpr int M = 8 / bwd_width<ST>;  // twice the chunks where a lane takes half
  if (c <= 512) return go(integral_constant<int, 512>{}, integral_constant<int, 64>{}, integral_constant<int, 1 * M>{});
  if (c <= 1024) return go(integral_constant<int, 512>{}, integral_constant<int, 64>{}, integral_constant<int, 2 * M>{});
  if (c <= 2048) return go(integral_constant<int, 512>{}, integral_constant<int, 256>{}, integral_constant<int, 1 * M>{});
  if (c <= 4096) return go(integral_constant<int, 512>{}, integral_constant<int, 256>{}, integral_constant<int, 2 * M>{});
  if (c <= 8192) return go(integral_constant<int, 512>{}, integral_constant<int, 512>{}, integral_constant<int, 2 * M>{});
  return go(integral_constant<int, 1024>{}, integral_constant<int, 1024>{}, integral_constant<int, 2 * M>{});
}

}  // namespace

int64_t norm_bwd_parts(int64_t rows) { return std::min<int64_t>(rows, kNormBwdParts); }

hipError_t launch_rms_norm(const NormArgs& n, int cus, hipStream_t s) {
  if (n.rows == 0) return hipSuccess;
  NormFwd a{n.x, n.residual, n.w, n.w_fp32, n.rows, n.ld_x, n.ld_res, (int)n.cols, n.eps, n.sum, (uint16_t*)n.y,
            n.codes, n.scale, n.rstd};
  const bool vec = n.cols % 8 == 0 && n.cols <= kNormMaxVecCols && n.ld_x % 8 == 0 && n.ld_res % 8 == 0 &&
                   aligned16(n.x) && aligned16(n.residual) && aligned16(n.w) && aligned16(n.sum) && aligned16(n.y);
  if (!vec && n.codes) return hipErrorInvalidValue;  // refused by the caller's checks
  if (!n.residual)
    n.x_fp32 ? pick_fwd<float, void>(a, vec, cus, s) : pick_fwd<uint16_t, void>(a, vec, cus, s);
  else if (n.x_fp32)
    pick_fwd<float, float>(a, vec, cus, s);
  else
    n.res_fp32 ? pick_fwd<uint16_t, float>(a, vec, cus, s) : pick_fwd<uint16_t, uint16_t>(a, vec, cus, s);
  return hipGetLastError();
}

hipError_t launch_rms_norm_bwd(const NormBwdArgs& n, hipStream_t s) {
  const int cols = (int)n.cols;
  if (n.rows == 0) {
    zero_dw<<<(cols + 255) / 256, 256, 0, s>>>(n.dw, cols, n.w_fp32);
    return hipGetLastError();
  }
  NormBwd a{(const uint16_t*)n.dy, n.s, n.dsum, n.w, n.rstd, n.w_fp32, n.rows, n.ld_dy, n.ld_s, n.ld_dsum, cols,
            n.ds, (uint16_t*)n.dx, n.dw_part};
  const bool vec = n.cols % 8 == 0 && n.cols <= kNormMaxVecCols && n.ld_dy % 8 == 0 && n.ld_s % 8 == 0 &&
                   n.ld_dsum % 8 == 0 && aligned16(n.dy) && aligned16(n.s) && aligned16(n.dsum) && aligned16(n.w) &&
                   aligned16(n.ds) && aligned16(n.dx);
  auto with_dsum = [&](auto st, auto wt) {
    using ST = decltype(st);
    using WT = decltype(wt);
    return n.dsum ? run_bwd<ST, WT, true>(a, vec, s) : run_bwd<ST, WT, false>(a, vec, s);
  };
  auto with_weight = [&](auto st) { return n.w_fp32 ? with_dsum(st, float{}) : with_dsum(st, uint16_t{}); };
  const int grid = n.s_fp32 ? with_weight(float{}) : with_weight(uint16_t{});
  MOK_HIP_TRY(hipGetLastError());
  reduce_dw_part<<<(cols + 63) / 64, 1024, 0, s>>>(n.dw_part, grid, cols, n.dw, n.w_fp32);
  return hipGetLastError();
}

}  // namespace mok
