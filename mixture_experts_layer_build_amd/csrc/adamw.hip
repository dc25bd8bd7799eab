// AdamW over many tensors in one launch, moments in fp32 or in MXFP8.
//
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (lr / bc1) m / (sqrt(v) / sqrt(bc2) + eps),   bc = 1 - beta^step
//
// fp32 arithmetic. p is the fp32 master where there is one (the bf16
// parameter is then its rounding), else the parameter itself.
//
// 8-bit states: m and r = sqrt(v), in 32-element blocks of E4M3 codes with
// one E8M0 scale each: the smallest power of two that keeps the block's
// largest magnitude within 448 of it (the quantizer's rule would clip the
// top eighth of a binade, and do so again at every step). The root halves
// the range: a block spans 2^35 in v. m is rounded to the nearest code. r
// is not: a step moves v by a (1 - b2)-th at most downwards, which is less
// than half a code, so the nearest code would be the old one for ever, and
// v would only ever grow. r goes to one of its two neighbouring codes a < b,
// up with the probability (r^2 - a^2) / (b^2 - a^2) that makes the mean of
// its square v. The probability meets u, one of 65536 midpoints of [0, 1)
// hashed from the element's number in the call and the call's seed, so a
// call with the same seed gives the same bits. A positive v below the
// smallest code is kept as that code: a moment that vanished would let the
// next update through undivided.
//
// Bound by HBM: 10 (bf16, 8 bits, no master) to 28 (bf16, fp32 states and
// master) bytes per element. 8 elements per lane and turn, lanes on
// consecutive chunks, a 32-element block in 4 neighbouring lanes. The
// tensors' addresses travel in the kernel's arguments, up to 48 per launch:
// nothing is copied to the device and nothing is kept between calls.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mok_internal.h"
#include "wave_ops.h"

namespace mok {
namespace {

constexpr int kMaxTensors = 48;
constexpr int kThreads = 256;
constexpr int kTurn = kThreads * 8;  // elements a workgroup handles at once

struct AdamTensor {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  uint32_t chunk0;   // first workgroup of the tensor in this launch
  uint32_t number0;  // number of its first element in the call (mod 2^32), a multiple of 32
  uint32_t vec;      // every address allows 16-byte (states in 8 bits: 8-byte) access
  uint32_t pad;
};

struct AdamArgs {
  AdamTensor t[kMaxTensors];
  const float* grad_scale;
  int32_t count;
  uint32_t chunk;  // elements per workgroup, a multiple of kTurn
  uint32_t seed;
  float b1, c1, b2, c2;    // c = 1 - b
  float keep, rate, rbc2, eps;  // 1 - lr wd, lr / bc1, 1 / sqrt(bc2)
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

// u for elements 2i and 2i + 1: one 32-bit hash (multiply and xor-shift
// rounds over the pair's number and the seed), 16 bits each.
__device__ __forceinline__ uint32_t pair_bits(uint32_t pair, uint32_t seed) {
  uint32_t x = pair * 0x9E3779B1u + seed;
  x ^= x >> 16;
  x *= 0x85157AF5u;
  x ^= x >> 15;
  x *= 0x2C1B3C6Du;
  x ^= x >> 16;
  return x;
}

// Smallest X with amax <= 448 * 2^X, from amax's bits; -127 for 0.
__device__ __forceinline__ int state_exponent(uint32_t amax) {
  if (amax == 0) return -127;
  const int x = mx_block_exponent(amax);
  return (amax >= 0x00800000u && (amax & 0x7FFFFFu) > 0x600000u) ? min(x + 1, 127) : x;
}

// The products and sums below are rounded one by one, as they are written
// (no fused multiply-add), and the root of an 8-bit state correctly: codes
// of 4 significant bits and bf16 gradients make exact ties common, and which
// way they go should not depend on the compiler's contraction.
#pragma clang fp contract(off)

// One of the two E4M3 values around r >= 0 (r <= 448), r^2 = sq: up where
// u * (hi^2 - lo^2) < sq - lo^2.
__device__ __forceinline__ float round_root(float r, float sq, float u) {
  // normal codes keep 3 bits of fp32's mantissa; below 2^-6 the codes are multiples of 2^-9
  const float lo_n = u2f(f2u(r) & 0xFFF00000u), hi_n = u2f((f2u(r) & 0xFFF00000u) + 0x100000u);
  const float lo_s = __builtin_floorf(r * 512.f) * 0x1p-9f;
  const bool normal = r >= 0x1p-6f;
  const float lo = normal ? lo_n : lo_s, hi = normal ? hi_n : lo_s + 0x1p-9f;
  float q = u * (hi * hi - lo * lo) < sq - lo * lo ? hi : lo;
  q = __builtin_fminf(q, 448.f);
  return sq > 0.f ? __builtin_fmaxf(q, 0x1p-9f) : q;
}

template <typename T>
__device__ __forceinline__ void get8(const T* p, int64_t i, int64_t n, bool vec, float (&v)[8]) {
  if (vec) {
    load8(p + i, v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = i + q < n ? load1(p + i + q) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int64_t i, int64_t n, bool vec, const float (&v)[8]) {
  if (vec) {
    store8(p + i, v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q < n) store1(p + i + q, v[q]);
  }
}
__device__ __forceinline__ uint2 get_codes(const uint8_t* p, int64_t i, int64_t n, bool vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p + i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (i + q < n) w[q >> 2] |= (uint32_t)p[i + q] << (8 * (q & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(uint8_t* p, int64_t i, int64_t n, bool vec, uint2 c) {
  if (vec) {
    *reinterpret_cast<uint2*>(p + i) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (i + q < n) p[i + q] = (uint8_t)(w[q >> 2] >> (8 * (q & 3)));
}
// Values of 8 codes under scale byte s (0xFF: NaN).
__device__ __forceinline__ void decode8(uint2 c, uint32_t s, float (&v)[8]) {
  const float scale = s == 0xFFu ? __builtin_nanf("") : u2f(s ? s << 23 : 0x00400000u);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = e4m3_decode_byte_scaled(c.x, q, 1.0f) * scale;
    v[4 + q] = e4m3_decode_byte_scaled(c.y, q, 1.0f) * scale;
  }
}

template <typename PT, bool MASTER, typename GT, bool S8>
__global__ void __launch_bounds__(kThreads) adamw_tensors(AdamArgs a) {
  // the workgroup's tensor: the last one that begins at or before it
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].chunk0 <= blockIdx.x)
      lo = mid;
    else
      hi = mid - 1;
  }
  const AdamTensor& t = a.t[lo];
  const int64_t n = t.n;
  const int64_t begin = (int64_t)(blockIdx.x - t.chunk0) * a.chunk;
  const int64_t end = min(n, begin + (int64_t)a.chunk);
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  // every thread makes the same number of turns (lanes of a block exchange maxima)
  for (int64_t i0 = begin; i0 < end; i0 += kTurn) {
    const int64_t i = i0 + (int64_t)threadIdx.x * 8;
    const bool in = i < n;
    const bool vec = t.vec && i + 8 <= n;
    float g[8], p[8], m[8], v[8];
    get8((const GT*)t.g, i, n, vec, g);
    if constexpr (MASTER)
      get8((const float*)t.master, i, n, vec, p);
    else
      get8((const PT*)t.p, i, n, vec, p);
    if constexpr (S8) {
      const uint2 cm = get_codes((const uint8_t*)t.m, i, n, vec), cv = get_codes((const uint8_t*)t.v, i, n, vec);
      decode8(cm, in ? t.ms[i >> 5] : 0u, m);
      decode8(cv, in ? t.vs[i >> 5] : 0u, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= v[q];
    } else {
      get8((const float*)t.m, i, n, vec, m);
      get8((const float*)t.v, i, n, vec, v);
    }
    float r[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[q] *= gs;
      m[q] = a.b1 * m[q] + a.c1 * g[q];
      v[q] = a.b2 * v[q] + a.c2 * (g[q] * g[q]);
      r[q] = S8 ? __builtin_sqrtf(v[q]) : __builtin_amdgcn_sqrtf(v[q]);
      p[q] = p[q] * a.keep - a.rate * m[q] * __builtin_amdgcn_rcpf(r[q] * a.rbc2 + a.eps);
    }
    if (in) {
      put8((PT*)t.p, i, n, vec, p);
      if constexpr (MASTER) put8(t.master, i, n, vec, p);
    }
    if constexpr (S8) {
      uint32_t mm = 0, mr = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        mm = max(mm, f2u(m[q]) & 0x7FFFFFFFu);
        mr = max(mr, f2u(r[q]) & 0x7FFFFFFFu);
      }
      mm = quad_max(mm);
      mr = quad_max(mr);
      const int xm = state_exponent(mm), xr = state_exponent(mr);
      const float down = __builtin_ldexpf(1.0f, -xr);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t bits = pair_bits((t.number0 + (uint32_t)i) / 2 + h, a.seed);
        const float rs0 = r[2 * h] * down, rs1 = r[2 * h + 1] * down;
        const float s0 = v[2 * h] * down * down, s1 = v[2 * h + 1] * down * down;
        r[2 * h] = round_root(rs0, s0, ((float)(bits & 0xFFFFu) + 0.5f) * 0x1p-16f);
        r[2 * h + 1] = round_root(rs1, s1, ((float)(bits >> 16) + 0.5f) * 0x1p-16f);
      }
      if (in) {
        put_codes((uint8_t*)t.m, i, n, vec,
                  make_uint2(e4m3x4_encode_scaled(m[0], m[1], m[2], m[3], xm),
                             e4m3x4_encode_scaled(m[4], m[5], m[6], m[7], xm)));
        put_codes((uint8_t*)t.v, i, n, vec,
                  make_uint2(e4m3x4_encode_scaled(r[0], r[1], r[2], r[3], 0),
                             e4m3x4_encode_scaled(r[4], r[5], r[6], r[7], 0)));
        if ((i & 31) == 0) {
          t.ms[i >> 5] = mm >= 0x7F800000u ? 0xFFu : (uint8_t)(xm + 127);
          t.vs[i >> 5] = mr >= 0x7F800000u ? 0xFFu : (uint8_t)(xr + 127);
        }
      }
    } else if (in) {
      put8((float*)t.m, i, n, vec, m);
      put8((float*)t.v, i, n, vec, v);
    }
  }
}

bool aligned(const void* p, uintptr_t to) { return (((uintptr_t)p) & (to - 1)) == 0; }

}  // namespace

hipError_t launch_adamw(const mok_adamw& u, int cus, hipStream_t s) {
  AdamArgs a{};
  a.grad_scale = u.grad_scale;
  a.seed = u.seed;
  a.b1 = (float)u.beta1, a.c1 = (float)(1.0 - u.beta1);
  a.b2 = (float)u.beta2, a.c2 = (float)(1.0 - u.beta2);
  a.keep = (float)(1.0 - u.lr * u.weight_decay);
  a.rate = (float)(u.lr / (1.0 - std::pow(u.beta1, (double)u.step)));
  a.rbc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(u.beta2, (double)u.step)));
  a.eps = (float)u.eps;
  int64_t total = 0;
  for (int i = 0; i < u.count; ++i) total += u.numels[i];
  // a workgroup takes 4 turns where that still gives every compute unit
  // several workgroups, else one
  a.chunk = total >= (int64_t)cus * 4 * 8 * kTurn ? 4 * kTurn : kTurn;
  auto launch = [&](int64_t blocks) -> hipError_t {
    auto go = [&](auto pt, auto master, auto gt, auto s8) {
      adamw_tensors<decltype(pt), decltype(master)::value, decltype(gt), decltype(s8)::value>
          <<<(unsigned)blocks, kThreads, 0, s>>>(a);
    };
    auto with_state = [&](auto pt, auto master, auto gt) {
      u.state_bits == 8 ? go(pt, master, gt, std::true_type{}) : go(pt, master, gt, std::false_type{});
    };
    auto with_grad = [&](auto pt, auto master) {
      u.grad_fp32 ? with_state(pt, master, float{}) : with_state(pt, master, uint16_t{});
    };
    if (u.param_fp32)
      with_grad(float{}, std::false_type{});
    else if (u.masters)
      with_grad(uint16_t{}, std::true_type{});
    else
      with_grad(uint16_t{}, std::false_type{});
    return hipGetLastError();
  };
  uint32_t number = 0;
  int64_t blocks = 0;
  for (int i = 0; i < u.count; ++i) {
    const int64_t n = u.numels[i];
    const int64_t need = (n + a.chunk - 1) / a.chunk;
    if (need > 0) {
      if (a.count == kMaxTensors || (a.count > 0 && blocks + need > 0x7FFFFFFF)) {
        MOK_HIP_TRY(launch(blocks));
        a.count = 0;
        blocks = 0;
      }
      AdamTensor& t = a.t[a.count++];
      t.p = u.params[i];
      t.g = u.grads[i];
      t.master = u.masters ? (float*)u.masters[i] : nullptr;
      t.m = u.exp_avgs[i];
      t.v = u.exp_avg_sqs[i];
      t.ms = u.state_bits == 8 ? (uint8_t*)u.exp_avg_scales[i] : nullptr;
      t.vs = u.state_bits == 8 ? (uint8_t*)u.exp_avg_sq_scales[i] : nullptr;
      t.n = n;
      t.chunk0 = (uint32_t)blocks;
      t.number0 = number;
      const uintptr_t st = u.state_bits == 8 ? 8 : 16;
      t.vec = aligned(t.p, 16) && aligned(t.g, 16) && aligned(t.master, 16) && aligned(t.m, st) && aligned(t.v, st);
      blocks += need;
    }
    number += (uint32_t)((n + 31) / 32 * 32);
  }
  return a.count > 0 ? launch(blocks) : hipSuccess;
}

}  // namespace mok
