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
// master) bytes per element. 8 elements per lane and turn. With 8-bit states
// they are neighbours, so that a 32-element block lies in 4 lanes; with fp32
// states, whose 32 bytes per lane would touch every line and fill none, they
// are two groups of 4, each of which fills lines with every instruction.
// The tensors' addresses travel in the kernel's arguments, up to 48 per
// launch: nothing is copied to the device and nothing is kept between calls.
//
// Measured now: 1e8 bf16 elements with masters 464-473 us with fp32 states
// (5.9-6.0 TB/s), 260 with 8 bits (6.2 TB/s), 165-170 with 8 bits and no masters
// (6.0-6.1 TB/s); 1e8 fp32 elements 470 with fp32 states, 274 with 8 bits.
//
// What led there, each pair timed in turn on the code of its time (1e8 bf16
// elements unless a number is given):
//   8-bit update with packed conversions, the hardware's root and no clamps (it
//     was bound by its instructions): no masters 229 -> 165 us
//   stores past the caches always, loads only where the tensors exceed the
//     last-level cache (STREAM): 8 bits with masters 329 -> 289, fp32 states with
//     masters 517 with loads through the caches, 473 past them; 1e7 elements, which
//     the cache holds, 41 and 46, so there they go through it
//   one turn per workgroup instead of four: see TABLE below
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
// rounds over the pair's number and the seed), 16 bits each. x = the pair's
// number * kPairStep + seed. Of the odd multipliers this asks only that any
// flipped bit of x flips each bit of the hash about every other time (between
// 49.1 and 50.9 % over 2^20 draws) and that the two halves, and neighbouring
// pairs, are not correlated (below 0.2 %). The oracle holds the same ones.
constexpr uint32_t kPairStep = 0x9E3779B1u;
__device__ __forceinline__ uint32_t pair_bits(uint32_t x) {
  x ^= x >> 16;
  x *= 0x85157AF5u;
  x ^= x >> 15;
  x *= 0x2C1B3C6Du;
  x ^= x >> 16;
  return x;
}

// Smallest X >= -127 with amax <= 448 * 2^X, from amax's bits: 448 is 1.75 *
// 2^8. (At most 120, for the largest fp32 values.)
__device__ __forceinline__ int state_exponent(uint32_t amax) {
  return max((int)(amax >> 23) - (127 + 8) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0), -127);
}

// The products and sums of the moments are rounded one by one, as they are
// written (no fused multiply-add): codes of 4 significant bits and bf16
// gradients make exact ties common, and which way they go should not depend
// on the compiler's contraction.
#pragma clang fp contract(off)

// One of the two E4M3 values around r (at most 448), r^2 = sq: up where u *
// (hi^2 - lo^2) < sq - lo^2. An r that its own rounding carried across a
// code decides the same way from either side of it.
__device__ __forceinline__ float round_between(float lo, float hi, float sq, float u) {
  const float lo2 = lo * lo;
  return u * (hi * hi - lo2) < sq - lo2 ? hi : lo;
}
// Normal codes keep 3 bits of fp32's mantissa.
__device__ __forceinline__ float round_root(float r, float sq, float u) {
  const uint32_t lo = f2u(r) & 0xFFF00000u;
  return round_between(u2f(lo), u2f(lo + 0x100000u), sq, u);
}
// Below 2^-6 the codes are multiples of 2^-9; a positive r keeps at least one.
__device__ __forceinline__ float round_small_root(float r, float sq, float u) {
  const float lo = __builtin_floorf(r * 512.f) * 0x1p-9f;
  const float q = round_between(lo, lo + 0x1p-9f, sq, u);
  return sq > 0.f ? __builtin_fmaxf(q, 0x1p-9f) : q;
}

template <bool NT, typename T>
__device__ __forceinline__ void get8(const T* p, int64_t i, int64_t n, bool vec, float (&v)[8]) {
  if (vec) {
    NT ? load8_once(p + i, v) : load8(p + i, v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = i + q < n ? load1(p + i + q) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int64_t i, int64_t n, bool vec, const float (&v)[8]) {
  if (vec) {
    store8_once(p + i, v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q < n) store1(p + i + q, v[q]);
  }
}
// The same for a lane's two groups of 4 elements, kHalf apart.
constexpr int kHalf = kThreads * 4;
template <bool NT, typename T>
__device__ __forceinline__ void get4x2(const T* p, int64_t i, int64_t n, bool vec, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h, i += kHalf) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec && i + 4 <= n) {
      load_lane<NT>(p + i, x);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q < n) x[q] = load1(p + i + q);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) v[4 * h + q] = x[q];
  }
}
template <typename T>
__device__ __forceinline__ void put4x2(T* p, int64_t i, int64_t n, bool vec, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h, i += kHalf) {
    const float x[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    if (vec && i + 4 <= n) {
      store_once(p + i, x);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q < n) store1(p + i + q, x[q]);
    }
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
#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ bool is_subnormal(float x) { return __builtin_amdgcn_classf(x, 0x90); }
// Values of 8 codes under scale byte s (not 0xFF), two per instruction.
__device__ __forceinline__ void decode8(uint2 c, uint32_t s, float (&v)[8]) {
  const float scale = u2f(s ? s << 23 : 0x00400000u);
  const f32x2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, scale, false);
  const f32x2v b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, scale, true);
  const f32x2v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, scale, false);
  const f32x2v e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, scale, true);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = d[0], v[5] = d[1], v[6] = e[0], v[7] = e[1];
}
// Codes of 8 values, all at most 448 in magnitude.
__device__ __forceinline__ uint2 encode8(const float (&v)[8]) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const float s = 1.0f;
  s16x2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[0], v[1], s, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[2], v[3], s, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[4], v[5], s, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[6], v[7], s, true);
  return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}
#else
__device__ bool is_subnormal(float x);  // device only
__device__ void decode8(uint2 c, uint32_t s, float (&v)[8]);
__device__ uint2 encode8(const float (&v)[8]);
#endif

// 2^k as the math library's power function gives it: exact, or half an ulp
// below (k = 16 to 20, 22, 24, 25, 28, 29, 32, ...). The states are scaled by
// it because elementary tensor operations on this GPU scale so, and a step
// gives the codes that those operations give, bit for bit. The half ulp shows
// only where m is half way between two codes, both equally near: then the
// smaller one is taken, not the even one. That is no rare case: a bf16 gradient
// and a code of 4 bits often add up to few bits (0.25 % of the codes of a step
// on gradients of a normal distribution), and with the exact power two steps'
// parameters differ from those of the elementary operations by 5e-5 of them.
// (The base is hidden, or the compiler would take exp2.)
__device__ __forceinline__ float library_power(int k) {
  return powf(u2f((uint32_t)opaque(0x40000000)), (float)k);
}

// TABLE: the workgroup makes a table of the powers first and takes four turns;
// else it takes one turn and finds them as it goes. Workgroups of one turn
// sweep memory as a closer front: with fp32 states, which need no powers, 541
// -> 514 us against four turns (1e8 bf16 elements with masters, 8 neighbouring
// elements per lane then), with 8 bits 280 -> 260 (fp32 parameters 287 -> 274).
// Where an element moves only 10 bytes (8 bits, bf16, no masters) the powers'
// instructions weigh more than that: 165 us with the table, 188 without.
template <typename PT, bool MASTER, typename GT, bool S8, bool TABLE, bool STREAM>
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
  // 2^-X and 2^-2X for scale byte X + 127
  __shared__ float down[TABLE ? 256 : 1], down2[TABLE ? 256 : 1];
  if constexpr (TABLE) {
    static_assert(kThreads == 256, "a thread per scale byte");
    down[threadIdx.x] = library_power(127 - (int)threadIdx.x);
    down2[threadIdx.x] = library_power(2 * (127 - (int)threadIdx.x));
    __syncthreads();
  }
  // every thread makes the same number of turns (lanes of a block exchange maxima)
  for (int64_t i0 = begin; i0 < end; i0 += kTurn) {
    const int64_t i = i0 + (int64_t)threadIdx.x * (S8 ? 8 : 4);
    const bool in = i < n;
    const bool vec = t.vec && (!S8 || i + 8 <= n);
    auto get = [&](auto* p, float(&v)[8]) {
      if constexpr (S8)
        get8<STREAM>(p, i, n, vec, v);
      else
        get4x2<STREAM>(p, i, n, vec, v);
    };
    auto put = [&](auto* p, const float(&v)[8]) {
      if constexpr (!S8)
        put4x2(p, i, n, vec, v);
      else if (in)
        put8(p, i, n, vec, v);
    };
    float g[8], p[8], m[8], v[8];
    get((const GT*)t.g, g);
    if constexpr (MASTER)
      get((const float*)t.master, p);
    else
      get((const PT*)t.p, p);
    if constexpr (S8) {
      const uint2 cm = get_codes((const uint8_t*)t.m, i, n, vec), cv = get_codes((const uint8_t*)t.v, i, n, vec);
      const uint32_t sm = in ? t.ms[i >> 5] : 0u, sv = in ? t.vs[i >> 5] : 0u;
      decode8(cm, sm, m);
      decode8(cv, sv, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= v[q];
      if (max(sm, sv) == 0xFFu) {  // NaN
#pragma unroll
        for (int q = 0; q < 8; ++q) m[q] = sm == 0xFFu ? __builtin_nanf("") : m[q], v[q] = sv == 0xFFu ? __builtin_nanf("") : v[q];
      }
    } else {
      get((const float*)t.m, m);
      get((const float*)t.v, v);
    }
    float r[8];
    bool tiny = false;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[q] *= gs;
      m[q] = a.b1 * m[q] + a.c1 * g[q];
      v[q] = a.b2 * v[q] + a.c2 * (g[q] * g[q]);
      r[q] = __builtin_amdgcn_sqrtf(v[q]);
      tiny |= is_subnormal(v[q]);
    }
    if (tiny) {  // the hardware's root takes a subnormal v for 0
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (is_subnormal(v[q])) r[q] = __builtin_amdgcn_sqrtf(v[q] * 0x1p64f) * 0x1p-32f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float inv = __builtin_amdgcn_rcpf(__builtin_fmaf(r[q], a.rbc2, a.eps));
      p[q] = __builtin_fmaf(-a.rate * m[q], inv, p[q] * a.keep);
    }
    put((PT*)t.p, p);
    if constexpr (MASTER) put(t.master, p);
    if constexpr (S8) {
      // a moment that is not finite comes with a v that is not
      float mm = 0.f;
      uint32_t mr = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        mm = __builtin_fmaxf(mm, __builtin_fabsf(m[q]));
        mr = max(mr, f2u(r[q]));
      }
      mr = quad_max(mr);
      const int xm = state_exponent(quad_max(f2u(mm))), xr = state_exponent(min(mr, 0x7F7FFFFFu));
      float fm, fv;  // 2^-X of m, 2^-2X of r
      if constexpr (TABLE) {
        fm = down[xm + 127], fv = down2[xr + 127];
      } else {  // even lanes of the block's four find the one, odd ones the other
        const float power = library_power(threadIdx.x & 1 ? -2 * xr : -xm);
        fm = dpp_movf<kQuadLane0>(power), fv = dpp_movf<kQuadLane1>(power);
      }
      fv = mr ? fv : 0.f;
      const float fr = u2f((uint32_t)(127 - xr) << 23);
      uint32_t x = (t.number0 + (uint32_t)i) / 2 * kPairStep + a.seed;
      bool small = false;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        m[q] *= fm;
        r[q] *= fr;
        v[q] = fv < __builtin_inff() ? v[q] * fv : v[q] * fr * fr;
        small |= r[q] < 0x1p-6f;
      }
      float u[8];
#pragma unroll
      for (int h = 0; h < 4; ++h, x += kPairStep) {
        const uint32_t bits = pair_bits(x);
        u[2 * h] = __builtin_fmaf((float)(bits & 0xFFFFu), 0x1p-16f, 0x1p-17f);
        u[2 * h + 1] = __builtin_fmaf((float)(bits >> 16), 0x1p-16f, 0x1p-17f);
      }
      if (small) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          r[q] = r[q] < 0x1p-6f ? round_small_root(r[q], v[q], u[q]) : round_root(r[q], v[q], u[q]);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = round_root(r[q], v[q], u[q]);
      }
      if (in) {
        put_codes((uint8_t*)t.m, i, n, vec, encode8(m));
        put_codes((uint8_t*)t.v, i, n, vec, encode8(r));
        if ((i & 31) == 0) {
          const bool finite = mr < 0x7F800000u;
          t.ms[i >> 5] = finite ? (uint8_t)(xm + 127) : 0xFFu;
          t.vs[i >> 5] = finite ? (uint8_t)(xr + 127) : 0xFFu;
        }
      }
    } else {
      put((float*)t.m, m);
      put((float*)t.v, v);
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
  // (four turns only where that still gives every compute unit several workgroups)
  const bool table =
      u.state_bits == 8 && !u.param_fp32 && !u.masters && total >= (int64_t)cus * 4 * 8 * kTurn;
  a.chunk = table ? 4 * kTurn : kTurn;
  const int64_t each = (u.param_fp32 ? 4 : u.masters ? 6 : 2) + (u.grad_fp32 ? 4 : 2) + (u.state_bits == 8 ? 2 : 8);
  const bool stream = total * each > kCacheBytes;
  auto launch = [&](int64_t blocks) -> hipError_t {
    auto go = [&](auto pt, auto master, auto gt, auto s8, auto tab) {
      using PT = decltype(pt);
      using GT = decltype(gt);
      constexpr bool M = decltype(master)::value, S8 = decltype(s8)::value, TABLE = decltype(tab)::value;
      if (stream)
        adamw_tensors<PT, M, GT, S8, TABLE, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
      else
        adamw_tensors<PT, M, GT, S8, TABLE, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    };
    const std::true_type yes;
    const std::false_type no;
    auto with_state = [&](auto pt, auto master, auto gt) {
      if (u.state_bits != 8) return go(pt, master, gt, no, no);
      if constexpr (std::is_same<decltype(pt), uint16_t>::value && !decltype(master)::value)
        if (table) return go(pt, master, gt, yes, yes);
      go(pt, master, gt, yes, no);
    };
    auto with_grad = [&](auto pt, auto master) {
      u.grad_fp32 ? with_state(pt, master, float{}) : with_state(pt, master, uint16_t{});
    };
    if (u.param_fp32)
      with_grad(float{}, no);
    else if (u.masters)
      with_grad(uint16_t{}, yes);
    else
      with_grad(uint16_t{}, no);
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
