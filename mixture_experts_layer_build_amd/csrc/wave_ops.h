// Cross-lane reductions on DPP (data-parallel primitives): the operand of a
// VALU instruction comes from another lane of the same row of 16, so a step
// costs one instruction and no LDS round trip. Rotating a row by 8, 4, 2 and
// 1 lanes leaves the row's result in every lane; the four rows of a wave64
// are then joined through scalar registers. Every order is fixed, so a sum
// has the same bits on every run.
//
// All 64 lanes of the wave must be active.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.h"

namespace mok {

#if defined(__HIP_DEVICE_COMPILE__)
template <int CTRL>
__device__ __forceinline__ int dpp_mov(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, true);
}
#else
template <int CTRL>
__device__ int dpp_mov(int x);  // device only
#endif
template <int CTRL>
__device__ __forceinline__ float dpp_movf(float x) {
  return u2f((uint32_t)dpp_mov<CTRL>((int)f2u(x)));
}

constexpr int kMirror = 0x140, kHalfMirror = 0x141;                        // row_mirror, row_half_mirror
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;  // row_ror:n
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;                          // quad_perm:[1,0,3,2], [2,3,0,1]
constexpr int kQuadLane0 = 0x00, kQuadLane1 = 0x55;                        // quad_perm:[0,0,0,0], [1,1,1,1]

// Over 8 consecutive lanes.
__device__ __forceinline__ float octet_sum(float x) {
  x += dpp_movf<kQuadXor1>(x);
  x += dpp_movf<kQuadXor2>(x);
  return x + dpp_movf<kHalfMirror>(x);
}
__device__ __forceinline__ float octet_maxf(float x) {
  x = __builtin_fmaxf(x, dpp_movf<kQuadXor1>(x));
  x = __builtin_fmaxf(x, dpp_movf<kQuadXor2>(x));
  return __builtin_fmaxf(x, dpp_movf<kHalfMirror>(x));
}
__device__ __forceinline__ int octet_min(int x) {
  x = min(x, dpp_mov<kQuadXor1>(x));
  x = min(x, dpp_mov<kQuadXor2>(x));
  return min(x, dpp_mov<kHalfMirror>(x));
}

// x, as a value the compiler knows nothing of.
__device__ __forceinline__ int opaque(int x) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(x));
#endif
  return x;
}

// Over the 16 lanes of a row.
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_movf<kRor8>(x);
  x += dpp_movf<kRor4>(x);
  x += dpp_movf<kRor2>(x);
  x += dpp_movf<kRor1>(x);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
  x = __builtin_fmaxf(x, dpp_movf<kRor8>(x));
  x = __builtin_fmaxf(x, dpp_movf<kRor4>(x));
  x = __builtin_fmaxf(x, dpp_movf<kRor2>(x));
  x = __builtin_fmaxf(x, dpp_movf<kRor1>(x));
  return x;
}
__device__ __forceinline__ int row_min(int x) {
  x = min(x, dpp_mov<kRor8>(x));
  x = min(x, dpp_mov<kRor4>(x));
  x = min(x, dpp_mov<kRor2>(x));
  x = min(x, dpp_mov<kRor1>(x));
  return x;
}

// Lane l's value in every lane (a scalar register).
__device__ __forceinline__ int lane_value(int x, int l) { return __builtin_amdgcn_readlane(x, l); }
__device__ __forceinline__ float lane_valuef(float x, int l) {
  return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(x), l));
}

// Over the 64 lanes of the wave.
__device__ __forceinline__ float wave_sum(float x) {
  x = row_sum(x);
  return (lane_valuef(x, 0) + lane_valuef(x, 16)) + (lane_valuef(x, 32) + lane_valuef(x, 48));
}
// The same in fp64: a sum whose last additions should not round.
template <int CTRL>
__device__ __forceinline__ double dpp_movd(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)dpp_mov<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp_mov<CTRL>((int)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_valued(double x, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)lane_value((int)(uint32_t)u, l), hi = (uint32_t)lane_value((int)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double x) {
  x += dpp_movd<kRor8>(x);
  x += dpp_movd<kRor4>(x);
  x += dpp_movd<kRor2>(x);
  x += dpp_movd<kRor1>(x);
  return (lane_valued(x, 0) + lane_valued(x, 16)) + (lane_valued(x, 32) + lane_valued(x, 48));
}
__device__ __forceinline__ float wave_max(float x) {
  x = row_max(x);
  return __builtin_fmaxf(__builtin_fmaxf(lane_valuef(x, 0), lane_valuef(x, 16)),
                         __builtin_fmaxf(lane_valuef(x, 32), lane_valuef(x, 48)));
}
__device__ __forceinline__ int wave_min(int x) {
  x = row_min(x);
  return min(min(lane_value(x, 0), lane_value(x, 16)), min(lane_value(x, 32), lane_value(x, 48)));
}

// Orders a wave's LDS accesses before and behind it among its own lanes (LDS
// serves a wave's instructions in order; this keeps the compiler from moving
// them).
__device__ __forceinline__ void wave_lds_fence() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#endif
}

// Largest value of 8 consecutive lanes (a block at 4 elements per lane).
__device__ __forceinline__ uint32_t quad_max(uint32_t x);
__device__ __forceinline__ uint32_t octet_max(uint32_t x) {
  x = quad_max(x);
  return max(x, (uint32_t)dpp_mov<kHalfMirror>((int)x));
}

// Largest value of 4 consecutive lanes (a 32-element block at 8 per lane).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, (uint32_t)dpp_mov<kQuadXor1>((int)x));
  return max(x, (uint32_t)dpp_mov<kQuadXor2>((int)x));
}

// 8 consecutive elements as fp32, from 16-byte aligned bf16 or fp32.
__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = u2f(w[i] << 16);
    v[2 * i + 1] = u2f(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
// The last-level cache: launches that touch more load past it where that
// measured faster.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;
// The same past the caches' keeping (non-temporal), for data that one launch
// streams through and none reads again soon. bf16 lanes fill whole lines per
// instruction; fp32 ones, at 32 bytes a lane, only with the second, so for
// them it depends on the rest of the launch and is measured case by case.
typedef __attribute__((ext_vector_type(4))) float f32x4nt;
__device__ __forceinline__ uint4 load16_once(const void* p) {
  const u32x4 r = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store16_once(void* p, uint4 r) {
  __builtin_nontemporal_store((u32x4){r.x, r.y, r.z, r.w}, reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void load8_once(const uint16_t* p, float (&v)[8]) { unpack8(load16_once(p), v); }
__device__ __forceinline__ void load8_once(const float* p, float (&v)[8]) {
  const f32x4nt a = __builtin_nontemporal_load(reinterpret_cast<const f32x4nt*>(p)),
                b = __builtin_nontemporal_load(reinterpret_cast<const f32x4nt*>(p + 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void store8_once(uint16_t* p, const float (&v)[8]) {
  store16_once(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7])));
}
__device__ __forceinline__ void store8_once(float* p, const float (&v)[8]) {
  __builtin_nontemporal_store((f32x4nt){v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4nt*>(p));
  __builtin_nontemporal_store((f32x4nt){v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4nt*>(p + 4));
}
// W = 8 or 4 elements per lane, past the caches if STREAM. fp32 takes 4: one
// 16-byte access, which fills whole lines.
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2nt;
template <bool STREAM>
__device__ __forceinline__ void load_lane(const uint16_t* p, float (&v)[8]) {
  STREAM ? load8_once(p, v) : load8(p, v);
}
template <bool STREAM>
__device__ __forceinline__ void load_lane(const uint16_t* p, float (&v)[4]) {
  const u32x2nt* q = reinterpret_cast<const u32x2nt*>(p);
  const u32x2nt r = STREAM ? __builtin_nontemporal_load(q) : *q;
  v[0] = u2f(r[0] << 16), v[1] = u2f(r[0] & 0xFFFF0000u), v[2] = u2f(r[1] << 16), v[3] = u2f(r[1] & 0xFFFF0000u);
}
template <bool STREAM>
__device__ __forceinline__ void load_lane(const float* p, float (&v)[4]) {
  const f32x4nt* q = reinterpret_cast<const f32x4nt*>(p);
  const f32x4nt r = STREAM ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = r[i];
}
template <bool STREAM>
__device__ __forceinline__ void load_lane(const float* p, float (&v)[8]) {
  load8(p, v);
}
__device__ __forceinline__ void store_once(uint16_t* p, const float (&v)[8]) { store8_once(p, v); }
__device__ __forceinline__ void store_once(uint16_t* p, const float (&v)[4]) {
  __builtin_nontemporal_store((u32x2nt){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, reinterpret_cast<u32x2nt*>(p));
}
__device__ __forceinline__ void store_once(float* p, const float (&v)[4]) {
  __builtin_nontemporal_store((f32x4nt){v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4nt*>(p));
}

// A lane's elements as they lie in memory, 16 bytes of the wider type beside
// them: 8 of bf16, or 4 with fp32 rows. fresh() makes the compiler forget what
// the registers were converted to, so that a later pair() converts again
// instead of keeping the fp32 values alive.
template <typename T, int W>
struct Raw;
template <>
struct Raw<uint16_t, 8> {
  uint4 r = make_uint4(0, 0, 0, 0);
  template <bool STREAM>
  __device__ __forceinline__ void load(const uint16_t* p) {
    r = STREAM ? load16_once(p) : *reinterpret_cast<const uint4*>(p);
  }
  // elements 2j and 2j + 1
  __device__ __forceinline__ void pair(int j, float& a, float& b) const {
    const uint32_t x = j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w;
    a = u2f(x << 16), b = u2f(x & 0xFFFF0000u);
  }
  __device__ __forceinline__ void set(int j, float a, float b) {
    (j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w) = pack_bf16x2(a, b);
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(uint16_t* p) const {
    if (STREAM)
      store16_once(p, r);
    else
      *reinterpret_cast<uint4*>(p) = r;
  }
  __device__ __forceinline__ void fresh() {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(r.x), "+v"(r.y), "+v"(r.z), "+v"(r.w));
#endif
  }
};
template <>
struct Raw<uint16_t, 4> {
  uint32_t r[2] = {};
  template <bool STREAM>
  __device__ __forceinline__ void load(const uint16_t* p) {
    const u32x2nt* q = reinterpret_cast<const u32x2nt*>(p);
    const u32x2nt x = STREAM ? __builtin_nontemporal_load(q) : *q;
    r[0] = x[0], r[1] = x[1];
  }
  __device__ __forceinline__ void pair(int j, float& a, float& b) const {
    a = u2f(r[j] << 16), b = u2f(r[j] & 0xFFFF0000u);
  }
  __device__ __forceinline__ void set(int j, float a, float b) { r[j] = pack_bf16x2(a, b); }
  template <bool STREAM>
  __device__ __forceinline__ void store(uint16_t* p) const {
    u32x2nt* q = reinterpret_cast<u32x2nt*>(p);
    const u32x2nt x = {r[0], r[1]};
    if (STREAM)
      __builtin_nontemporal_store(x, q);
    else
      *q = x;
  }
  __device__ __forceinline__ void fresh() {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(r[0]), "+v"(r[1]));
#endif
  }
};
template <int W>
struct Raw<float, W> {
  f32x4nt v_[W / 4] = {};
  template <bool STREAM>
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const f32x4nt* q = reinterpret_cast<const f32x4nt*>(p) + i;
      v_[i] = STREAM && W == 4 ? __builtin_nontemporal_load(q) : *q;
    }
  }
  __device__ __forceinline__ void pair(int j, float& a, float& b) const {
    a = v_[j / 2][2 * (j & 1)], b = v_[j / 2][2 * (j & 1) + 1];
  }
  __device__ __forceinline__ void set(int j, float a, float b) {
    v_[j / 2][2 * (j & 1)] = a, v_[j / 2][2 * (j & 1) + 1] = b;
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(float* p) const {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      f32x4nt* q = reinterpret_cast<f32x4nt*>(p) + i;
      if (STREAM && W == 4)
        __builtin_nontemporal_store(v_[i], q);
      else
        *q = v_[i];
    }
  }
  __device__ __forceinline__ void fresh() {}
};
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

}  // namespace mok
