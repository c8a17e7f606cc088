// Device helpers shared by the gfx950 kernels: lane-vector types and loads,
// widening and rounding, the workgroup sum, gradient inputs and one element's
// clip + AdamW.  Every floating-point step is one IEEE-rounded operation (the
// library is built without contraction).  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gro {
namespace {

// Lanes per workgroup, a compile-time launch-shape knob.  The norm's
// per-chunk summation order depends on it, so a build has one fixed value.
#ifndef GRO_BLOCK
#define GRO_BLOCK 256
#endif
constexpr int kBlock = GRO_BLOCK;      // lanes per workgroup (waves of 64)
constexpr int kWaves = kBlock / 64;
static_assert(kBlock % 64 == 0 && kBlock <= 1024, "whole wave64s");

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// x / d for a positive integer d.  When d is a power of two its reciprocal
// is exact and x * (1/d) is the same correctly rounded value as x / d, so
// the multiply is used; otherwise an IEEE division.
struct Divisor {
  float d;
  float inv;
  int pow2;
};

__host__ __device__ inline Divisor make_divisor(int d) {
  Divisor r;
  r.d = float(d);
  r.inv = 1.0f / float(d);
  r.pow2 = (d & (d - 1)) == 0;
  return r;
}

__device__ __forceinline__ float divide(float x, const Divisor& q) {
  return q.pow2 ? x * q.inv : x / q.d;
}

// The same choice made at compile time, for the branch-free full-chunk paths:
// kNoDiv (nothing to divide), kMulInv (power-of-two divisor), kIeeeDiv.
enum DivMode { kNoDiv = 0, kMulInv = 1, kIeeeDiv = 2 };
__host__ __device__ inline int div_mode(const Divisor& q) { return q.pow2 ? kMulInv : kIeeeDiv; }
template <int M>
__device__ __forceinline__ float divide_m(float x, const Divisor& q) {
  if constexpr (M == kMulInv) return x * q.inv;
  else if constexpr (M == kIeeeDiv) return x / q.d;
  else return x;
}

// Four BF16 (two 32-bit words, element 0 in the low half) widened exactly.
__device__ __forceinline__ f32x4 widen4(const u32x2 r) {
  f32x4 x;
  x.x = __uint_as_float(r.x << 16);
  x.y = __uint_as_float(r.x & 0xffff0000u);
  x.z = __uint_as_float(r.y << 16);
  x.w = __uint_as_float(r.y & 0xffff0000u);
  return x;
}

__device__ __forceinline__ float widen1(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// FP32 -> BF16, round to nearest even, two per v_cvt_pk_bf16_f32:
// lo in bits 0..15, hi in 16..31.
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint16_t bf16_bits(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

__device__ __forceinline__ f32x4 ld4f(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void st4f(float* p, const f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
// Streaming variants with the non-temporal cache policy.  They are used for
// every stream a step touches once -- the gradient contributions and
// AdamW's p, m, v and BF16 copy -- so that these do not push the FP32
// accumulator out of the memory-side Infinity Cache between the pass that
// writes it and the AdamW pass that reads it, and so that AdamW leaves few
// dirty lines for the next step's first pass to drain.  The accumulator
// itself keeps the default policy.
__device__ __forceinline__ u32x2 ld2u_nt(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
}
__device__ __forceinline__ f32x4 ld4f_nt(const float* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
}
__device__ __forceinline__ void st4f_nt(float* p, const f32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(p));
}
__device__ __forceinline__ void st2u_nt(uint16_t* p, const u32x2 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x2*>(p));
}
// An accumulator store with the policy fixed at compile time (a run-time
// choice between the two stores is merged into one plain store by the
// compiler).
template <bool NT>
__device__ __forceinline__ void st4f_acc(float* p, const f32x4 v) {
  if constexpr (NT) st4f_nt(p, v);
  else st4f(p, v);
}

// Sum over the workgroup in a fixed order: a wave64 butterfly (every lane
// ends with the same bits because IEEE addition commutes), then the wave
// totals in wave order.  Returned in every lane.
[[maybe_unused]] __device__ double block_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  __shared__ double part[kWaves];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double t = part[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) t += part[w];
  return t;
}

// Chunk index of this workgroup, placed so that q == blockIdx.x (mod 8).
__device__ __forceinline__ int64_t chunk_of_block(int64_t q_begin) {
  return q_begin - (q_begin & 7) + int64_t(blockIdx.x);
}

__device__ __forceinline__ double sq(float x) {
  const double d = double(x);
  return d * d;
}

// ------------------------------------------------------ gradient inputs
// A bucket's gradient contributions are BF16 (widened exactly) or FP32 (used
// as they are); the element type is a template parameter of every path.
// Vector loads of contributions are non-temporal (each is read once a step).
struct Bf16In {
  typedef u32x2 raw_t;
  static __device__ __forceinline__ raw_t load(const void* base, int64_t e) {
    return ld2u_nt(static_cast<const uint16_t*>(base) + e);
  }
  static __device__ __forceinline__ f32x4 widen(const raw_t r) { return widen4(r); }
  static __device__ __forceinline__ float load1(const void* base, int64_t i) {
    return widen1(static_cast<const uint16_t*>(base)[i]);
  }
};
struct F32In {
  typedef f32x4 raw_t;
  static __device__ __forceinline__ raw_t load(const void* base, int64_t e) {
    return ld4f_nt(static_cast<const float*>(base) + e);
  }
  static __device__ __forceinline__ f32x4 widen(const raw_t r) { return r; }
  static __device__ __forceinline__ float load1(const void* base, int64_t i) {
    return static_cast<const float*>(base)[i];
  }
};

// ------------------------------------------------------- clip + AdamW
struct AdamScalars {
  Divisor wdiv;
  float coef, decay, b1, b2, omb1, omb2, step_size, sbc2, eps;
};

// g = acc/n; g^ = g*coef; p = p*decay; m = b1*m + (1-b1)*g^;
// v = b2*v + (1-b2)*(g^*g^); p = p - step_size*(m/(sqrt(v)/sqrt_bc2 + eps)).
template <int WM>
__device__ __forceinline__ void adamw_elem(float a, float& p, float& m, float& v, const AdamScalars& k) {
  const float g = WM == kNoDiv ? divide(a, k.wdiv) : divide_m<WM>(a, k.wdiv);
  const float gh = g * k.coef;
  p = p * k.decay;
  m = k.b1 * m + k.omb1 * gh;
  v = k.b2 * v + k.omb2 * (gh * gh);
  const float d = sqrtf(v) / k.sbc2 + k.eps;
  p = p - k.step_size * (m / d);
}

template <int WM>
__device__ __forceinline__ void adamw4(const f32x4 a, f32x4& p, f32x4& m, f32x4& v, const AdamScalars& k) {
  float pp[4] = {p.x, p.y, p.z, p.w}, mm[4] = {m.x, m.y, m.z, m.w}, vv[4] = {v.x, v.y, v.z, v.w};
  const float aa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) adamw_elem<WM>(aa[e], pp[e], mm[e], vv[e], k);
  p = f32x4{pp[0], pp[1], pp[2], pp[3]};
  m = f32x4{mm[0], mm[1], mm[2], mm[3]};
  v = f32x4{vv[0], vv[1], vv[2], vv[3]};
}

__device__ __forceinline__ void store_bf16x4(uint16_t* pb, const f32x4 p) {
  st2u_nt(pb, u32x2{bf16x2_bits(p.x, p.y), bf16x2_bits(p.z, p.w)});
}

// The accumulator's load: the default policy, so that a step's last
// accumulate pass's final stretch is met in the Infinity Cache, or (NT) the
// non-temporal one, for accumulators that pass stored non-temporally.
template <bool NT>
__device__ __forceinline__ f32x4 ld4f_acc(const float* p) {
  if constexpr (NT) return ld4f_nt(p);
  else return ld4f(p);
}

}  // namespace
}  // namespace gro
