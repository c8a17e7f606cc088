// 8-bit Adam moments, device side.
//
// A block is kCodedBlock = 64 consecutive elements with one FP32 scale for
// each moment.
//   m: s = max |m| over the block (0 when that is below 2^-100: such a block is
//      held as zeros); code = the FP8 e4m3 value (4 exponent, 3 mantissa bits,
//      bias 7, one sign) nearest 256 * m / s.  m = code * (s / 256).
//   v: r = sqrt(v), s = max r (FP32's largest root where that is infinite);
//      code = the unsigned float of 4 exponent bits (bias 15) and 4 mantissa
//      bits with gradual underflow nearest r / s, at least the smallest nonzero
//      one when r > 0.  v = (code * s)^2.
// The root halves v's exponent range, so that 16 binades of codes reach 2^-36
// of the block's largest v, and a v > 0 never becomes 0, which would turn
// m / (sqrt(v) + eps) into m / eps.  A block's largest element gets the code of
// exactly 256 (m) or 1 (v), so decoding it gives the scale's own bits, and
// encoding a decoded block gives the same codes and scales again.
// Rounding is to nearest even, half a step at most: 2^-4 of m, 2^-5 of sqrt(v).
//
// A lane holds 4 consecutive elements, so a block is one DPP row of 16 lanes:
// its maximum takes four row rotations, no LDS.  All comparisons are of the
// bits of non-negative floats as unsigned integers, which order like the
// floats with every NaN above infinity: a NaN reaches the scale and through it
// the whole block, instead of being dropped as a floating-point maximum would.
#pragma once

#include "lane.h"
#include "plan.h"

namespace gro {
namespace {

constexpr float kCodeTop = 256.0f;        // e4m3 value of a block's largest |m|
constexpr uint32_t kRootTop = 240;        // v's code of 1.0
constexpr float kScaleFloor = 0x1p-100f;  // 256 / s stays far from overflow above it
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kRootMaxBits = 0x5f7fffffu;  // the largest FP32 whose square is finite: 2^64 - 2^40

// 1 / x rounded to nearest: the hardware reciprocal and one Newton step, for x
// from 2^-108 to 2^120 (a scale, or a scale / 256), where neither it nor the
// remainder leaves the normal range.  Equal to the IEEE division for every
// mantissa, tested at exponents near both ends and between them, at 6 issue
// slots -- a transcendental instruction takes 4 -- instead of 13.
__device__ __forceinline__ float reciprocal(float x) {
  const float y = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, y, 1.0f), y, y);
}

// Maximum of an unsigned value over each row of 16 lanes, in every lane.
// All 64 lanes of the wave must be active.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  // DPP control 0x120 + n rotates a row right by n lanes.
  x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x128, 0xf, 0xf, true)));
  x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x124, 0xf, 0xf, true)));
  x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x122, 0xf, 0xf, true)));
  x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x121, 0xf, 0xf, true)));
  return x;
}

__device__ __forceinline__ uint32_t max4_bits(const f32x4 x) {
  return max(max(__float_as_uint(x.x), __float_as_uint(x.y)), max(__float_as_uint(x.z), __float_as_uint(x.w)));
}

// Four e4m3 codes (element 0 in the low byte) times s / 256.
__device__ __forceinline__ f32x4 decode_m4(uint32_t c, float scale) {
  const float k = scale * (1.0f / kCodeTop);
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(c), false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(c), true);
  return f32x4{lo.x * k, lo.y * k, hi.x * k, hi.y * k};
}

// The four second moments: a code is bits 6..13 of the FP16 of its value.
__device__ __forceinline__ f32x4 decode_v4(uint32_t c, float scale) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint16_t h = uint16_t(((c >> (8 * e)) & 0xffu) << 6);
    const float r = float(__builtin_bit_cast(_Float16, h)) * scale;
    v[e] = r * r;
  }
  return v;
}

// Codes of one lane's four elements and their block's scale; elements that do
// not exist are passed as 0.
struct Coded4 {
  uint32_t codes;
  float scale;
};

__device__ __forceinline__ Coded4 encode_m4(const f32x4 m) {
  const f32x4 a = {fabsf(m.x), fabsf(m.y), fabsf(m.z), fabsf(m.w)};
  float s = __uint_as_float(row_max(max4_bits(a)));
  if (s < kScaleFloor) s = 0.0f;
  const float inv = s == 0.0f ? 0.0f : reciprocal(s * (1.0f / kCodeTop));
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(m.x * inv, m.y * inv, 0, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(m.z * inv, m.w * inv, c, true);
  return Coded4{uint32_t(c), s};
}

// r: the square roots.  r / s times 2^-112 has the code's exponent and
// mantissa in its own top bits (gradual underflow included, as FP32's own
// subnormals), so rounding to a code is an integer add and a shift.
__device__ __forceinline__ Coded4 encode_root4(const f32x4 r) {
  uint32_t top = row_max(max4_bits(r));
  if (top == kInfBits) top = kRootMaxBits;
  const float s = __uint_as_float(top);
  const float inv = top == 0 ? 0.0f : reciprocal(s);
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t z = __float_as_uint((r[e] * inv) * 0x1p-112f);
    uint32_t c = (z + 0x3ffffu + ((z >> 19) & 1u)) >> 19;
    c = min(max(c, min(__float_as_uint(r[e]), 1u)), kRootTop);
    codes |= c << (8 * e);
  }
  return Coded4{codes, s};
}

}  // namespace
}  // namespace gro
