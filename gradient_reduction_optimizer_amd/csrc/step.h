// One chunk's clip + AdamW with the moments in 32 bits or in 8-bit codes,
// device side.  A lane owns 4-element vectors lane, lane + kBlock, ... of its
// chunk, as in every pass, so with 8-bit moments a block of 64 elements is
// one row of 16 lanes (see coded.h).
//
//   g^ = g / window * coef;  m = b1 m + (1-b1) g^;  v = b2 v + (1-b2) g^^2
//   p = p decay - step_size m / (sqrt(v) / sbc2 + eps)
//
// All of it is one pass over memory: 18.25 bytes an element with 8-bit moments
// and a BF16 copy on an FP32 accumulator, 28 with FP32 moments on BF16
// gradients.  Four vectors per lane in flight measured best: an 8-bit step of
// 167M elements 446 us against 477 with two and 480 with one.
#pragma once

#include "coded.h"
#include "kernels.h"

namespace gro {
namespace {

struct StepScalars : AdamScalars {
  float inv_sbc2;      // 1 / sbc2 rounded to nearest
};

// The step's scalars with the clip coefficient of the norm.
__device__ __forceinline__ StepScalars step_scalars(const AdamWConsts& c, double norm, bool decayed) {
  StepScalars k;
  k.wdiv = make_divisor(c.window);
  k.coef = 1.0f;
  if (c.clip_on) {
    const double r = c.max_norm / (norm + 1e-6);
    k.coef = float(r < 1.0 ? r : 1.0);
  }
  k.decay = decayed ? c.decay : 1.0f;
  k.b1 = c.beta1;
  k.b2 = c.beta2;
  k.omb1 = c.one_minus_beta1;
  k.omb2 = c.one_minus_beta2;
  k.step_size = c.step_size;
  k.sbc2 = c.sqrt_bc2;
  k.inv_sbc2 = c.inv_sqrt_bc2;
  k.eps = c.eps;
  return k;
}

// r = sqrt(v) and q = r / sbc2, both rounded to nearest as the IEEE operations
// round.  For v from 2^-96 to the largest finite value, which is every v of a
// vector but in odd cases, with fewer issue slots (about 15 instead of 31):
//   r: the hardware reciprocal root y, g = v y, r = g + (v - g^2) y/2.  Equal to
//      the IEEE root for every FP32 in that range (all of them tested); below,
//      v - g^2 would round.
//   q: Markstein's division by a number whose reciprocal is rounded to nearest
//      (IBM J. Res. Dev. 34, 1990): a quotient within one step of the true one,
//      which the first correction gives, and one more correction round to
//      nearest.  r lies in [2^-48, 2^64] and sbc2 in [2^-27, 1], so no
//      remainder leaves the normal range.
__device__ __forceinline__ void roots4(const f32x4 v, const StepScalars& k, f32x4& r, f32x4& q) {
  const uint32_t b0 = __float_as_uint(v.x), b1 = __float_as_uint(v.y), b2 = __float_as_uint(v.z),
                 b3 = __float_as_uint(v.w);
  constexpr uint32_t kLow = 0x0f800000u, kInf = 0x7f800000u;  // 2^-96, infinity
  if (min(min(b0, b1), min(b2, b3)) >= kLow && max(max(b0, b1), max(b2, b3)) < kInf) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = __builtin_amdgcn_rsqf(v[e]);
      const float g = v[e] * y;
      r[e] = __builtin_fmaf(__builtin_fmaf(-g, g, v[e]), 0.5f * y, g);
      float t = r[e] * k.inv_sbc2;
      t = __builtin_fmaf(__builtin_fmaf(-t, k.sbc2, r[e]), k.inv_sbc2, t);
      q[e] = __builtin_fmaf(__builtin_fmaf(-t, k.sbc2, r[e]), k.inv_sbc2, t);
    }
  } else {  // zeros, NaN, infinities and roots below 2^-48
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = sqrtf(v[e]);
      q[e] = r[e] / k.sbc2;
    }
  }
}

// adamw_elem's operations on four elements; r returns sqrt(v) of the new v.
template <int WM>
__device__ __forceinline__ void step4(const f32x4 a, f32x4& p, f32x4& m, f32x4& v, f32x4& r, const StepScalars& k) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float g = WM == kNoDiv ? divide(a[e], k.wdiv) : divide_m<WM>(a[e], k.wdiv);
    const float gh = g * k.coef;
    m[e] = k.b1 * m[e] + k.omb1 * gh;
    v[e] = k.b2 * v[e] + k.omb2 * (gh * gh);
  }
  f32x4 q;
  roots4(v, k, r, q);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float d = q[e] + k.eps;
    p[e] = p[e] * k.decay - k.step_size * (m[e] / d);
  }
}

// The gradient as an FP32 accumulator, with the load policy it was stored for.
template <bool NT>
struct AccIn {
  typedef f32x4 raw_t;
  static __device__ __forceinline__ raw_t load(const void* base, int64_t e) {
    return ld4f_acc<NT>(static_cast<const float*>(base) + e);
  }
  static __device__ __forceinline__ f32x4 widen(const raw_t r) { return r; }
  static __device__ __forceinline__ float load1(const void* base, int64_t i) {
    return static_cast<const float*>(base)[i];
  }
};

// A chunk's arrays, each at the chunk's first element.
struct StepChunk {
  const void* g;      // gradient (the type is a template parameter)
  float* p;
  void* m;            // FP32, or one code byte per element
  void* v;
  float* m_scale;     // one per block of kCodedBlock elements (8-bit moments)
  float* v_scale;
  uint16_t* pb;       // BF16 copy, may be null
  int len;
};

__device__ __forceinline__ uint32_t ld1u_nt(const void* p, int64_t byte) {
  return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + byte));
}
__device__ __forceinline__ void st1u_nt(void* p, int64_t byte, uint32_t x) {
  __builtin_nontemporal_store(x, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + byte));
}

// Up to four elements from element e on, the first n of them in the array and
// the others 0; `wide`: one vector access is allowed when all four are there.
template <typename In>
__device__ __forceinline__ f32x4 load_part(const void* a, int64_t e, int n, bool wide) {
  if (wide && n == 4) return In::widen(In::load(a, e));
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) x[i] = In::load1(a, e + i);
  return x;
}
__device__ __forceinline__ void store_part(float* a, int64_t e, int n, bool wide, const f32x4 x) {
  if (wide && n == 4) {
    st4f_nt(a + e, x);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) a[e + i] = x[i];
}
__device__ __forceinline__ uint32_t load_codes(const void* a, int64_t e, int n, bool wide) {
  if (wide && n == 4) return ld1u_nt(a, e);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) c |= uint32_t(static_cast<const uint8_t*>(a)[e + i]) << (8 * i);
  return c;
}
__device__ __forceinline__ void store_codes(void* a, int64_t e, int n, bool wide, uint32_t c) {
  if (wide && n == 4) {
    st1u_nt(a, e, c);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) static_cast<uint8_t*>(a)[e + i] = uint8_t(c >> (8 * i));
}
__device__ __forceinline__ void store_copy(uint16_t* a, int64_t e, int n, bool wide, const f32x4 p) {
  if (wide && n == 4) {
    store_bf16x4(a + e, p);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) a[e + i] = bf16_bits(p[i]);
}

// A chunk of any length whose arrays are only element-aligned, one element at a
// time.  Every lane makes every trip, because a block's maximum needs its
// whole row of lanes; elements past the end enter as zeros and are not stored.
template <typename In, bool CODED>
__device__ void step_any(const StepChunk& c, const StepScalars& k) {
  const int trips = (c.len + 4 * kBlock - 1) / (4 * kBlock);
  for (int t = 0; t < trips; ++t) {
    const int e = 4 * (t * kBlock + int(threadIdx.x));
    const int n = min(max(c.len - e, 0), 4);
    const int b = e / kCodedBlock;
    f32x4 g = load_part<In>(c.g, e, n, false);
    f32x4 p = load_part<F32In>(c.p, e, n, false);
    f32x4 m, v;
    if (CODED) {
      m = decode_m4(load_codes(c.m, e, n, false), n > 0 ? c.m_scale[b] : 0.0f);
      v = decode_v4(load_codes(c.v, e, n, false), n > 0 ? c.v_scale[b] : 0.0f);
    } else {
      m = load_part<F32In>(c.m, e, n, false);
      v = load_part<F32In>(c.v, e, n, false);
    }
    f32x4 r;
    step4<kNoDiv>(g, p, m, v, r, k);
    store_part(c.p, e, n, false, p);
    if (c.pb) store_copy(c.pb, e, n, false, p);
    if (CODED) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i >= n) m[i] = r[i] = 0.0f;
      const Coded4 cm = encode_m4(m);
      const Coded4 cv = encode_root4(r);
      store_codes(c.m, e, n, false, cm.codes);
      store_codes(c.v, e, n, false, cv.codes);
      if ((threadIdx.x & 15) == 0 && n > 0) {
        c.m_scale[b] = cm.scale;
        c.v_scale[b] = cv.scale;
      }
    } else {
      store_part(static_cast<float*>(c.m), e, n, false, m);
      store_part(static_cast<float*>(c.v), e, n, false, v);
    }
  }
}

// U vectors per lane of arrays that take four-element accesses: a stretch of
// U * kPartElems elements, of which `len` are there.  FULL: all of them, and the
// window division (WM) and the BF16 copy (COPY) are fixed at compile time: no
// bounds checks.  Every load is issued before one is used.  Same operations as
// step_any.
constexpr int kPartElems = 4 * kBlock;  // one vector per lane
constexpr int kVecsPerLane = kChunkElems / kPartElems;  // 4 with 4096-element chunks and 256 lanes
static_assert(kVecsPerLane >= 1 && kChunkElems == kVecsPerLane * kPartElems, "a chunk is whole vectors per lane");
static_assert(kPartElems % kCodedBlock == 0, "whole blocks per part of a chunk");
enum CopyMode { kNoCopy = 0, kCopy = 1, kMaybeCopy = 2 };

template <typename In, bool CODED, int U, bool FULL, int WM, int COPY>
__device__ __forceinline__ void step_wide(const StepChunk& c, const StepScalars& k) {
  f32x4 g[U], p[U], m[U], v[U];
  typename In::raw_t raw[U];
  uint32_t mc[U], vc[U];
  float ms[U], vs[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!FULL && u > 0 && u * kPartElems >= c.len) break;
    const int e = 4 * (int(threadIdx.x) + u * kBlock);
    const int n = FULL ? 4 : min(max(c.len - e, 0), 4);
    if (FULL) {
      raw[u] = In::load(c.g, e);
      p[u] = ld4f_nt(c.p + e);
    } else {
      g[u] = load_part<In>(c.g, e, n, true);
      p[u] = load_part<F32In>(c.p, e, n, true);
    }
    if (CODED) {
      mc[u] = FULL ? ld1u_nt(c.m, e) : load_codes(c.m, e, n, true);
      vc[u] = FULL ? ld1u_nt(c.v, e) : load_codes(c.v, e, n, true);
      ms[u] = n > 0 ? c.m_scale[e / kCodedBlock] : 0.0f;
      vs[u] = n > 0 ? c.v_scale[e / kCodedBlock] : 0.0f;
    } else if (FULL) {
      m[u] = ld4f_nt(static_cast<const float*>(c.m) + e);
      v[u] = ld4f_nt(static_cast<const float*>(c.v) + e);
    } else {
      m[u] = load_part<F32In>(c.m, e, n, true);
      v[u] = load_part<F32In>(c.v, e, n, true);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!FULL && u > 0 && u * kPartElems >= c.len) break;
    const int e = 4 * (int(threadIdx.x) + u * kBlock);
    const int n = FULL ? 4 : min(max(c.len - e, 0), 4);
    if (FULL) g[u] = In::widen(raw[u]);
    if (CODED) {
      m[u] = decode_m4(mc[u], ms[u]);
      v[u] = decode_v4(vc[u], vs[u]);
    }
    f32x4 r;
    step4<WM>(g[u], p[u], m[u], v[u], r, k);
    store_part(c.p, e, n, true, p[u]);
    if (COPY == kCopy || (COPY == kMaybeCopy && c.pb)) store_copy(c.pb, e, n, true, p[u]);
    if (CODED) {
      if (!FULL) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i >= n) m[u][i] = r[i] = 0.0f;
      }
      const Coded4 cm = encode_m4(m[u]);
      const Coded4 cv = encode_root4(r);
      store_codes(c.m, e, n, true, cm.codes);
      store_codes(c.v, e, n, true, cv.codes);
      if ((threadIdx.x & 15) == 0 && n > 0) {
        c.m_scale[e / kCodedBlock] = cm.scale;
        c.v_scale[e / kCodedBlock] = cv.scale;
      }
    } else {
      store_part(static_cast<float*>(c.m), e, n, true, m[u]);
      store_part(static_cast<float*>(c.v), e, n, true, v[u]);
    }
  }
}

// A chunk by one workgroup: all of it in one sweep of kVecsPerLane vectors per
// lane.  SPLIT: one vector per lane of it, for few chunks (see kSplitChunks).
template <typename In, bool CODED, bool SPLIT>
__device__ __forceinline__ void step_chunk(const StepChunk& c, const StepScalars& k, bool wide) {
  if (!wide) {
    step_any<In, CODED>(c, k);
  } else if (SPLIT) {
    step_wide<In, CODED, 1, false, kNoDiv, kMaybeCopy>(c, k);
  } else if (c.len != kChunkElems) {
    step_wide<In, CODED, kVecsPerLane, false, kNoDiv, kMaybeCopy>(c, k);
  } else if (div_mode(k.wdiv) == kMulInv) {
    if (c.pb) step_wide<In, CODED, kVecsPerLane, true, kMulInv, kCopy>(c, k);
    else step_wide<In, CODED, kVecsPerLane, true, kMulInv, kNoCopy>(c, k);
  } else {
    if (c.pb) step_wide<In, CODED, kVecsPerLane, true, kIeeeDiv, kCopy>(c, k);
    else step_wide<In, CODED, kVecsPerLane, true, kIeeeDiv, kNoCopy>(c, k);
  }
}

// Up to this many chunks a step takes kVecsPerLane (four) workgroups per chunk,
// one vector per lane each, instead of one with four: few workgroups leave most
// of the 256 CUs idle, and a lane's four vectors are four times the arithmetic
// in a row.
// Group steps of n full chunks, split against whole, us: n = 16, 32-bit
// moments 3.9 / 5.3, 8-bit 5.5 / 6.4; n = 64 5.5 / 5.9 and 5.9 / 6.7; n = 128
// 6.6 / 6.3 and 6.8 / 7.0; n = 256 8.0 / 7.7 and 8.3 / 7.7; n = 4096 78 / 78 and
// 70 / 52.
#ifndef GRO_SPLIT_CHUNKS
#define GRO_SPLIT_CHUNKS 128
#endif
constexpr int64_t kSplitChunks = GRO_SPLIT_CHUNKS;

// The part of a chunk that workgroup `part` of its kVecsPerLane takes.
template <typename In, bool CODED>
__device__ __forceinline__ void take_part(StepChunk& c, int part) {
  const int e = part * kPartElems;
  constexpr int moment = CODED ? 1 : int(sizeof(float));
  c.g = static_cast<const char*>(c.g) + e * int(sizeof(typename In::raw_t) / 4);
  c.p += e;
  c.m = static_cast<char*>(c.m) + e * moment;
  c.v = static_cast<char*>(c.v) + e * moment;
  if (CODED) {
    c.m_scale += e / kCodedBlock;
    c.v_scale += e / kCodedBlock;
  }
  if (c.pb) c.pb += e;
  c.len = min(max(c.len - e, 0), kPartElems);
}

}  // namespace
}  // namespace gro
