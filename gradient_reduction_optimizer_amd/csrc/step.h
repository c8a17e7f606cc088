// One chunk's clip + AdamW with the moments in 32 bits or in 8-bit codes,
// device side.  A lane owns 4-element vectors lane, lane + kBlock, ... of its
// chunk, as in every pass, so with 8-bit moments a block of 64 elements is
// one row of 16 lanes (see coded.h).
#pragma once

#include "coded.h"
#include "kernels.h"

namespace gro {
namespace {

// The step's scalars with the clip coefficient of the norm on the device.
__device__ __forceinline__ AdamScalars step_scalars(const AdamWConsts& c, const double* scalars, bool decayed) {
  AdamScalars k;
  k.wdiv = make_divisor(c.window);
  k.coef = 1.0f;
  if (c.clip_on) {
    const double r = c.max_norm / (scalars[kNorm] + 1e-6);
    k.coef = float(r < 1.0 ? r : 1.0);
  }
  k.decay = decayed ? c.decay : 1.0f;
  k.b1 = c.beta1;
  k.b2 = c.beta2;
  k.omb1 = c.one_minus_beta1;
  k.omb2 = c.one_minus_beta2;
  k.step_size = c.step_size;
  k.sbc2 = c.sqrt_bc2;
  k.eps = c.eps;
  return k;
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

__device__ __forceinline__ f32x4 sqrt4(const f32x4 v) {
  return f32x4{sqrtf(v.x), sqrtf(v.y), sqrtf(v.z), sqrtf(v.w)};
}

// Any chunk: any length, any element-aligned arrays (`wide`: all of them may
// be accessed four elements at a time).  Every lane makes every trip, because
// a block's maximum needs its whole row of lanes; elements past the end enter
// as zeros and are not stored.
template <typename In, bool CODED>
__device__ void step_any(const StepChunk& c, const AdamScalars& k, bool wide) {
  const int trips = (c.len + 4 * kBlock - 1) / (4 * kBlock);
  for (int t = 0; t < trips; ++t) {
    const int e = 4 * (t * kBlock + int(threadIdx.x));
    const int n = min(max(c.len - e, 0), 4);
    const int b = e / kCodedBlock;
    f32x4 g = load_part<In>(c.g, e, n, wide);
    f32x4 p = load_part<F32In>(c.p, e, n, wide);
    f32x4 m, v;
    if (CODED) {
      m = decode_m4(load_codes(c.m, e, n, wide), n > 0 ? c.m_scale[b] : 0.0f);
      v = decode_v4(load_codes(c.v, e, n, wide), n > 0 ? c.v_scale[b] : 0.0f);
    } else {
      m = load_part<F32In>(c.m, e, n, wide);
      v = load_part<F32In>(c.v, e, n, wide);
    }
    adamw4<kNoDiv>(g, p, m, v, k);
    store_part(c.p, e, n, wide, p);
    if (c.pb) store_copy(c.pb, e, n, wide, p);
    if (CODED) {
      const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i >= n) m[i] = v[i] = none[i];
      const Coded4 cm = encode_m4(m);
      const Coded4 cv = encode_root4(sqrt4(v));
      store_codes(c.m, e, n, wide, cm.codes);
      store_codes(c.v, e, n, wide, cv.codes);
      if ((threadIdx.x & 15) == 0 && n > 0) {
        c.m_scale[b] = cm.scale;
        c.v_scale[b] = cv.scale;
      }
    } else {
      store_part(static_cast<float*>(c.m), e, n, wide, m);
      store_part(static_cast<float*>(c.v), e, n, wide, v);
    }
  }
}

// A full chunk of arrays that take four-element accesses, the window division
// (WM) and the BF16 copy fixed at compile time: kStepUnroll vectors of every
// array are loaded before any is used, no bounds checks.  Same operations as
// step_any.
#ifndef GRO_STEP_UNROLL
#define GRO_STEP_UNROLL 4
#endif
constexpr int kStepUnroll = GRO_STEP_UNROLL;
static_assert((kChunkElems / 4) % (kStepUnroll * kBlock) == 0, "whole sweeps per chunk");

template <typename In, bool CODED, int WM, bool COPY>
__device__ __forceinline__ void step_full(const StepChunk& c, const AdamScalars& k) {
#pragma unroll 1
  for (int v0 = threadIdx.x; v0 < kChunkElems / 4; v0 += kStepUnroll * kBlock) {
    typename In::raw_t g[kStepUnroll];
    f32x4 p[kStepUnroll], m[kStepUnroll], v[kStepUnroll];
    uint32_t mc[kStepUnroll], vc[kStepUnroll];
    float ms[kStepUnroll], vs[kStepUnroll];
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) {
      const int e = 4 * (v0 + u * kBlock);
      g[u] = In::load(c.g, e);
      p[u] = ld4f_nt(c.p + e);
      if (CODED) {
        mc[u] = ld1u_nt(c.m, e);
        vc[u] = ld1u_nt(c.v, e);
        ms[u] = c.m_scale[e / kCodedBlock];
        vs[u] = c.v_scale[e / kCodedBlock];
      } else {
        m[u] = ld4f_nt(static_cast<const float*>(c.m) + e);
        v[u] = ld4f_nt(static_cast<const float*>(c.v) + e);
      }
    }
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) {
      const int e = 4 * (v0 + u * kBlock);
      if (CODED) {
        m[u] = decode_m4(mc[u], ms[u]);
        v[u] = decode_v4(vc[u], vs[u]);
      }
      adamw4<WM>(In::widen(g[u]), p[u], m[u], v[u], k);
      st4f_nt(c.p + e, p[u]);
      if (COPY) store_bf16x4(c.pb + e, p[u]);
      if (CODED) {
        const Coded4 cm = encode_m4(m[u]);
        const Coded4 cv = encode_root4(sqrt4(v[u]));
        st1u_nt(c.m, e, cm.codes);
        st1u_nt(c.v, e, cv.codes);
        if ((threadIdx.x & 15) == 0) {
          c.m_scale[e / kCodedBlock] = cm.scale;
          c.v_scale[e / kCodedBlock] = cv.scale;
        }
      } else {
        st4f_nt(static_cast<float*>(c.m) + e, m[u]);
        st4f_nt(static_cast<float*>(c.v) + e, v[u]);
      }
    }
  }
}

template <typename In, bool CODED>
__device__ __forceinline__ void step_chunk(const StepChunk& c, const AdamScalars& k, bool wide) {
  if (!wide || c.len != kChunkElems) {
    step_any<In, CODED>(c, k, wide);
  } else if (div_mode(k.wdiv) == kMulInv) {
    if (c.pb) step_full<In, CODED, kMulInv, true>(c, k);
    else step_full<In, CODED, kMulInv, false>(c, k);
  } else {
    if (c.pb) step_full<In, CODED, kIeeeDiv, true>(c, k);
    else step_full<In, CODED, kIeeeDiv, false>(c, k);
  }
}

}  // namespace
}  // namespace gro
