// Host helpers shared by the entry points that launch kernels: argument
// checks and the AdamW step's scalars.  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "plan.h"

namespace gro {

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

inline int hip_fail(hipError_t e, const char* what) {
  return set_error(GRO_E_HIP, "%s: %s", what, hipGetErrorString(e));
}

// The checks of a clip + AdamW call that no state depends on.
inline int check_step_args(const gro_adamw_hparams* hp, int64_t step, double max_norm) {
  if (hp == nullptr) return set_error(GRO_E_INVALID, "hp is NULL");
  if (step < 1) return set_error(GRO_E_INVALID, "step must be >= 1");
  if (std::isnan(max_norm)) return set_error(GRO_E_INVALID, "max_norm is NaN");
  if (!(hp->lr >= 0.0) || !std::isfinite(hp->lr) || !(hp->eps >= 0.0) || !std::isfinite(hp->eps) ||
      !(hp->weight_decay >= 0.0) || !std::isfinite(hp->weight_decay) || !(hp->beta1 >= 0.0) ||
      !(hp->beta1 < 1.0) || !(hp->beta2 >= 0.0) || !(hp->beta2 < 1.0))
    return set_error(GRO_E_INVALID, "hyper-parameters out of range (lr, eps, wd >= 0; 0 <= beta < 1)");
  return GRO_OK;
}

// Per-step scalars in FP64 from the hyper-parameters as given, each rounded
// once to FP32.
inline AdamWConsts adamw_consts(const gro_adamw_hparams& hp, int64_t step, double max_norm, int32_t window) {
  const double bc1 = 1.0 - std::pow(hp.beta1, double(step));
  const double bc2 = 1.0 - std::pow(hp.beta2, double(step));
  AdamWConsts k;
  k.max_norm = max_norm;
  k.clip_on = (max_norm > 0.0 && !std::isinf(max_norm)) ? 1 : 0;
  k.window = window;
  k.beta1 = float(hp.beta1);
  k.beta2 = float(hp.beta2);
  k.one_minus_beta1 = float(1.0 - hp.beta1);
  k.one_minus_beta2 = float(1.0 - hp.beta2);
  k.step_size = float(hp.lr / bc1);
  k.sqrt_bc2 = float(std::sqrt(bc2));
  k.inv_sqrt_bc2 = 1.0f / k.sqrt_bc2;
  k.eps = float(hp.eps);
  k.decay = float(1.0 - hp.lr * hp.weight_decay);
  return k;
}

// A device array that a call writes (or must not find written).
struct Range {
  uintptr_t at;
  uint64_t bytes;
  bool operator<(const Range& o) const { return at < o.at; }
};

// Sorts the n ranges by address and returns the index of the first that
// begins before the one in front of it ends, or -1.  Empty ranges count for
// nothing.
inline int64_t first_overlap(Range* r, size_t n) {
  if (n < 2) return -1;
  Range* end = std::remove_if(r, r + n, [](const Range& x) { return x.bytes == 0; });
  std::sort(r, end);
  for (Range* x = r + 1; x < end; ++x)
    if (x->at - (x - 1)->at < (x - 1)->bytes) return x - r;
  return -1;
}

}  // namespace gro
