// Groups of tensors that stay where they lie: host tables (group_abi.hip) and
// kernels (group.hip).  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "kernels.h"
#include "plan.h"

namespace gro {

// Gradient pointers that travel in one launch's kernel arguments (under 4 KB).
constexpr int kGroupPointers = 448;

// A chunk of one tensor with everything a kernel needs of it, so that one load
// leads to the arrays.  Pointers are those of the chunk's first element.
struct GroupChunkDev {     // 64 B
  float* p;
  void* m;
  void* v;
  float* m_scale;          // null for FP32 moments
  float* v_scale;
  uint16_t* pb;            // may be null
  int64_t begin;           // first element within the tensor
  int32_t tensor;
  uint16_t len;            // 1..kChunkElems
  uint16_t flags;
};
static_assert(sizeof(GroupChunkDev) == 64 && kChunkElems <= 65535, "group chunk entry is 64 bytes");
enum GroupChunkFlag : uint16_t {
  kChunkDecayed = 1,
  kChunkFp32 = 2,          // FP32 gradient
  kChunkWide = 4,          // the arrays above take four-element accesses
};

struct GroupNormArgs {
  const GroupChunkDev* chunks;
  int64_t q_begin, q_end;
  const void** chunk_grads;   // out: every chunk's gradient, for the step
  double* partials;
  int32_t window;
  int32_t t_first;            // tensor of grads[0]
};
template <int N>
struct GroupNormLaunch {
  GroupNormArgs a;
  const void* grads[N];
};
// Most groups' pointers fit the short form, whose launch copies 512 bytes
// instead of 3.6 KB.
constexpr int kGroupPointersShort = 64;

struct GroupStepLaunch {
  const GroupChunkDev* chunks;
  int64_t q_begin, q_end;
  const void* const* chunk_grads;
  const double* scalars;
  const double* partials;  // n_partials > 0: the norm's partials, added up by
  int32_t n_partials;      // every workgroup itself (see kFoldChunks)
  AdamWConsts k;
};

// In a group of up to this many chunks the step's workgroups add the norm's
// partials up themselves, in the order of the second stage (so to the same
// bits), and no second stage is launched.  Norm and step of n chunks with 8-bit
// moments, folded against three launches, us: n = 256 10.0 / 13.2, n = 512 13.5 /
// 16.3, n = 1024 20.9 / 23.3, n = 2048 34.5 / 36.3; 32-bit moments the same
// differences.  Beyond kNormGroup chunks the second stage has another level.
constexpr int64_t kFoldChunks = kNormGroup;

template <int N>
hipError_t launch_group_norm(const GroupNormLaunch<N>& a, hipStream_t s);
// The chunks of [q_begin, q_end) all have gradients of one type and moments
// of one kind.
hipError_t launch_group_step(const GroupStepLaunch& a, bool fp32, bool coded, hipStream_t s);

}  // namespace gro

struct gro_group {
  int32_t n_tensors = 0;
  int64_t n_elems = 0;
  // Tensors with elements, sorted by kind (gradient type, moment type) and
  // given order within a kind.
  struct Entry {
    int32_t given;         // index as given
    uint32_t flags;
    int64_t numel;
    int64_t first_chunk;
  };
  std::vector<Entry> entries;
  int64_t n_chunks = 0;
  int64_t kind_chunk[5] = {0, 0, 0, 0, 0};  // first chunk of each kind, and the end
  uint64_t scalar_off = 0, chunk_off = 0, grad_off = 0, partial_off = 0, group_off = 0,
           counter_off = 0, counter_bytes = 0, total = 0;

  char* d_ws = nullptr;
  bool bound = false;
  int device = -1;
  bool norm_done = false;   // gradients and norm (or its partials) of a step are on the device
  bool norm_valid = false;  // some norm has been computed since binding
  int32_t window = 0;
  void* norm_stream = nullptr;
};
