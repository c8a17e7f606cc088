// Groups of tensors that stay where they lie: host tables (group_abi.hip) and
// kernels (group.hip).  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "kernels.h"
#include "plan.h"

namespace gro {

// Gradient pointers that travel in one norm launch's kernel arguments.
constexpr int kGroupPointers = 448;

struct GroupTensorDev {    // 64 B
  float* p;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  uint16_t* pb;
  int64_t decayed;
  int64_t wide;            // every array above takes four-element accesses
};
static_assert(sizeof(GroupTensorDev) == 64, "group tensor entry is 64 bytes");

struct GroupNormLaunch {
  const ChunkDev* chunks;  // begin: first element within the tensor; bucket: the tensor
  int64_t q_begin, q_end;
  const void** table;      // gradient pointer of every tensor, left for the step
  double* partials;
  int32_t t_first;         // tensor of grads[0]
  int32_t fp32;            // gradients of the range are FP32
  int32_t window;
  int32_t reserved;
  const void* grads[kGroupPointers];
};

struct GroupStepLaunch {
  const ChunkDev* chunks;
  int64_t q_begin, q_end;
  const GroupTensorDev* tensors;
  const void* const* table;
  const double* scalars;
  AdamWConsts k;
};

hipError_t launch_group_norm(const GroupNormLaunch& a, hipStream_t s);
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
  int64_t kind_chunk[5] = {0, 0, 0, 0, 0};  // first chunk of each kind, and the end
  int32_t kind_entry[5] = {0, 0, 0, 0, 0};
  std::vector<gro::ChunkDev> chunks;
  uint64_t scalar_off = 0, tensor_off = 0, table_off = 0, chunk_off = 0, partial_off = 0, group_off = 0,
           counter_off = 0, counter_bytes = 0, total = 0;

  char* d_ws = nullptr;
  bool bound = false;
  int device = -1;
  bool norm_done = false;   // gradients and norm of a step are on the device
  bool norm_valid = false;  // some norm has been computed since binding
  int32_t window = 0;
  void* norm_stream = nullptr;
};
