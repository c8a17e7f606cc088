// C-ABI entry points of groups: tensors that stay where they lie.  As for
// plans, every check happens on the host before the first launch, so a call
// that is refused has enqueued nothing.
#include <hip/hip_runtime.h>

#include <cstring>
#include <exception>
#include <vector>

#include "group.h"
#include "host.h"

using namespace gro;

namespace {

// Whether the norm's second stage is left to the step's workgroups.
bool folded(const gro_group* g) { return g->n_chunks <= kFoldChunks; }

// A kind's number, 0..3: gradient type and moment type.
int kind_of(uint32_t flags) { return ((flags & GRO_FP32_GRAD) ? 2 : 0) + ((flags & GRO_CODED_MOMENTS) ? 1 : 0); }

int check_group(const gro_group* g) {
  if (g == nullptr) return set_error(GRO_E_INVALID, "group is NULL");
  if (!g->bound) return set_error(GRO_E_STATE, "group is not bound to a workspace");
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev != g->device)
    return set_error(GRO_E_STATE, "group is bound on device %d, current device is %d", g->device, dev);
  return GRO_OK;
}

double* dev_scalars(const gro_group* g) { return reinterpret_cast<double*>(g->d_ws + g->scalar_off); }
const GroupChunkDev* dev_chunks(const gro_group* g) {
  return reinterpret_cast<const GroupChunkDev*>(g->d_ws + g->chunk_off);
}
const void** dev_grads(const gro_group* g) { return reinterpret_cast<const void**>(g->d_ws + g->grad_off); }
double* dev_partials(const gro_group* g) { return reinterpret_cast<double*>(g->d_ws + g->partial_off); }

hipError_t launch_final(const gro_group* g, hipStream_t s) {
  NormFinalLaunch f;
  f.partials = dev_partials(g);
  f.n_chunks = g->n_chunks;
  f.group_sums = reinterpret_cast<double*>(g->d_ws + g->group_off);
  f.counter = reinterpret_cast<uint32_t*>(g->d_ws + g->counter_off);
  f.scalars = dev_scalars(g);
  return launch_norm_final(f, s);
}

// The norm's first stage, N tensors' gradient pointers to a launch.
template <int N>
hipError_t launch_norms(const gro_group* g, const GroupNormArgs& args, const void* const* d_grads, hipStream_t s) {
  const int32_t n = int32_t(g->entries.size());
  hipError_t e = hipSuccess;
  for (int32_t t = 0; t < n && e == hipSuccess; t += N) {
    const int32_t te = std::min(n, t + N);
    GroupNormLaunch<N> l = {};
    l.a = args;
    l.a.q_begin = g->entries[size_t(t)].first_chunk;
    l.a.q_end = te < n ? g->entries[size_t(te)].first_chunk : g->n_chunks;
    l.a.t_first = t;
    for (int32_t i = t; i < te; ++i) l.grads[i - t] = d_grads[g->entries[size_t(i)].given];
    e = launch_group_norm(l, s);
  }
  return e;
}

int64_t chunks_of(int64_t numel) { return (numel + kChunkElems - 1) / kChunkElems; }

int fill_group(gro_group* g, const gro_group_desc* tensors, int32_t n) {
  g->n_tensors = n;
  for (int32_t i = 0; i < n; ++i) {
    const gro_group_desc& d = tensors[i];
    if (d.numel < 0 || d.numel > kMaxNumel)
      return set_error(GRO_E_INVALID, "tensor %d: %lld elements", i, (long long)d.numel);
    if ((d.flags & ~(GRO_NO_DECAY | GRO_FP32_GRAD | GRO_CODED_MOMENTS)) || d.reserved != 0)
      return set_error(GRO_E_PLACEMENT, "tensor %d: unknown flags 0x%x or nonzero reserved field", i, d.flags);
    g->n_chunks += chunks_of(d.numel);
    // one workgroup of kBlock lanes per chunk, fewer than 2^32 lanes a launch
    if (g->n_chunks >= (int64_t(1) << 24) - 1)
      return set_error(GRO_E_INVALID, "group too large: more chunks than one launch grid addresses");
    g->n_elems += d.numel;
  }
  int64_t q = 0;
  for (int kind = 0; kind < 4; ++kind) {
    g->kind_chunk[kind] = q;
    for (int32_t i = 0; i < n; ++i) {
      const gro_group_desc& d = tensors[i];
      if (d.numel == 0 || kind_of(d.flags) != kind) continue;
      g->entries.push_back(gro_group::Entry{i, d.flags, d.numel, q});
      q += chunks_of(d.numel);
    }
  }
  g->kind_chunk[4] = q;

  uint64_t off = 0;
  const auto place = [&off](uint64_t bytes) {
    const uint64_t at = off;
    off = uint64_t(align_up(int64_t(off + bytes), 256));
    return at;
  };
  const uint64_t chunks = uint64_t(g->n_chunks);
  g->scalar_off = place(256);
  g->chunk_off = place(chunks * sizeof(GroupChunkDev));
  g->grad_off = place(chunks * sizeof(void*));
  g->partial_off = place(chunks * sizeof(double));
  g->group_off = place(uint64_t(norm_groups(g->n_chunks)) * sizeof(double));
  g->counter_bytes = 256;
  g->counter_off = place(g->counter_bytes);
  g->total = off;
  return GRO_OK;
}

// The device chunk table from the caller's pointers, for a workspace at ws.
int fill_chunks(const gro_group* g, const gro_group_tensor* tensors, const char* ws, std::vector<GroupChunkDev>& out) {
  std::vector<Range> written;
  written.reserve(g->entries.size() * 6 + 1);
  written.push_back(Range{reinterpret_cast<uintptr_t>(ws), g->total});
  int32_t index = 0;
  for (const gro_group::Entry& e : g->entries) {
    const gro_group_tensor& t = tensors[e.given];
    const bool coded = (e.flags & GRO_CODED_MOMENTS) != 0;
    const uintptr_t moment = coded ? 1 : sizeof(float);
    if (t.master == nullptr || t.m == nullptr || t.v == nullptr || !aligned_to(t.master, 4) ||
        !aligned_to(t.m, moment) || !aligned_to(t.v, moment) || !aligned_to(t.param_bf16, 2))
      return set_error(GRO_E_INVALID, "tensor %d: master, m or v is NULL, or an array is not aligned to its elements",
                       e.given);
    if (coded && (t.m_scale == nullptr || t.v_scale == nullptr || !aligned_to(t.m_scale, 4) || !aligned_to(t.v_scale, 4)))
      return set_error(GRO_E_INVALID, "tensor %d: scales of 8-bit moments are NULL or not 4-byte aligned", e.given);
    const uint64_t n = uint64_t(e.numel);
    const uint64_t scales = coded ? (n + kCodedBlock - 1) / kCodedBlock * sizeof(float) : 0;
    const auto add = [&written](const void* a, uint64_t bytes) {
      if (a != nullptr) written.push_back(Range{reinterpret_cast<uintptr_t>(a), bytes});
    };
    add(t.master, n * 4);
    add(t.m, n * moment);
    add(t.v, n * moment);
    add(t.param_bf16, n * 2);
    add(t.m_scale, scales);
    add(t.v_scale, scales);
    const bool wide = aligned_to(t.master, 16) && aligned_to(t.m, 4 * moment) && aligned_to(t.v, 4 * moment) &&
                      aligned_to(t.param_bf16, 8);
    for (int64_t begin = 0; begin < e.numel; begin += kChunkElems) {
      GroupChunkDev c;
      c.p = t.master + begin;
      c.m = static_cast<char*>(t.m) + begin * int64_t(moment);
      c.v = static_cast<char*>(t.v) + begin * int64_t(moment);
      c.m_scale = coded ? t.m_scale + begin / kCodedBlock : nullptr;
      c.v_scale = coded ? t.v_scale + begin / kCodedBlock : nullptr;
      c.pb = t.param_bf16 ? t.param_bf16 + begin : nullptr;
      c.begin = begin;
      c.tensor = index;
      c.len = uint16_t(std::min<int64_t>(e.numel - begin, kChunkElems));
      c.flags = uint16_t(((e.flags & GRO_NO_DECAY) ? 0 : kChunkDecayed) |
                         ((e.flags & GRO_FP32_GRAD) ? kChunkFp32 : 0) | (wide ? kChunkWide : 0));
      out.push_back(c);
    }
    ++index;
  }
  if (first_overlap(written.data(), written.size()) >= 0)
    return set_error(GRO_E_DUPLICATE, "two of the group's arrays, or one and the workspace, overlap");
  return GRO_OK;
}

int bind_group(gro_group* g, const gro_group_tensor* tensors, char* ws, hipStream_t s) {
  std::vector<GroupChunkDev> chunks;
  chunks.reserve(size_t(g->n_chunks));
  const int rc = fill_chunks(g, tensors, ws, chunks);
  if (rc != GRO_OK) return rc;
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  // The norm's completion counter must start at zero; every kernel that
  // counts returns it there.
  g->bound = false;
  e = hipMemsetAsync(ws + g->counter_off, 0, g->counter_bytes, s);
  if (e == hipSuccess && !chunks.empty())
    e = hipMemcpyAsync(ws + g->chunk_off, chunks.data(), chunks.size() * sizeof(GroupChunkDev), hipMemcpyHostToDevice, s);
  const hipError_t done = hipStreamSynchronize(s);
  if (e == hipSuccess) e = done;
  if (e != hipSuccess) return hip_fail(e, "gro_group_bind upload");
  g->d_ws = ws;
  g->bound = true;
  g->device = dev;
  g->norm_done = false;
  g->norm_valid = false;
  return GRO_OK;
}

}  // namespace

extern "C" int gro_group_create(const gro_group_desc* tensors, int32_t n_tensors, gro_group** out) {
  clear_error();
  if (out == nullptr) return set_error(GRO_E_INVALID, "out is NULL");
  *out = nullptr;
  if (n_tensors < 0) return set_error(GRO_E_INVALID, "n_tensors < 0");
  if (n_tensors > 0 && tensors == nullptr) return set_error(GRO_E_INVALID, "tensors is NULL");
  gro_group* g = nullptr;
  try {
    g = new gro_group();
    const int rc = fill_group(g, tensors, n_tensors);
    if (rc == GRO_OK) *out = g;
    else delete g;
    return rc;
  } catch (const std::exception&) {
    delete g;
    return set_error(GRO_E_INVALID, "out of host memory");
  }
}

extern "C" void gro_group_destroy(gro_group* group) { delete group; }

extern "C" int gro_group_get_info(const gro_group* g, gro_group_info* info) {
  clear_error();
  if (g == nullptr || info == nullptr) return set_error(GRO_E_INVALID, "NULL argument");
  std::memset(info, 0, sizeof(*info));
  info->n_tensors = g->n_tensors;
  info->chunk_elems = kChunkElems;
  info->n_chunks = g->n_chunks;
  info->n_elems = g->n_elems;
  info->workspace_bytes = g->total;
  return GRO_OK;
}

extern "C" int gro_group_bind(gro_group* g, const gro_group_tensor* tensors, void* d_workspace, uint64_t bytes,
                              void* stream) {
  clear_error();
  if (g == nullptr || d_workspace == nullptr || (tensors == nullptr && g->n_tensors > 0))
    return set_error(GRO_E_INVALID, "NULL argument");
  if (!aligned_to(d_workspace, 256)) return set_error(GRO_E_INVALID, "workspace must be 256-byte aligned");
  if (bytes < g->total)
    return set_error(GRO_E_INVALID, "workspace has %llu bytes, group needs %llu", (unsigned long long)bytes,
                     (unsigned long long)g->total);
  try {
    return bind_group(g, tensors, static_cast<char*>(d_workspace), static_cast<hipStream_t>(stream));
  } catch (const std::exception&) {
    return set_error(GRO_E_INVALID, "out of host memory");
  }
}

extern "C" int gro_group_norm(gro_group* g, const void* const* d_grads, int32_t window_size, void* stream) {
  clear_error();
  const int rc = check_group(g);
  if (rc != GRO_OK) return rc;
  if (window_size < 1) return set_error(GRO_E_INVALID, "window_size must be >= 1");
  if (d_grads == nullptr && g->n_tensors > 0) return set_error(GRO_E_INVALID, "d_grads is NULL");
  for (const gro_group::Entry& e : g->entries)
    if (!aligned_to(d_grads[e.given], (e.flags & GRO_FP32_GRAD) ? 4 : 2))
      return set_error(GRO_E_INVALID, "gradient of tensor %d is not aligned to its elements", e.given);

  hipStream_t s = static_cast<hipStream_t>(stream);
  // From here on the pointers and partials of an earlier call are being
  // replaced: a launch that fails midway leaves no norm at all.
  g->norm_done = false;
  g->norm_valid = false;
  GroupNormArgs a;
  a.chunks = dev_chunks(g);
  a.chunk_grads = dev_grads(g);
  a.partials = dev_partials(g);
  a.window = window_size;
  const int32_t n = int32_t(g->entries.size());
  hipError_t e = hipSuccess;
  if (n <= kGroupPointersShort) e = launch_norms<kGroupPointersShort>(g, a, d_grads, s);
  else e = launch_norms<kGroupPointers>(g, a, d_grads, s);
  if (e != hipSuccess) return hip_fail(e, "group norm launch");
  if (!folded(g)) {
    e = launch_final(g, s);
    if (e != hipSuccess) return hip_fail(e, "group norm stage-2 launch");
  }
  g->norm_done = true;
  g->norm_valid = true;
  g->window = window_size;
  g->norm_stream = stream;
  return GRO_OK;
}

extern "C" int gro_group_clip_adamw(gro_group* g, double max_norm, const gro_adamw_hparams* hp, int64_t step,
                                    void* stream) {
  clear_error();
  int rc = check_group(g);
  if (rc != GRO_OK) return rc;
  rc = check_step_args(hp, step, max_norm);
  if (rc != GRO_OK) return rc;
  if (!g->norm_done) return set_error(GRO_E_STATE, "gro_group_norm of this step has not run");
  GroupStepLaunch a;
  a.chunks = dev_chunks(g);
  a.chunk_grads = dev_grads(g);
  a.scalars = dev_scalars(g);
  a.partials = dev_partials(g);
  a.n_partials = folded(g) ? int32_t(g->n_chunks) : 0;
  a.k = adamw_consts(*hp, step, max_norm, g->window);
  g->norm_done = false;  // one update for one norm, also when a launch fails after others have updated their kind
  for (int kind = 0; kind < 4; ++kind) {
    a.q_begin = g->kind_chunk[kind];
    a.q_end = g->kind_chunk[kind + 1];
    const hipError_t e = launch_group_step(a, (kind & 2) != 0, (kind & 1) != 0, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "group clip+AdamW launch");
  }
  return GRO_OK;
}

extern "C" int gro_group_get_norm(gro_group* g, double* norm, double* norm_sq, int32_t* finite) {
  clear_error();
  const int rc = check_group(g);
  if (rc != GRO_OK) return rc;
  if (!g->norm_valid) return set_error(GRO_E_STATE, "no gro_group_norm since the group was bound");
  double host[kNumScalars];
  hipStream_t s = static_cast<hipStream_t>(g->norm_stream);
  hipError_t e = folded(g) ? launch_final(g, s) : hipSuccess;
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e == hipSuccess) e = hipMemcpy(host, dev_scalars(g), sizeof(host), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return hip_fail(e, "reading the norm");
  if (norm) *norm = host[kNorm];
  if (norm_sq) *norm_sq = host[kNormSq];
  if (finite) *finite = host[kFinite] != 0.0 ? 1 : 0;
  return GRO_OK;
}
