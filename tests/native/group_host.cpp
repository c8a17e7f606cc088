// The group entry points' host side (csrc/group_abi.hip) compiled by a plain
// C++ compiler, with stand-ins for the HIP runtime and for the launches that
// can be made to fail.  No device, no kernel: every pointer is made up.
#include "group_abi.hip"

#include <cstdio>
#include <cstdlib>
#include <string>

static int g_norms, g_finals, g_steps;  // launches asked for
static int g_fail_norm = -1, g_fail_final = -1, g_fail_step = -1;  // that one fails

static hipError_t note(int* n, int fail) { return (*n)++ == fail ? hipErrorLaunchFailure : hipSuccess; }
namespace gro {
template <int N>
hipError_t launch_group_norm(const GroupNormLaunch<N>&, hipStream_t) { return note(&g_norms, g_fail_norm); }
template hipError_t launch_group_norm(const GroupNormLaunch<kGroupPointersShort>&, hipStream_t);
template hipError_t launch_group_norm(const GroupNormLaunch<kGroupPointers>&, hipStream_t);
hipError_t launch_norm_final(const NormFinalLaunch&, hipStream_t) { return note(&g_finals, g_fail_final); }
hipError_t launch_group_step(const GroupStepLaunch&, bool, bool, hipStream_t) { return note(&g_steps, g_fail_step); }
int set_error(int code, const char*, ...) { return code; }
void clear_error() {}
}  // namespace gro

extern "C" {
const char* hipGetErrorString(hipError_t) { return ""; }
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipMemsetAsync(void*, int, size_t, hipStream_t) { return hipSuccess; }
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipMemcpy(void* dst, const void*, size_t n, hipMemcpyKind) { std::memset(dst, 0, n); return hipSuccess; }
}

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

struct Group {
  gro_group* g = nullptr;
  std::vector<const void*> grads;
  std::vector<gro_group_tensor> rows;
  uint64_t bytes = 0;

  explicit Group(const std::vector<gro_group_desc>& d) {
    CHECK(gro_group_create(d.data(), int32_t(d.size()), &g) == GRO_OK);
    gro_group_info info;
    CHECK(gro_group_get_info(g, &info) == GRO_OK);
    bytes = info.workspace_bytes;
    uintptr_t at = 1 << 30;
    const auto next = [&at](int64_t n) { const uintptr_t p = at; at += uintptr_t((n + 255) / 256 * 256); return p; };
    for (const gro_group_desc& x : d) {
      gro_group_tensor t = {};
      t.master = reinterpret_cast<float*>(next(4 * x.numel));
      t.m = reinterpret_cast<void*>(next(4 * x.numel));
      t.v = reinterpret_cast<void*>(next(4 * x.numel));
      t.m_scale = reinterpret_cast<float*>(next(4 * x.numel));
      t.v_scale = reinterpret_cast<float*>(next(4 * x.numel));
      rows.push_back(t);
      grads.push_back(reinterpret_cast<void*>(next(4 * x.numel)));
    }
    CHECK(bind(1 << 20) == GRO_OK);
    g_norms = g_finals = g_steps = 0;
    g_fail_norm = g_fail_final = g_fail_step = -1;
  }
  ~Group() { gro_group_destroy(g); }
  int bind(uintptr_t ws) { return gro_group_bind(g, rows.data(), reinterpret_cast<void*>(ws), bytes, nullptr); }
  int norm() { return gro_group_norm(g, grads.data(), 1, nullptr); }
  int step() {
    const gro_adamw_hparams hp = {1e-3, 0.9, 0.999, 1e-8, 0.0};
    return gro_group_clip_adamw(g, 1.0, &hp, 1, nullptr);
  }
  int get() { return gro_group_get_norm(g, nullptr, nullptr, nullptr); }
};

// A launch error after other kinds of tensors have been updated: asked again,
// the step must not update those twice.
static void step_launch_fails() {
  const std::vector<gro_group_desc> kinds = {{100, 0, 0}, {100, GRO_CODED_MOMENTS, 0}, {100, GRO_FP32_GRAD, 0},
                                             {100, GRO_CODED_MOMENTS | GRO_FP32_GRAD, 0}};
  for (int k = 0; k < 4; ++k) {
    Group x(kinds);
    CHECK(x.norm() == GRO_OK);
    g_fail_step = k;
    CHECK(x.step() == GRO_E_HIP && g_steps == k + 1);
    CHECK(x.step() == GRO_E_STATE && g_steps == k + 1);
    CHECK(x.norm() == GRO_OK && x.step() == GRO_OK && g_steps == k + 5);
  }
}

// A launch error between the launches of a norm: what the workspace holds is
// neither this norm nor the last one.
static void norm_launch_fails() {
  const std::vector<gro_group_desc> many(1000, {50, 0, 0});
  const std::vector<gro_group_desc> large = {{int64_t(kChunkElems) * (kFoldChunks + 1), 0, 0}};
  for (int k = 0; k < 3; ++k) {
    Group x(many);
    CHECK(x.norm() == GRO_OK && x.get() == GRO_OK && g_norms == 3);
    g_fail_norm = 3 + k;
    CHECK(x.norm() == GRO_E_HIP);
    CHECK(x.get() == GRO_E_STATE && x.step() == GRO_E_STATE && g_steps == 0);
    CHECK(x.norm() == GRO_OK && x.get() == GRO_OK && x.step() == GRO_OK);
  }
  Group x(large);
  CHECK(x.norm() == GRO_OK && x.get() == GRO_OK && g_finals == 1);
  g_fail_final = 1;
  CHECK(x.norm() == GRO_E_HIP && x.get() == GRO_E_STATE && x.step() == GRO_E_STATE);
}

int main(int argc, char** argv) {
  const std::string which = argc > 1 ? argv[1] : "";
  if (which == "step") step_launch_fails();
  else if (which == "norm") norm_launch_fails();
  else return 2;
  std::printf("ok\n");
  return 0;
}
