// optim_driver.cpp — the optimizer's C-ABI layer (gb_optim_api.cpp) under
// AddressSanitizer and UndefinedBehaviorSanitizer on the host: plans over
// random tensors, whose tables the stand-in launcher writes into a workspace
// of exactly gb_optim_plan_bytes, then read back and checked; refusals; and a
// launch failure injected at every upload.  Test infrastructure: nothing here
// runs in the library.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

#include "../../gradient_all_reduce_amd/csrc/gb_internal.h"
#include "../../gradient_all_reduce_amd/csrc/gb_optim.h"

extern "C" const char* hipGetErrorString(hipError_t) { return "injected"; }

namespace {

long g_uploads = 0, g_fail_at = 0, g_failed = 0;
char g_message[512];

void expect(bool ok, const char* what) {
  if (ok) return;
  g_failed++;
  std::printf("FAILED: %s (last error: %s)\n", what, g_message);
}

}  // namespace

namespace gb {

gb_status fail_status(gb_status s, const char* msg) {
  std::snprintf(g_message, sizeof g_message, "%s", msg);
  return s;
}
bool call_hooks_on() { return false; }
gb_status finish_call(const char*, void*, int, size_t, int, gb_status s, double) { return s; }

// What the upload kernel writes, on the host.
hipError_t launch_optim_upload(OptimTensor* tensors, OptimChunk* chunks, const OptimUpload& up, hipStream_t) {
  if (++g_uploads == g_fail_at) return hipErrorLaunchFailure;
  if (up.count < 1 || up.count > (uint32_t)kOptimUpload) std::abort();
  for (uint32_t i = 0; i < up.count; i++) {
    tensors[up.first_tensor + i] = up.t[i];
    const uint32_t count = (uint32_t)((up.t[i].n + kOptimChunk - 1) / kOptimChunk);
    for (uint32_t c = 0; c < count; c++) chunks[up.first_chunk[i] + c] = OptimChunk{up.first_tensor + i, c};
  }
  return hipSuccess;
}
OptimPlan g_seen;
hipError_t launch_optim_begin(const OptimPlan& plan, gb_optim_control*, double, hipStream_t) {
  g_seen = plan;
  return hipSuccess;
}
hipError_t launch_optim_begin_clip(const OptimPlan& plan, gb_optim_control*, double, double, hipStream_t) {
  g_seen = plan;
  return hipSuccess;
}
hipError_t launch_adamw(const OptimPlan& plan, const gb_optim_control*, hipStream_t) {
  g_seen = plan;
  return hipSuccess;
}

}  // namespace gb

namespace {

// Made-up device addresses, disjoint; nothing reads them.
uintptr_t g_next = 0x100000000ull;
void* address(size_t bytes, size_t off = 0) {
  g_next = (g_next + 255) / 256 * 256;
  void* p = reinterpret_cast<void*>(g_next + off);
  g_next += bytes + off + 64;
  return p;
}

gb_optim_tensor tensor(size_t n, int dtype, int state, bool copy) {
  gb_optim_tensor t = {};
  const size_t e = dtype == GB_DTYPE_F32 ? 4 : 2, blocks = (n + 255) / 256;
  t.n = n;
  t.dtype = dtype;
  t.state = state;
  t.lr_scale = 1.0f;
  if (n == 0) return t;
  t.param = static_cast<float*>(address(4 * n, 4));
  t.grad = address(e * n, e);
  t.copy_dtype = dtype == GB_DTYPE_F32 ? GB_DTYPE_BF16 : dtype;
  if (copy) t.copy = address(2 * n, 2);
  t.m = address(4 * n);
  t.v = address(4 * n);
  if (state == GB_STATE_E4M3) {
    t.m_scale = static_cast<float*>(address(4 * blocks, 4));
    t.v_scale = static_cast<float*>(address(4 * blocks, 4));
  }
  return t;
}

void check_plan(const std::vector<gb_optim_tensor>& ts, void* control) {
  std::vector<size_t> ns;
  for (const auto& t : ts) ns.push_back(t.n);
  const size_t bytes = gb_optim_plan_bytes(ns.data(), (int)ns.size());
  expect(bytes > 0, "plan bytes");
  void* ws = std::aligned_alloc(256, (bytes + 255) / 256 * 256);
  gb_optim_handle h;
  expect(gb_optim_plan(&h, ts.data(), (int)ts.size(), 0.9, 0.999, 1e-8, 7, ws, bytes, nullptr) == GB_OK, "plan");
  expect(gb_optim_begin(&h, control, 1.0, nullptr) == GB_OK, "begin");
  expect(gb_optim_begin_clip(&h, control, INFINITY, 0.5, nullptr) == GB_OK, "begin_clip");
  expect(gb_adamw_step(&h, control, nullptr) == GB_OK, "step");
  const gb::OptimPlan& p = gb::g_seen;
  // every chunk of every tensor once, in the range of its kind
  std::vector<std::vector<char>> seen;
  size_t block = 0, grad = 0;
  for (size_t i = 0; i < ts.size(); i++) {
    seen.emplace_back((ts[i].n + gb::kOptimChunk - 1) / gb::kOptimChunk);
    grad += ts[i].n * (ts[i].dtype == GB_DTYPE_F32 ? 4 : 2);
    if (ts[i].n == 0) continue;
    const gb::OptimTensor& d = p.tensors[i];
    expect(d.n == ts[i].n && d.p == ts[i].param && d.g == ts[i].grad && d.copy == ts[i].copy && d.m == ts[i].m &&
               d.v == ts[i].v && d.ms == ts[i].m_scale && d.vs == ts[i].v_scale && d.first_block == block,
           "a tensor's entry");
    block += (ts[i].n + 255) / 256;
  }
  expect(p.grad_bytes == grad, "bytes of gradients");
  for (int k = 0; k < gb::kOptimKinds; k++) {
    for (uint32_t c = p.first[k]; c < p.first[k + 1]; c++) {
      const gb::OptimChunk e = p.chunks[c];
      if (e.tensor >= ts.size() || e.chunk >= seen[e.tensor].size() || seen[e.tensor][e.chunk]++ ||
          gb::optim_kind(ts[e.tensor].dtype, ts[e.tensor].state) != k) {
        expect(false, "a chunk's entry");
        k = gb::kOptimKinds;
        break;
      }
    }
  }
  for (const auto& s : seen) {
    for (char c : s) expect(c == 1, "a chunk is missing");
  }
  for (uint32_t b = 0; b < gb::kNormGroups; b++) p.partials[b] = 1.0;  // the last bytes of the workspace
  std::free(ws);
}

}  // namespace

int main() {
  void* control = address(64);
  check_plan({}, control);
  check_plan({tensor(0, 0, 0, false)}, control);
  unsigned rng = 12345;
  auto next = [&](unsigned m) {
    rng = rng * 1664525u + 1013904223u;
    return (rng >> 8) % m;
  };
  for (int round = 0; round < 40; round++) {
    std::vector<gb_optim_tensor> ts;
    const int count = (int)next(round < 20 ? 8 : 300);
    for (int i = 0; i < count; i++) {
      const size_t n = next(5) == 0 ? 0 : next(4) == 0 ? next(100000) : next(3000);
      ts.push_back(tensor(n, (int)next(3), (int)next(2), next(2) == 0));
    }
    check_plan(ts, control);
  }

  // a failure at each upload of a plan of 100 tensors
  std::vector<gb_optim_tensor> ts;
  std::vector<size_t> ns(100, 700);
  for (int i = 0; i < 100; i++) ts.push_back(tensor(700, i % 3, i % 2, false));
  const size_t bytes = gb_optim_plan_bytes(ns.data(), 100);
  void* ws = std::aligned_alloc(256, (bytes + 255) / 256 * 256);
  for (long at = 1; at <= 3; at++) {
    g_uploads = 0;
    g_fail_at = at;
    gb_optim_handle h;
    std::memset(&h, 0, sizeof h);
    expect(gb_optim_plan(&h, ts.data(), 100, 0.9, 0.999, 1e-8, 7, ws, bytes, nullptr) == GB_ERR_HIP, "failed upload");
    expect(g_uploads == at, "nothing is launched after a failure");
    expect(gb_adamw_step(&h, control, nullptr) == GB_ERR_INVALID_ARG, "a failed plan is no plan");
  }
  g_fail_at = 0;
  gb_optim_handle h;
  g_uploads = 0;
  // refusals launch nothing
  expect(gb_optim_plan(&h, ts.data(), 100, 0.9, 0.999, 1e-8, 7, ws, bytes - 1, nullptr) == GB_ERR_WORKSPACE, "short");
  std::vector<gb_optim_tensor> twice = {ts[0], ts[1], ts[0]};
  expect(gb_optim_plan(&h, twice.data(), 3, 0.9, 0.999, 1e-8, 7, ws, bytes, nullptr) == GB_ERR_INVALID_ARG, "twice");
  size_t huge[3] = {GB_MAX_N, 1, ~(size_t)0};
  expect(gb_optim_plan_bytes(huge, 1) > 0 && gb_optim_plan_bytes(huge, 2) == 0 && gb_optim_plan_bytes(huge + 2, 1) == 0,
         "sizes beyond GB_MAX_N");
  gb_optim_tensor over = ts[0];
  over.n = ~(size_t)0;
  expect(gb_optim_plan(&h, &over, 1, 0.9, 0.999, 1e-8, 7, ws, bytes, nullptr) == GB_ERR_INVALID_ARG, "n wraps");
  expect(g_uploads == 0, "a refusal launched something");
  std::free(ws);
  std::printf("%ld failed\n", g_failed);
  return g_failed != 0;
}
