// gb_optim_api.cpp — the C ABI of the optimizer step (include/gbreduce.h):
// argument validation, the plan's layout, kernel launch.  Nothing is enqueued
// unless every argument is valid; no call allocates device memory.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

#include "gb_internal.h"
#include "gb_optim.h"
#include "gb_overlap.h"

namespace {

constexpr uint64_t kMagic = 0x67626f7074696d31ull;
constexpr size_t kWorkspaceAlign = 256;

gb_status fail(gb_status s, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return gb::fail_status(s, msg);
}

gb_status from_hip(hipError_t e, const char* what) {
  if (e == hipSuccess) return GB_OK;
  return fail(GB_ERR_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
size_t nblocks(size_t n) { return (n + GB_BLOCK - 1) / GB_BLOCK; }
size_t nchunks(size_t n) { return (n + gb::kOptimChunk - 1) / gb::kOptimChunk; }
size_t elem_size(int dtype) { return dtype == GB_DTYPE_F32 ? 4 : 2; }

// Byte offsets in a plan's workspace: tensors, chunks, partial sums.
struct Layout {
  size_t chunks, partials, total;
};
Layout layout(size_t count, size_t chunks) {
  Layout l;
  l.chunks = round_up(count * sizeof(gb::OptimTensor), kWorkspaceAlign);
  l.partials = l.chunks + round_up(chunks * sizeof(gb::OptimChunk), kWorkspaceAlign);
  l.total = l.partials + gb::kNormGroups * sizeof(double);
  return l;
}

// Sums of the plan's sizes; false when they exceed GB_MAX_N (the chunk and
// block numbers of the tables then still fit 32 bits).
bool add_size(size_t n, size_t* values, size_t* chunks) {
  if (n > GB_MAX_N) return false;
  *values += round_up(n, GB_BLOCK);
  *chunks += nchunks(n);
  return *values <= GB_MAX_N;
}

bool known_plan(const gb_optim_handle* plan, gb::OptimPlan* out) {
  if (plan == nullptr) return false;
  std::memcpy(out, plan, sizeof *out);
  return out->magic == kMagic;
}

gb_status check_pointer(const void* p, size_t align, const char* fn, int i, const char* name) {
  if (p == nullptr) return fail(GB_ERR_INVALID_ARG, "%s: tensors[%d].%s is NULL", fn, i, name);
  if (!aligned(p, align)) {
    return fail(GB_ERR_MISALIGNED, "%s: tensors[%d].%s = %p is not %zu-byte aligned", fn, i, name, p, align);
  }
  return GB_OK;
}

gb_status check_tensor(const gb_optim_tensor& t, const char* fn, int i) {
  if (t.dtype != GB_DTYPE_F32 && t.dtype != GB_DTYPE_F16 && t.dtype != GB_DTYPE_BF16) {
    return fail(GB_ERR_UNSUPPORTED, "%s: tensors[%d].dtype %d is not float32, float16 or bfloat16", fn, i, t.dtype);
  }
  if (t.state != GB_STATE_F32 && t.state != GB_STATE_E4M3) {
    return fail(GB_ERR_UNSUPPORTED, "%s: tensors[%d].state %d is unknown", fn, i, t.state);
  }
  if (!std::isfinite(t.lr_scale) || !std::isfinite(t.weight_decay)) {
    return fail(GB_ERR_INVALID_ARG, "%s: tensors[%d]: lr_scale %g or weight_decay %g is not finite", fn, i,
                (double)t.lr_scale, (double)t.weight_decay);
  }
  gb_status s;
  if ((s = check_pointer(t.param, 4, fn, i, "param")) != GB_OK) return s;
  if ((s = check_pointer(t.grad, elem_size(t.dtype), fn, i, "grad")) != GB_OK) return s;
  if ((s = check_pointer(t.m, GB_ALIGN, fn, i, "m")) != GB_OK) return s;
  if ((s = check_pointer(t.v, GB_ALIGN, fn, i, "v")) != GB_OK) return s;
  if (t.state == GB_STATE_E4M3) {
    if ((s = check_pointer(t.m_scale, 4, fn, i, "m_scale")) != GB_OK) return s;
    if ((s = check_pointer(t.v_scale, 4, fn, i, "v_scale")) != GB_OK) return s;
  } else if (t.m_scale != nullptr || t.v_scale != nullptr) {
    return fail(GB_ERR_INVALID_ARG, "%s: tensors[%d] has scales, but float32 moments", fn, i);
  }
  if (t.copy != nullptr) {
    if (t.copy_dtype != GB_DTYPE_F16 && t.copy_dtype != GB_DTYPE_BF16) {
      return fail(GB_ERR_UNSUPPORTED, "%s: tensors[%d].copy_dtype %d is not float16 or bfloat16", fn, i, t.copy_dtype);
    }
    if ((s = check_pointer(t.copy, elem_size(t.copy_dtype), fn, i, "copy")) != GB_OK) return s;
  }
  return GB_OK;
}

void add_spans(const gb_optim_tensor& t, long i, gb::Spans* outs, gb::Spans* ins) {
  const bool coded = t.state == GB_STATE_E4M3;
  const size_t moment = coded ? t.n : 4 * t.n, scales = 4 * nblocks(t.n);
  outs->add(t.param, 4 * t.n, "param", i);
  outs->add(t.copy, elem_size(t.copy_dtype) * t.n, "copy", i);
  outs->add(t.m, moment, "m", i);
  outs->add(t.v, moment, "v", i);
  if (coded) {
    outs->add(t.m_scale, scales, "m_scale", i);
    outs->add(t.v_scale, scales, "v_scale", i);
  }
  ins->add(t.grad, elem_size(t.dtype) * t.n, "grad", i);
}

gb_status make_plan(const char* fn, gb_optim_handle* handle, const gb_optim_tensor* tensors, int count, double beta1,
                    double beta2, double eps, uint64_t seed, void* workspace, size_t workspace_bytes,
                    hipStream_t stream) {
  if (handle == nullptr) return fail(GB_ERR_INVALID_ARG, "%s: plan is NULL", fn);
  if (count < 0 || count > GB_OPTIM_MAX_TENSORS) {
    return fail(GB_ERR_INVALID_ARG, "%s: count = %d is outside 0..%d", fn, count, GB_OPTIM_MAX_TENSORS);
  }
  if (count > 0 && tensors == nullptr) return fail(GB_ERR_INVALID_ARG, "%s: tensors is NULL", fn);
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) {
    return fail(GB_ERR_INVALID_ARG, "%s: beta1 = %g or beta2 = %g is outside [0, 1)", fn, beta1, beta2);
  }
  if (!((float)eps > 0.0f) || !std::isfinite((float)eps)) {
    return fail(GB_ERR_INVALID_ARG, "%s: eps = %g is not above 0 in binary32", fn, eps);
  }
  size_t values = 0, chunks = 0;
  for (int i = 0; i < count; i++) {
    if (!add_size(tensors[i].n, &values, &chunks)) {
      return fail(GB_ERR_INVALID_ARG, "%s: the tensors up to tensors[%d] exceed GB_MAX_N = %zu values", fn, i,
                  GB_MAX_N);
    }
  }
  const Layout l = layout((size_t)count, chunks);
  if (workspace == nullptr || workspace_bytes < l.total) {
    return fail(GB_ERR_WORKSPACE, "%s: workspace %p of %zu bytes, %zu needed", fn, workspace, workspace_bytes,
                l.total);
  }
  if (!aligned(workspace, kWorkspaceAlign)) {
    return fail(GB_ERR_MISALIGNED, "%s: workspace = %p is not %zu-byte aligned", fn, workspace, kWorkspaceAlign);
  }
  gb::Spans outs, ins;
  outs.add(workspace, l.total, "workspace");
  for (int i = 0; i < count; i++) {
    if (tensors[i].n == 0) continue;
    gb_status s = check_tensor(tensors[i], fn, i);
    if (s != GB_OK) return s;
    add_spans(tensors[i], i, &outs, &ins);
  }
  gb_status s = gb::check_disjoint(fn, outs, ins);
  if (s != GB_OK) return s;

  char* ws = static_cast<char*>(workspace);
  gb::OptimTensor* table = reinterpret_cast<gb::OptimTensor*>(ws);
  gb::OptimChunk* map = reinterpret_cast<gb::OptimChunk*>(ws + l.chunks);
  gb::OptimPlan plan = {};
  plan.magic = kMagic;
  plan.tensors = table;
  plan.chunks = map;
  plan.partials = reinterpret_cast<double*>(ws + l.partials);
  plan.beta1 = beta1;
  plan.beta2 = beta2;
  plan.seed = seed;
  plan.eps = (float)eps;
  for (int i = 0; i < count; i++) {
    if (tensors[i].n == 0) continue;
    plan.grad_bytes += elem_size(tensors[i].dtype) * tensors[i].n;
    plan.first[gb::optim_kind(tensors[i].dtype, tensors[i].state) + 1] += (uint32_t)nchunks(tensors[i].n);
  }
  for (int k = 0; k < gb::kOptimKinds; k++) plan.first[k + 1] += plan.first[k];

  uint32_t next[gb::kOptimKinds];
  std::memcpy(next, plan.first, sizeof next);
  size_t block = 0;
  hipError_t e = hipSuccess;
  gb::OptimUpload up = {};
  auto flush = [&]() {
    if (e == hipSuccess) e = gb::launch_optim_upload(table, map, up, stream);
    up.first_tensor += up.count;
    up.count = 0;
  };
  for (int i = 0; i < count; i++) {
    const gb_optim_tensor& t = tensors[i];
    gb::OptimTensor d = {};
    if (t.n != 0) {
      d = {t.n, t.param, t.grad, t.copy, t.m, t.v, t.m_scale, t.v_scale, (uint32_t)block,
           (uint32_t)t.dtype | (t.copy != nullptr ? (uint32_t)t.copy_dtype << 16 : 0u), t.lr_scale, t.weight_decay};
      uint32_t& at = next[gb::optim_kind(t.dtype, t.state)];
      up.first_chunk[up.count] = at;
      at += (uint32_t)nchunks(t.n);
      block += nblocks(t.n);
    }
    up.t[up.count++] = d;
    if (up.count == gb::kOptimUpload) flush();
  }
  if (up.count > 0) flush();
  if (e != hipSuccess) return from_hip(e, fn);
  std::memset(handle, 0, sizeof *handle);
  std::memcpy(handle, &plan, sizeof plan);
  return GB_OK;
}

gb_status check_step(const char* fn, const gb_optim_handle* handle, const void* control, gb::OptimPlan* plan) {
  if (!known_plan(handle, plan)) return fail(GB_ERR_INVALID_ARG, "%s: plan was not made by gb_optim_plan", fn);
  if (control == nullptr) return fail(GB_ERR_INVALID_ARG, "%s: control is NULL", fn);
  if (!aligned(control, GB_ALIGN)) {
    return fail(GB_ERR_MISALIGNED, "%s: control = %p is not %d-byte aligned", fn, control, GB_ALIGN);
  }
  // the kernels follow the addresses in the workspace's tables (a handle of zeros but the mark has none)
  gb::Span c, w;
  c.lo = reinterpret_cast<uintptr_t>(control);
  c.hi = c.lo + GB_OPTIM_CONTROL_BYTES;
  c.name = "control";
  w.lo = reinterpret_cast<uintptr_t>(plan->tensors);
  w.hi = reinterpret_cast<uintptr_t>(plan->partials + gb::kNormGroups);
  w.name = "workspace";
  if (w.lo != 0 && c.lo < w.hi && w.lo < c.hi) return gb::overlap_error(fn, c, w);
  return GB_OK;
}

gb_status check_scale(const char* fn, double inv_scale) {
  if (!(inv_scale > 0.0) || !std::isfinite(inv_scale) || !((float)inv_scale > 0.0f) ||
      !std::isfinite((float)inv_scale)) {
    return fail(GB_ERR_INVALID_ARG, "%s: inv_scale = %g is not finite and above 0 in binary32", fn, inv_scale);
  }
  return GB_OK;
}

}  // namespace

extern "C" {

size_t gb_optim_plan_bytes(const size_t* ns, int count) {
  if (count < 0 || count > GB_OPTIM_MAX_TENSORS || (count > 0 && ns == nullptr)) return 0;
  size_t values = 0, chunks = 0;
  for (int i = 0; i < count; i++) {
    if (!add_size(ns[i], &values, &chunks)) return 0;
  }
  return layout((size_t)count, chunks).total;
}

gb_status gb_optim_plan(gb_optim_handle* plan, const gb_optim_tensor* tensors, int count, double beta1, double beta2,
                        double eps, uint64_t seed, void* workspace, size_t workspace_bytes, void* stream) {
  return gb::traced_call("gb_optim_plan", stream, -1, count < 0 ? 0 : (size_t)count, -1,
                         [&](const char* fn) -> gb_status {
    try {
      return make_plan(fn, plan, tensors, count, beta1, beta2, eps, seed, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
    } catch (const std::bad_alloc&) {  // the overlap check's lists: nothing was enqueued
      return fail(GB_ERR_INVALID_ARG, "%s: no host memory to check %d tensors", fn, count);
    }
  });
}

gb_status gb_optim_begin(const gb_optim_handle* plan, void* control, double inv_scale, void* stream) {
  return gb::traced_call("gb_optim_begin", stream, -1, gb::kNoSize, -1, [&](const char* fn) -> gb_status {
    gb::OptimPlan p;
    gb_status s = check_step(fn, plan, control, &p);
    if (s == GB_OK) s = check_scale(fn, inv_scale);
    if (s != GB_OK) return s;
    return from_hip(gb::launch_optim_begin(p, static_cast<gb_optim_control*>(control), inv_scale,
                                           static_cast<hipStream_t>(stream)),
                    fn);
  });
}

gb_status gb_optim_begin_clip(const gb_optim_handle* plan, void* control, double max_norm, double inv_scale,
                              void* stream) {
  return gb::traced_call("gb_optim_begin_clip", stream, -1, gb::kNoSize, -1, [&](const char* fn) -> gb_status {
    gb::OptimPlan p;
    gb_status s = check_step(fn, plan, control, &p);
    if (s == GB_OK) s = check_scale(fn, inv_scale);
    if (s != GB_OK) return s;
    if (!(max_norm > 0.0)) return fail(GB_ERR_INVALID_ARG, "%s: max_norm = %g is not above 0", fn, max_norm);
    return from_hip(gb::launch_optim_begin_clip(p, static_cast<gb_optim_control*>(control), max_norm, inv_scale,
                                                static_cast<hipStream_t>(stream)),
                    fn);
  });
}

gb_status gb_adamw_step(const gb_optim_handle* plan, const void* control, void* stream) {
  return gb::traced_call("gb_adamw_step", stream, -1, gb::kNoSize, -1, [&](const char* fn) -> gb_status {
    gb::OptimPlan p;
    gb_status s = check_step(fn, plan, control, &p);
    if (s != GB_OK) return s;
    return from_hip(gb::launch_adamw(p, static_cast<const gb_optim_control*>(control),
                                     static_cast<hipStream_t>(stream)),
                    fn);
  });
}

}  // extern "C"
