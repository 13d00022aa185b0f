// layers_driver.cpp — the token-sum layers' C-ABI layer (gb_layers_api.cpp)
// under AddressSanitizer and UndefinedBehaviorSanitizer on the host: random
// calls, whose stand-in launchers write every part of a workspace of exactly
// the size the library asks for and every row of the outputs, all in buffers
// of their exact extent; refusals; and a launch that fails.  Test
// infrastructure: nothing here runs in the library.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <random>

#include "../../gradient_all_reduce_amd/csrc/gb_internal.h"
#include "../../gradient_all_reduce_amd/csrc/gb_layers.h"

extern "C" const char* hipGetErrorString(hipError_t) { return "injected"; }

namespace {

long g_launches = 0, g_failed = 0, g_fail = 0;
char g_message[512];

void expect(bool ok, const char* what) {
  if (ok) return;
  g_failed++;
  std::printf("FAILED: %s (last error: %s)\n", what, g_message);
}
size_t size_of(int dtype) { return dtype == GB_DTYPE_I64 ? 8 : dtype == GB_DTYPE_F32 || dtype == GB_DTYPE_I32 ? 4 : 2; }
void write_rows(const gb::Rows& r, size_t rows, size_t cols, size_t size) {
  if (r.p == nullptr) return;
  for (size_t i = 0; i < rows; i++) std::memset((char*)r.p + i * r.stride * size, 1, cols * size);
}
int read_bytes(const void* p, size_t n) {
  int s = 0;
  for (size_t i = 0; i < n; i++) s += ((const char*)p)[i];
  return s;
}
volatile int g_sink;

}  // namespace

namespace gb {

gb_status fail_status(gb_status s, const char* msg) {
  std::snprintf(g_message, sizeof g_message, "%s", msg);
  return s;
}
bool call_hooks_on() { return false; }
gb_status finish_call(const char*, void*, int, size_t, int, gb_status s, double) { return s; }

uint32_t norm_grad_groups(size_t rows, size_t, int dtype) {
  const size_t g = (rows + dtype) / (1 + dtype);
  return (uint32_t)(g < 200 ? g : 200);
}
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t) {
  g_launches++;
  write_rows(a.y, a.rows, a.cols, size_of(a.dtype));
  for (size_t r = 0; r < a.rows; r++) {
    g_sink = read_bytes((char*)a.x.p + r * a.x.stride * size_of(a.dtype), a.cols * size_of(a.dtype));
    if (a.mean != nullptr) a.mean[r] = 0;
    if (a.rstd != nullptr) a.rstd[r] = 0;
  }
  return g_fail ? hipErrorLaunchFailure : hipSuccess;
}
hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t) {
  g_launches++;
  const size_t e = size_of(a.dtype);
  for (size_t r = 0; r < a.rows; r++) {
    g_sink = read_bytes((char*)a.dy.p + r * a.dy.stride * e, a.cols * e);
    g_sink = read_bytes(&a.mean[r], 4) + read_bytes(&a.rstd[r], 4);
  }
  write_rows(a.dx, a.rows, a.cols, e);
  if (a.dw != nullptr || a.db != nullptr) {
    const size_t groups = norm_grad_groups(a.rows, a.cols, a.dtype);
    for (size_t i = 0; i < groups * 2 * a.partial_stride; i++) a.partials[i] = 0;
    if (a.dw != nullptr) std::memset(a.dw, 0, a.cols * size_of(a.grad_dtype));
    if (a.db != nullptr) std::memset(a.db, 0, a.cols * size_of(a.grad_dtype));
  }
  return g_fail ? hipErrorLaunchFailure : hipSuccess;
}
hipError_t launch_embedding(const LookArgs& a, hipStream_t) {
  g_launches++;
  write_rows(a.out, a.tokens, a.dim, size_of(a.out_dtype));
  g_sink = read_bytes(a.ids, a.tokens * size_of(a.id_dtype));
  return g_fail ? hipErrorLaunchFailure : hipSuccess;
}
hipError_t launch_embedding_grad(const LookGradArgs& a, hipStream_t) {
  g_launches++;
  write_rows(a.dtable, a.vocab, a.dim, size_of(a.grad_dtype));
  if (a.tokens == 0) return hipSuccess;
  const LookGradLayout l = look_grad_layout(a.tokens, a.vocab, a.dim);
  // every part, each with a mark of its own that no other part may touch
  struct Part {
    size_t at, bytes;
  };
  const bool digits = a.tokens > kSortSmall;
  const Part parts[] = {{l.count, 8},
                        {l.keys[0], 4 * a.tokens},
                        {l.tokens[0], 4 * a.tokens},
                        {l.keys[1], digits ? 4 * a.tokens : 0},
                        {l.tokens[1], digits ? 4 * a.tokens : 0},
                        {l.hist, digits ? ((size_t)sort_blocks(a.tokens) * 4 << kSortDigitBits) : 0},
                        {l.named, (a.vocab + 15) / 16 * 16},
                        {l.long_runs, kLongRunBytes * (a.tokens / (kFold + 1))},
                        {l.partials, a.tokens > kFold ? 8 * look_windows(a.tokens) * look_partial_stride(a.dim) : 0}};
  int mark = 1;
  for (const Part& p : parts) std::memset(a.workspace + p.at, mark++, p.bytes);
  mark = 1;
  for (const Part& p : parts) {
    bool whole = p.at % 16 == 0;
    for (size_t i = 0; i < p.bytes; i++) whole = whole && a.workspace[p.at + i] == mark;
    expect(whole, "a part of the workspace is its own");
    mark++;
  }
  return g_fail ? hipErrorLaunchFailure : hipSuccess;
}

}  // namespace gb

namespace {

std::mt19937 g_rng(7);
size_t pick(size_t lo, size_t hi) { return std::uniform_int_distribution<size_t>(lo, hi)(g_rng); }
// `bytes` bytes at the very end of an allocation
struct Exact {
  std::unique_ptr<char[]> p;
  explicit Exact(size_t bytes) : p(new char[bytes]()) {}
  char* get() const { return p.get(); }
};
size_t extent(size_t rows, size_t stride, size_t cols) { return rows == 0 ? 0 : (rows - 1) * stride + cols; }

}  // namespace

int main() {
  const int types[] = {GB_DTYPE_F32, GB_DTYPE_F16, GB_DTYPE_BF16}, id_types[] = {GB_DTYPE_I32, GB_DTYPE_I64};
  for (int k = 0; k < 300; k++) {
    const int t = types[pick(0, 2)], pt = types[pick(0, 2)], gt = types[pick(0, 2)], it = id_types[pick(0, 1)];
    const size_t rows = pick(0, 40), cols = pick(1, 60), e = size_of(t);
    const size_t sx = cols + pick(0, 3), sy = cols + pick(0, 3), sd = cols + pick(0, 3);
    Exact x(extent(rows, sx, cols) * e), y(extent(rows, sy, cols) * e), dx(extent(rows, sd, cols) * e);
    Exact w(cols * size_of(pt)), mean(4 * rows), rstd(4 * rows), dw(cols * size_of(gt)), db(cols * size_of(gt));
    expect(gb_layer_norm_forward(t, y.get(), sy, x.get(), sx, rows, cols, pt, w.get(), k % 3 ? w.get() : nullptr, 1e-5,
                                 (float*)mean.get(), (float*)rstd.get(), nullptr) == GB_OK, "forward");
    const size_t need = gb_layer_norm_workspace_bytes(rows, cols);
    Exact ws(need);
    const bool sums = k % 4 != 0;
    expect(gb_layer_norm_backward(t, dx.get(), sd, y.get(), sy, x.get(), sx, rows, cols, (float*)mean.get(),
                                  (float*)rstd.get(), pt, w.get(), gt, sums ? dw.get() : nullptr,
                                  sums ? db.get() : nullptr, k % 2, ws.get(), need, nullptr) == GB_OK, "backward");
    if (sums && rows > 0) {
      expect(gb_layer_norm_backward(t, dx.get(), sd, y.get(), sy, x.get(), sx, rows, cols, (float*)mean.get(),
                                    (float*)rstd.get(), pt, w.get(), gt, dw.get(), db.get(), 0, ws.get(), need - 1,
                                    nullptr) == GB_ERR_WORKSPACE, "a byte too few");
    }
    const size_t tokens = k % 10 ? pick(0, 300) : pick(8000, 12000), vocab = pick(1, 100), dim = pick(1, 20);
    const size_t st = dim + pick(0, 3), so = dim + pick(0, 3);
    Exact table(extent(vocab, st, dim) * size_of(gt)), out(extent(tokens, so, dim) * e), ids(tokens * size_of(it));
    expect(gb_embedding_forward(t, out.get(), so, gt, table.get(), st, vocab, dim, it, ids.get(), tokens, -5, 2.0,
                                nullptr) == GB_OK, "lookup");
    const size_t space = gb_embedding_workspace_bytes(tokens, vocab, dim);
    Exact work(space);
    expect(gb_embedding_backward(gt, table.get(), st, vocab, dim, t, out.get(), so, it, ids.get(), tokens, 3, -1, 0.5,
                                 k % 2, work.get(), space, nullptr) == GB_OK, "table gradient");
    if (tokens > 0) {
      expect(gb_embedding_backward(gt, table.get(), st, vocab, dim, t, out.get(), so, it, ids.get(), tokens, 3, -1, 0.5,
                                   0, work.get(), space - 1, nullptr) == GB_ERR_WORKSPACE, "a byte too few");
      g_fail = 1;
      expect(gb_embedding_backward(gt, table.get(), st, vocab, dim, t, out.get(), so, it, ids.get(), tokens, 3, -1, 0.5,
                                   0, work.get(), space, nullptr) == GB_ERR_HIP, "a launch that fails");
      g_fail = 0;
    }
  }
  // the largest sizes: no product wraps
  const size_t most = GB_MAX_N;
  expect(gb_layer_norm_workspace_bytes(most, 1) > 0 && gb_layer_norm_workspace_bytes(~(size_t)0, 1) == 0, "rows");
  expect(gb_embedding_workspace_bytes(1 << 30, 1 << 30, 512) > 0, "tokens");
  expect(gb_embedding_workspace_bytes(~(size_t)0, ~(size_t)0, ~(size_t)0) == 0, "every size");
  float f[4] = {};
  expect(gb_layer_norm_forward(0, f, ~(size_t)0, f, ~(size_t)0, ~(size_t)0, 2, 0, nullptr, nullptr, 1e-5, nullptr,
                               nullptr, nullptr) == GB_ERR_INVALID_ARG, "rows beyond the largest");
  expect(gb_layer_norm_forward(0, f, ~(size_t)0, f, 1, 2, 1, 0, nullptr, nullptr, 1e-5, nullptr, nullptr, nullptr) ==
             GB_ERR_INVALID_ARG, "a stride beyond the largest");
  std::printf("%ld launches, %ld failed\n", g_launches, g_failed);
  return g_failed == 0 ? 0 : 1;
}
