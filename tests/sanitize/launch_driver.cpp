// launch_driver.cpp — the launches of the token-sum layers, recorded on the
// host: gb_norm.hip and gb_embed.hip compiled for the host alone, with the HIP
// runtime's launch calls stood in for here, are called through the C ABI at
// sizes up to the documented limits with made-up addresses.  Every launch has
// to stay within what the hardware's packets and the runtime take, and those
// of the table's sums have to take every piece of the work once.  Test
// infrastructure: nothing here runs in the library.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "../../gradient_all_reduce_amd/csrc/gb_internal.h"
#include "../../gradient_all_reduce_amd/csrc/gb_layers.h"

namespace {

struct Launch {
  std::string kernel;
  dim3 grid, block;
  gb::SumGrid sum;  // of embedding_sum_kernel
};
// by the address that a launch names; filled before this file's own variables are
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> n;
  return n;
}
std::vector<Launch> g_launches;
dim3 g_grid, g_block;
long g_failed = 0, g_seen = 0;
char g_message[512];

void expect(bool ok, const char* what, const std::string& call) {
  if (ok) return;
  g_failed++;
  std::printf("FAILED: %s: %s (last error: %s)\n", call.c_str(), what, g_message);
}
bool has(const std::string& s, const char* part) { return s.find(part) != std::string::npos; }

}  // namespace

extern "C" {
// the calls that a <<<>>> launch makes
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  g_grid = grid, g_block = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = g_grid, *block = g_block, *lds = 0, *stream = nullptr;
  return hipSuccess;
}
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*,
                           int*) {
  names()[host] = name;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  Launch l = {names()[f], grid, block, {}};
  if (has(l.kernel, "embedding_sum_kernel")) l.sum = *static_cast<const gb::SumGrid*>(args[2]);
  g_launches.push_back(l);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "injected"; }
}

namespace gb {
gb_status fail_status(gb_status s, const char* msg) {
  std::snprintf(g_message, sizeof g_message, "%s", msg);
  return s;
}
bool call_hooks_on() { return false; }
gb_status finish_call(const char*, void*, int, size_t, int, gb_status s, double) { return s; }
}  // namespace gb

namespace {

void* at(uint64_t tib) { return reinterpret_cast<void*>(tib << 44); }

void check_launches(const std::string& call) {
  expect(!g_launches.empty(), "nothing was launched", call);
  for (const Launch& l : g_launches) {
    const uint64_t x = (uint64_t)l.grid.x * l.block.x;
    expect(l.grid.x > 0 && l.grid.y > 0 && l.grid.z > 0, "an empty grid", call);
    expect(l.block.x * l.block.y * l.block.z <= 1024, "a workgroup of more than 1,024 lanes", call);
    expect(x < (uint64_t)1 << 32, (l.kernel + " has " + std::to_string(x) + " lanes").c_str(), call);
    g_seen++;
  }
}

// Every wavefront's window and slab, and every row without a token, in one
// workgroup of one launch of the table's sums.
void check_sums(const std::string& call, size_t tokens, size_t vocab, size_t dim, size_t cols, bool accumulate) {
  uint64_t next = 0, whole = 0;
  bool first = true;
  for (const Launch& l : g_launches) {
    if (!has(l.kernel, "embedding_sum_kernel")) continue;
    const gb::SumGrid& s = l.sum;
    if (first) {
      whole = (uint64_t)s.sums + s.zeros;
      const uint64_t slabs = (dim + cols - 1) / cols;
      expect(s.slabs == slabs && s.units == (tokens + 15) / 16 * slabs, "windows times slabs", call);
      expect((uint64_t)s.sums * 4 >= s.units, "a wavefront for each window and slab", call);
      expect(accumulate ? s.zeros == 0 : s.zeros % 8 == 0 && (uint64_t)s.zeros * s.zero_each >= vocab && s.zero_each <= 64,
             "a workgroup for each row", call);
      expect(s.sums % 8 == 0, "the zeros begin on the first XCD", call);
    }
    first = false;
    expect(s.base == next && s.base % 8 == 0, "launches one after the other", call);
    next += l.grid.x;
  }
  expect(!first && next == whole, "all workgroups launched", call);
}

}  // namespace

int main() {
  const int types[] = {GB_DTYPE_F32, GB_DTYPE_F16, GB_DTYPE_BF16};
  const size_t vocabs[] = {1, 1000, 131072, (1u << 30) - 1, 1u << 30, (1u << 30) + 1, GB_EMBEDDING_MAX_VOCAB};
  const size_t counts[] = {0, 1, 64, 8192, 8193, 1u << 20, (1u << 30) - 15, 1u << 30};
  const size_t dims[] = {1, 2, 16, 64, 255, 256, 257, 512, 4096, 65536, 1u << 20};
  for (size_t vocab : vocabs) {
    for (size_t tokens : counts) {
      for (size_t dim : dims) {
        if (tokens > GB_MAX_N / dim || vocab > GB_MAX_N / dim) continue;
        for (int t : types) {
          for (int g : types) {
            for (int accumulate = 0; accumulate < 2; accumulate++) {
              const std::string call = "table gradient of " + std::to_string(tokens) + " tokens, " +
                                       std::to_string(vocab) + " x " + std::to_string(dim) + ", types " +
                                       std::to_string(t) + " and " + std::to_string(g) +
                                       (accumulate ? ", added" : "");
              g_launches.clear();
              const size_t need = gb_embedding_workspace_bytes(tokens, vocab, dim);
              expect(tokens == 0 || need > 0, "no workspace size", call);
              expect(gb_embedding_backward(g, at(1), dim, vocab, dim, t, at(2), dim, GB_DTYPE_I64, at(3), tokens, 0, -1,
                                           1.0, accumulate, at(4), need, nullptr) == GB_OK,
                     "refused", call);
              if (tokens == 0 && accumulate) continue;
              check_launches(call);
              const size_t cols = t == GB_DTYPE_F32 || g == GB_DTYPE_F32 ? 256 : 512;
              check_sums(call, tokens, vocab, dim, cols, accumulate != 0);
            }
            if (tokens == 0) continue;
            const std::string call = "lookup of " + std::to_string(tokens) + " tokens, " + std::to_string(vocab) +
                                     " x " + std::to_string(dim);
            g_launches.clear();
            expect(gb_embedding_forward(t, at(1), dim, g, at(2), dim, vocab, dim, GB_DTYPE_I32, at(3), tokens, 0, 1.0,
                                        nullptr) == GB_OK,
                   "refused", call);
            check_launches(call);
          }
        }
      }
    }
  }
  for (size_t cols : {(size_t)1, (size_t)7, (size_t)64, (size_t)1000, (size_t)8192, (size_t)GB_NORM_MAX_COLS}) {
    for (size_t rows : {(size_t)1, (size_t)4097, GB_MAX_N / cols}) {
      for (int t : types) {
        const std::string call = "layer norm of " + std::to_string(rows) + " x " + std::to_string(cols);
        g_launches.clear();
        const size_t need = gb_layer_norm_workspace_bytes(rows, cols);
        expect(gb_layer_norm_forward(t, at(1), cols, at(2), cols, rows, cols, t, at(3), at(4), 1e-5, (float*)at(5),
                                     (float*)at(6), nullptr) == GB_OK,
               "refused", call);
        expect(gb_layer_norm_backward(t, at(1), cols, at(2), cols, at(3), cols, rows, cols, (float*)at(4),
                                      (float*)at(5), t, at(6), t, at(7), at(8), 0, at(9), need, nullptr) == GB_OK,
               "refused", call);
        check_launches(call);
      }
    }
  }
  std::printf("%ld launches, %ld failed\n", g_seen, g_failed);
  return g_failed == 0 ? 0 : 1;
}
