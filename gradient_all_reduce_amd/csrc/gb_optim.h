// gb_optim.h — what the optimizer's C-ABI layer (gb_optim_api.cpp) and its
// kernels (gb_optim.hip) share.  Not installed; the public ABI is
// include/gbreduce.h.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "gbreduce.h"

namespace gb {

// Values per chunk of a tensor: what one wavefront of the norm pass takes at a
// time, four vectors per lane, and four wavefronts of the step.  The table of
// chunks costs 8 bytes for each, below 0.1% of the step's traffic.
constexpr size_t kOptimChunk = 1024;

// A kind is the combination of gradient type and state that one step kernel
// serves; the chunks of a plan are sorted by kind.
constexpr int kOptimKinds = 6;
inline int optim_kind(int dtype, int state) { return state * 3 + dtype; }  // GB_DTYPE_F32, F16, BF16 are 0, 1, 2

// A tensor as the kernels read it from the plan's table.
struct OptimTensor {
  size_t n;
  float* p;
  const void* g;
  void* copy;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint32_t first_block;  // of 256 values, in the plan: where the dither counts from
  uint32_t types;        // the gradient's dtype, and the copy's from bit 16: a whole word, which the scalar unit loads
  float lr_scale;
  float weight_decay;
};
static_assert(sizeof(OptimTensor) == 80, "the table's entries stay 16-byte multiples");

// One entry of the chunk table: values [chunk * kOptimChunk, ...) of a tensor.
struct OptimChunk {
  uint32_t tensor;
  uint32_t chunk;
};

// Workgroups of the norm pass, and so partial sums, at most.
constexpr uint32_t kNormGroups = 1024;

// A plan's host part: what the handle's opaque words hold.
struct OptimPlan {
  uint64_t magic;
  const OptimTensor* tensors;
  const OptimChunk* chunks;  // sorted by kind
  double* partials;
  double beta1, beta2;
  uint64_t seed;
  size_t grad_bytes;  // of all gradients
  uint32_t first[kOptimKinds + 1];  // chunks [first[k], first[k + 1]) are of kind k
  float eps;
};
static_assert(sizeof(OptimPlan) <= sizeof(gb_optim_handle), "the handle holds the plan");

// Some tensors of a plan for the kernel that writes the tables, by value.
constexpr int kOptimUpload = 44;
struct OptimUpload {
  uint32_t count, first_tensor;
  uint32_t first_chunk[kOptimUpload];  // of each tensor, in the sorted table
  OptimTensor t[kOptimUpload];
};
static_assert(sizeof(OptimUpload) <= 3900, "an upload must fit the 4 KiB of kernel arguments");

// Writes the upload's entries (one at least) of both tables.
hipError_t launch_optim_upload(OptimTensor* tensors, OptimChunk* chunks, const OptimUpload& up, hipStream_t stream);
hipError_t launch_optim_begin(const OptimPlan& plan, gb_optim_control* control, double inv_scale, hipStream_t stream);
hipError_t launch_optim_begin_clip(const OptimPlan& plan, gb_optim_control* control, double max_norm,
                                   double inv_scale, hipStream_t stream);
// Every kind of the plan that has chunks.
hipError_t launch_adamw(const OptimPlan& plan, const gb_optim_control* control, hipStream_t stream);

}  // namespace gb
