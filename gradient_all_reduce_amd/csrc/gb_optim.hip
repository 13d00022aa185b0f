// gb_optim.hip — the optimizer step: the global gradient norm with clipping,
// and AdamW over the tensors of a plan with float32 or 8-bit moments.  The
// formulas stand in include/gbreduce.h.
//
// All of it streams HBM (no contraction, so no MFMA): the norm reads each
// gradient once, the step reads and writes each value of every buffer once.
// Measured on MI355X, algorithmic bytes over kernel time, where the best plain
// copy moves 6.6 TB/s and a plain read 7.1-7.5: the norm of 1e9 float32 values
// 567 us (7.06 TB/s), of 1e9 bfloat16 values 299 us (6.7 TB/s); the float32 step
// over 1e9 values 4,322 us (6.48 TB/s); over 67M values with bfloat16 gradients
// and copies 290 us (6.5 TB/s); the 8-bit step over 1e9 such values 2,586 us
// (6.2 TB/s).  Counted traffic over algorithmic bytes: the steps 1.0005 to 1.0013
// from 67M values on, 1.0012 (float32) and 1.0033 (8-bit) over ragged lists of
// 24-26M; the norm 1.008 (float32) and 1.016 (bfloat16), 32 bytes more a chunk,
// whose 8-byte table entries share lines that several XCDs read.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Wunused-function"  // of the shared helpers, some have no use here
#include "gb_device.h"
#pragma clang diagnostic pop
#include "gb_optim.h"

namespace gb {
namespace {

// A wavefront takes a block of 256 values, 4 consecutive ones per lane.
constexpr int kWave = 64;
constexpr int kWaves = kThreads / kWave;
// Up to this many chunks the norm is one launch of one workgroup: 64 chunks
// take 5.2 us there and 5.1 us in two launches of a replayed graph (4 chunks
// 2.9 and 4.6, 128 chunks 7.4 and 5.1), called from Python 5.1 and 8.2 us.
constexpr uint32_t kNormSmall = 64;
// Up to this many bytes of gradients the norm pass reads them without the
// non-temporal hint: the step that follows then finds some of them in the
// 256 MiB last-level cache.  Norm and step together, hint left out / given:
//   steps back to back, float32: 85 / 91 us at 67 MB of gradients, 162 / 175
//     at 134, 324 / 358 at 268, 684 / 710 at 537;
//   the gradients written last, as an all-reduce leaves them: float32 93 / 95,
//     173 / 181, 356 / 351, 709 / 714; bfloat16 with 8-bit moments 107 / 115
//     at 67 MB, 200 / 212 at 134, 388 / 404 at 268;
//   1 GiB of other values written last: 102 / 94, 198 / 179, 371 / 338, 718 /
//     670, since reads that stay in the cache push those values out first.
// At 4 GB of gradients, which the cache cannot hold, the norm pass alone
// takes 648 us without the hint and 581 with it.
constexpr size_t kNormKeepBytes = (size_t)640 << 20;

// ---------------------------------------------------------------------------
// Access through the plan's pointers.  They come out of a table in memory, so
// the compiler takes them for generic ones unless told otherwise: as global
// pointers their loads and stores need no aperture check and no wait on the
// LDS counter.  Parameters, gradients and copies may be views into a bucket
// that start at any value, so theirs are aligned to the element only.
// ---------------------------------------------------------------------------
#define GB_GLOBAL __attribute__((address_space(1)))
typedef f4 f4_any __attribute__((aligned(4)));
typedef u2 u2_any __attribute__((aligned(2)));

template <class V, class T>
__device__ __forceinline__ const GB_GLOBAL V* global_at(const T* p, size_t i) {
  return (const GB_GLOBAL V*)(p + i);
}
template <class V, class T>
__device__ __forceinline__ GB_GLOBAL V* global_at(T* p, size_t i) {
  return (GB_GLOBAL V*)(p + i);
}

// A lane's four values.  ANY: aligned to the element only.  The under-aligned
// types are named where the access is made: given as a template argument a
// type loses its alignment attribute, and the access would promise 16 bytes.
// KEEP: without the non-temporal hint, so that a later pass over the same
// values finds them in the last-level cache.
template <bool ANY, bool KEEP>
__device__ __forceinline__ f4 load_vec4(const float* p, size_t i) {
  if constexpr (ANY) {
    const GB_GLOBAL f4_any* v = (const GB_GLOBAL f4_any*)(p + i);
    if constexpr (KEEP) return *v;
    else return __builtin_nontemporal_load(v);
  } else {
    const GB_GLOBAL f4* v = (const GB_GLOBAL f4*)(p + i);
    if constexpr (KEEP) return *v;
    else return __builtin_nontemporal_load(v);
  }
}
template <bool KEEP>
__device__ __forceinline__ u2 load_vec4(const uint16_t* p, size_t i) {
  const GB_GLOBAL u2_any* v = (const GB_GLOBAL u2_any*)(p + i);
  if constexpr (KEEP) return *v;
  else return __builtin_nontemporal_load(v);
}

// Values [i, i + 4), zero at and beyond n.
template <bool ANY, bool FULL, bool KEEP = false>
__device__ __forceinline__ f4 load_f4(const float* p, size_t i, size_t n) {
  if (FULL || i + 4 <= n) return load_vec4<ANY, KEEP>(p, i);
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int e = 0; e < 3; e++) {
    if (i + e < n) v[e] = *global_at<float>(p, i + e);
  }
  return v;
}
template <bool ANY, bool FULL>
__device__ __forceinline__ void store_f4(float* p, size_t i, size_t n, f4 v) {
  if (FULL || i + 4 <= n) {
    if constexpr (ANY) __builtin_nontemporal_store(v, (GB_GLOBAL f4_any*)(p + i));
    else __builtin_nontemporal_store(v, (GB_GLOBAL f4*)(p + i));
    return;
  }
  for (int e = 0; e < 3; e++) {
    if (i + e < n) *global_at<float>(p, i + e) = v[e];
  }
}
// Four 2-byte values as two words.
template <bool FULL, bool KEEP = false>
__device__ __forceinline__ u2 load_half4(const void* p, size_t i, size_t n) {
  const uint16_t* h = static_cast<const uint16_t*>(p);
  if (FULL || i + 4 <= n) return load_vec4<KEEP>(h, i);
  uint32_t w[2] = {0u, 0u};
  for (int e = 0; e < 3; e++) {
    if (i + e < n) w[e >> 1] |= (uint32_t)*global_at<uint16_t>(h, i + e) << (16 * (e & 1));
  }
  return u2{w[0], w[1]};
}
template <bool FULL>
__device__ __forceinline__ void store_half4(void* p, size_t i, size_t n, u2 w) {
  uint16_t* h = static_cast<uint16_t*>(p);
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(w, (GB_GLOBAL u2_any*)(h + i));
    return;
  }
  const uint32_t ws[2] = {w.x, w.y};
  for (int e = 0; e < 3; e++) {
    if (i + e < n) *global_at<uint16_t>(h, i + e) = (uint16_t)(ws[e >> 1] >> (16 * (e & 1)));
  }
}
// Four codes as a word (the arrays are 16-byte aligned, i a multiple of 4).
template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const void* p, size_t i, size_t n) {
  const uint8_t* c = static_cast<const uint8_t*>(p);
  if (FULL || i + 4 <= n) return __builtin_nontemporal_load(global_at<uint32_t>(c, i));
  uint32_t w = 0;
  for (int e = 0; e < 3; e++) {
    if (i + e < n) w |= (uint32_t)*global_at<uint8_t>(c, i + e) << (8 * e);
  }
  return w;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void* p, size_t i, size_t n, uint32_t w) {
  uint8_t* c = static_cast<uint8_t*>(p);
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(w, global_at<uint32_t>(c, i));
    return;
  }
  for (int e = 0; e < 3; e++) {
    if (i + e < n) *global_at<uint8_t>(c, i + e) = (uint8_t)(w >> (8 * e));
  }
}
// Values [i, i + 4) of a gradient as binary32 (exact), zero at and beyond n.
template <int ET, bool FULL, bool KEEP = false>
__device__ __forceinline__ f4 load_grad4(const void* p, size_t i, size_t n) {
  if constexpr (ET == GB_DTYPE_F32) {
    return load_f4<true, FULL, KEEP>(static_cast<const float*>(p), i, n);
  } else {
    const u2 w = load_half4<FULL, KEEP>(p, i, n);
    if constexpr (ET == GB_DTYPE_BF16) return bf16_unpack4(w);
    const h4 h = __builtin_bit_cast(h4, w);
    return f4{(float)h.x, (float)h.y, (float)h.z, (float)h.w};
  }
}
// v, whose NaNs are canonical, rounded to the tensor's copy.
template <bool FULL>
__device__ __forceinline__ void store_copy4(const OptimTensor& t, size_t i, size_t n, f4 v) {
  void* p = t.copy;
  if (t.types >> 16 == GB_DTYPE_BF16) {
    // the converting instruction rounds to nearest even, two values at a
    // time, where bf16_pack4 takes seven instructions a value
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    store_half4<FULL>(p, i, n, __builtin_bit_cast(u2, __builtin_convertvector(v, b4)));
  } else {
    asm volatile("" : "+v"(v));  // binary32 first, then its rounding to float16 (gb_device.h, store_vals4_at)
    const h4 h = {(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
    store_half4<FULL>(p, i, n, __builtin_bit_cast(u2, h));
  }
}

// ---------------------------------------------------------------------------
// The plan's tables
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void optim_upload_kernel(OptimTensor* tensors, OptimChunk* chunks,
                                                                OptimUpload up) {
  const uint32_t i = blockIdx.x;
  if (i >= up.count) return;
  const uint32_t tensor = up.first_tensor + i;
  if (blockIdx.y == 0 && threadIdx.x == 0) tensors[tensor] = up.t[i];
  const uint32_t count = (uint32_t)((up.t[i].n + kOptimChunk - 1) / kOptimChunk);
  for (uint32_t c = blockIdx.y * kThreads + threadIdx.x; c < count; c += gridDim.y * kThreads) {
    chunks[up.first_chunk[i] + c] = OptimChunk{tensor, c};
  }
}

// ---------------------------------------------------------------------------
// Opening a step
// ---------------------------------------------------------------------------
struct StepArgs {
  double beta1, beta2, max_norm, inv_scale;
  uint64_t seed;
};

// b^t by squaring: the same sequence of binary64 products everywhere.
__device__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// What the next step's number alone decides.
struct Opening {
  int64_t step;
  float rate1, rate2;
  uint32_t key;
};
// 1 / (1 - b^t), or 1 / sqrt(1 - b^t).
__device__ float bias_rate(double b, int64_t t, bool root) {
  const double x = 1.0 - power(b, t);
  return (float)(1.0 / (root ? sqrt(x) : x));
}
__device__ uint32_t dither_key(uint64_t seed, int64_t t) {
  constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
  uint64_t z = seed + (uint64_t)t * kGolden;
  for (int i = 0; i < 3; i++) z = (z ^ (z >> 32)) * kGolden;
  return (uint32_t)(z >> 32);
}
__device__ Opening next_step(const gb_optim_control* c, const StepArgs& a) {
  const int64_t t = c->step + 1;
  return Opening{t, bias_rate(a.beta1, t, false), bias_rate(a.beta2, t, true), dither_key(a.seed, t)};
}
__device__ void open_step(gb_optim_control* c, const Opening& o, float coef) {
  c->step = o.step;
  c->skip = 0;
  c->coef = coef;
  c->rate1 = o.rate1;
  c->rate2 = o.rate2;
  c->key = o.key;
}

// Two lanes, one for each rate.  Both read the step count that one of them
// then writes, hence the barrier (in one wavefront, a wait).
__global__ __launch_bounds__(kWave) void optim_begin_kernel(gb_optim_control* c, StepArgs a) {
  const int64_t t = c->step + 1;
  const bool second = threadIdx.x != 0;
  const float rate = bias_rate(second ? a.beta2 : a.beta1, t, second);
  __syncthreads();
  if (second) c->rate2 = rate;
  else {
    c->rate1 = rate;
    c->step = t;
    c->skip = 0;
    c->coef = (float)a.inv_scale;
    c->key = dither_key(a.seed, t);
  }
}

__device__ void close_norm(gb_optim_control* c, const StepArgs& a, const Opening& o, double sum) {
  const double norm = a.inv_scale * sqrt(sum);
  c->norm = (float)norm;
  if (!(fabsf((float)norm) < __builtin_inff())) {
    c->coef = 0.0f;
    c->skip = 1;
    c->skipped += 1;
    return;
  }
  open_step(c, o, (float)(norm > a.max_norm ? a.inv_scale * a.max_norm / norm : a.inv_scale));
}

// Sum over the workgroup, in an order fixed by the lane numbers; every thread
// receives it.
template <int WAVES>
__device__ double group_sum(double s) {
  __shared__ double part[WAVES];
  for (int d = kWave / 2; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = s;
  __syncthreads();
  double sum = part[0];
#pragma unroll
  for (int w = 1; w < WAVES; w++) sum += part[w];
  return sum;
}

constexpr int kNormVecs = kOptimChunk / (4 * kWave);

// Adds the squares of a chunk to s, the wavefront's lanes 4 values apart.
// The product of two widened binary32 values is exact in binary64.
template <int ET, bool FULL, bool KEEP>
__device__ __forceinline__ double chunk_squares(const void* g, size_t i, size_t n, double s) {
  f4 x[kNormVecs];
#pragma unroll
  for (int j = 0; j < kNormVecs; j++) x[j] = load_grad4<ET, FULL, KEEP>(g, i + j * 4 * kWave, n);
#pragma unroll
  for (int j = 0; j < kNormVecs; j++) {
#pragma unroll
    for (int e = 0; e < 4; e++) s = fma((double)x[j][e], (double)x[j][e], s);
  }
  return s;
}
template <int ET, bool KEEP>
__device__ __forceinline__ double chunk_squares(const OptimTensor& t, uint32_t chunk, double s) {
  const size_t first = (size_t)chunk * kOptimChunk, i = first + threadIdx.x % kWave * 4;
  return first + kOptimChunk <= t.n ? chunk_squares<ET, true, KEEP>(t.g, i, t.n, s)
                                    : chunk_squares<ET, false, KEEP>(t.g, i, t.n, s);
}

// The sum of the squares of chunks wave, wave + waves, ...: one chunk at a
// time per wavefront, so that the tables are read as scalars and four loads
// per lane are in flight; the next chunk's entry is read ahead.
template <bool KEEP>
__device__ __forceinline__ double wave_squares(const OptimTensor* tensors, const OptimChunk* chunks, uint32_t count,
                                               uint32_t wave, uint32_t waves) {
  double s = 0.0;
  if (wave >= count) return s;
  OptimChunk next = chunks[wave];
  for (uint32_t b = wave; b < count; b += waves) {
    const OptimChunk c = next;
    if (b + waves < count) next = chunks[b + waves];
    const OptimTensor& t = tensors[c.tensor];
    const uint32_t dtype = t.types & 0xFFFFu;
    if (dtype == GB_DTYPE_F32) s = chunk_squares<GB_DTYPE_F32, KEEP>(t, c.chunk, s);
    else if (dtype == GB_DTYPE_F16) s = chunk_squares<GB_DTYPE_F16, KEEP>(t, c.chunk, s);
    else s = chunk_squares<GB_DTYPE_BF16, KEEP>(t, c.chunk, s);
  }
  return s;
}
__device__ __forceinline__ uint32_t wave_in_group() {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
}

// The norm in two launches: a partial sum per workgroup, then one workgroup
// that adds them and opens the step.  (Counting the workgroups instead, so
// that the last one adds, needs a release at device scope in each of them,
// which on this chip writes the XCD's L2 back: 78 us instead of 16 for
// 50 MB of gradients, and 19 us of that remain with relaxed atomics.)  Bound
// by the reads: 1,024 workgroups, 512, 2,048 or 16,384, contiguous shares or
// strided ones, one or two chunks at a time all stay within 3%, 6.7-7.0 TB/s
// for 4 GB of float32 (measured there only).  50 MB in 300 ragged bfloat16
// tensors take 14.8 us with the second launch: 11.0 in this kernel (4.6 TB/s,
// where the reads at full rate are 7.1 us) and 3.8 in the one that adds.
// Most of what is lost there is lost in this kernel: 4,096 wavefronts take six
// or seven chunks each, one after the other, table entries ahead of the data.
template <bool KEEP>
__global__ __launch_bounds__(kThreads) void optim_norm_kernel(const OptimTensor* tensors, const OptimChunk* chunks,
                                                              uint32_t count, double* partials) {
  const double s = group_sum<kWaves>(
      wave_squares<KEEP>(tensors, chunks, count, blockIdx.x * kWaves + wave_in_group(), gridDim.x * kWaves));
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}
// The last thread works out the new step's rates meanwhile: the powers are a
// chain of some 20 binary64 products and two divisions, about 1 us.
__global__ __launch_bounds__(kThreads) void optim_close_kernel(const double* partials, uint32_t count,
                                                               gb_optim_control* control, StepArgs a) {
  __shared__ Opening opening;
  double s = 0.0;
  for (uint32_t b = threadIdx.x; b < count; b += kThreads) s += partials[b];
  if (threadIdx.x == kThreads - 1) opening = next_step(control, a);
  s = group_sum<kWaves>(s);
  if (threadIdx.x == 0) close_norm(control, a, opening, s);
}
// Few chunks: one workgroup does both.
constexpr int kSmallThreads = 1024;
__global__ __launch_bounds__(kSmallThreads) void optim_norm_small_kernel(const OptimTensor* tensors,
                                                                         const OptimChunk* chunks, uint32_t count,
                                                                         gb_optim_control* control, StepArgs a) {
  constexpr int waves = kSmallThreads / kWave;
  __shared__ Opening opening;
  if (threadIdx.x == kSmallThreads - 1) opening = next_step(control, a);
  const double s = group_sum<waves>(wave_squares<true>(tensors, chunks, count, wave_in_group(), waves));
  if (threadIdx.x == 0) close_norm(control, a, opening, s);
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
struct AdamArgs {
  float beta1, gain1, beta2, gain2, eps;  // gain = 1 - beta
};

// The step's scalars of one tensor.
struct Rates {
  float coef, rate2, decay, step;
};
__device__ __forceinline__ Rates tensor_rates(const gb_optim_control* c, const OptimTensor& t) {
  const float lr = c->lr * t.lr_scale;
  return Rates{c->coef, c->rate2, 1.0f - lr * t.weight_decay, lr * c->rate1};
}

// m and v become m' and v', u becomes sqrt(v'), p becomes p'.
__device__ __forceinline__ void adamw4(const AdamArgs& a, const Rates& r, f4 g, f4& p, f4& m, f4& v, f4& u) {
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const float gs = g[e] * r.coef;
    m[e] = a.beta1 * m[e] + a.gain1 * gs;
    v[e] = a.beta2 * v[e] + a.gain2 * (gs * gs);
    u[e] = __builtin_sqrtf(v[e]);
    const float d = u[e] * r.rate2 + a.eps;
    p[e] = p[e] * r.decay - r.step * (m[e] / d);
  }
}

// A step workgroup is one wavefront that takes 256 values, a quarter of a
// chunk.  From one run on, consecutive workgroups take groups of 8 fronts
// 1 MiB of float32 apart (GroupOrder in gb_device.h says why).
// Chunks go to launches of at most kLaunchChunks, which keeps a launch's
// lanes below 2^32.
constexpr uint32_t kPerChunk = kOptimChunk / kBlock;
constexpr uint32_t kLaunchChunks = 1u << 23;
// The float32 step holds LDS it does not use, so that 14 workgroups share a
// CU, and 11 from 2^27 values in a launch; 64-lane workgroups leave room for
// 32, and fewer streams at once read and write faster.  Uncapped against 16:
// 67M bfloat16 values with a copy 304 against 297 us.  In one buffer per
// stream, 16, 14, 12, 11, 9 and 8 per CU, us:
//   float32: 2^24 values 73, 72, 72, 72, 74, 77; 2^26 299, 290, 288, 284, 294,
//     305; 2^27 575, 569, 567, 567, 580, 606; 2^29 2,380, 2,332, 2,293, 2,273,
//     2,312, 2,410;
//   bfloat16 with a copy: 72, 72, 72, 73, 76, 79; 298, 293, 290, 291, 301, 314;
//     590, 578, 578, 582, 601, 629; 2,398, 2,379, 2,364, 2,383, 2,447, 2,542.
// Over 1e9 values in 153 tensors 16 to 11 are level (4,466-4,500 and 4,570-
// 4,579).  The 8-bit step, with less than half the bytes in flight per
// wavefront, wants every wavefront it can have (5% slower with 20 per CU).
// LDS is handed out in granules: the occupancy query of the runtime does not
// know them, so these counts are from workgroups that noted their CU.
constexpr unsigned kLdsGranule = 1280, kLdsGranules = 128;
constexpr unsigned kFourteenPerCuLds = 9 * kLdsGranule, kElevenPerCuLds = 11 * kLdsGranule;
static_assert(kLdsGranules / (kFourteenPerCuLds / kLdsGranule) == 14 && kLdsGranules / (kElevenPerCuLds / kLdsGranule) == 11,
              "the reservations leave the workgroups they are named for");
constexpr uint32_t kElevenFromChunks = (uint32_t)(((size_t)1 << 27) / kOptimChunk);
using StepOrder = GroupOrder<8, 1024, 1>;

struct Piece {
  OptimTensor t;  // a copy: the entry is read once, ahead of every store
  size_t first;  // of 256 values
};
__device__ __forceinline__ Piece step_piece(const OptimTensor* tensors, const OptimChunk* chunks) {
  const uint32_t w = (uint32_t)group_index<StepOrder>();
  const OptimChunk c = chunks[w / kPerChunk];
  return Piece{tensors[c.tensor], (size_t)c.chunk * kOptimChunk + w % kPerChunk * kBlock};
}

// Bound by its reads and writes: 28 bytes a value.  One 16-byte vector per
// lane and stream is best: 2 or 4 of them per wavefront lose 2-5% at every
// occupancy, 256-lane workgroups in index order 6%.
template <int ET, bool FULL>
__device__ __forceinline__ void adamw_f32_piece(const OptimTensor& t, const AdamArgs& a, const Rates& r, size_t i) {
  const size_t n = t.n;
  const f4 g = load_grad4<ET, FULL>(t.g, i, n);
  f4 p = load_f4<true, FULL>(t.p, i, n);
  f4 m = load_f4<false, FULL>(static_cast<const float*>(t.m), i, n);
  f4 v = load_f4<false, FULL>(static_cast<const float*>(t.v), i, n);
  f4 u;
  adamw4(a, r, g, p, m, v, u);
  p = canon4(p);
  store_f4<true, FULL>(t.p, i, n, p);
  store_f4<false, FULL>(static_cast<float*>(t.m), i, n, canon4(m));
  store_f4<false, FULL>(static_cast<float*>(t.v), i, n, canon4(v));
  if (t.copy != nullptr) store_copy4<FULL>(t, i, n, p);
}

template <int ET>
__global__ __launch_bounds__(kWave) void adamw_f32_kernel(const OptimTensor* tensors, const OptimChunk* chunks,
                                                          const gb_optim_control* control, AdamArgs a) {
  const Piece w = step_piece(tensors, chunks);
  // one test, so that the control block's line and the tables' are on their
  // way together
  if ((control->skip != 0) | (w.first >= w.t.n)) return;
  const Rates r = tensor_rates(control, w.t);
  const size_t i = w.first + threadIdx.x * 4;
  if (w.first + kBlock <= w.t.n) adamw_f32_piece<ET, true>(w.t, a, r, i);
  else adamw_f32_piece<ET, false>(w.t, a, r, i);
}

// The largest magnitude of the wavefront's values, as a bit pattern; NaN
// counts as 0 (the maximum instruction passes over it).
__device__ __forceinline__ uint32_t wave_absmax(f4 x) {
  const float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
  const uint32_t top = row_max16(a == a ? fbits(a) : 0u);
  const uint32_t r0 = (uint32_t)__builtin_amdgcn_readlane((int)top, 0);
  const uint32_t r1 = (uint32_t)__builtin_amdgcn_readlane((int)top, 16);
  const uint32_t r2 = (uint32_t)__builtin_amdgcn_readlane((int)top, 32);
  const uint32_t r3 = (uint32_t)__builtin_amdgcn_readlane((int)top, 48);
  return max(max(r0, r1), max(r2, r3));
}
// The same over the finite values only: x with 0 for the others.
__device__ __forceinline__ f4 finite4(f4 x) {
#pragma unroll
  for (int e = 0; e < 4; e++) x[e] = fabsf(x[e]) < __builtin_inff() ? x[e] : 0.0f;
  return x;
}

// Exponent e of a block's scale 2^e: the smallest, at least -126, with
// a <= 448 * 2^e = 1.75 * 2^(e + 8); 0 for a = 0.  A finite a gives e <= 120.
__device__ __forceinline__ int scale_exponent(uint32_t abits) {
  if (abits == 0u) return 0;
  return max((int)((abits + 0x1FFFFFu) >> 23) - 135, -126);  // the sum carries where the fraction exceeds 0.75
}
__device__ __forceinline__ float pow2(int e) { return bitsf((uint32_t)(e + 127) << 23); }

// Four E4M3 codes of q by the dither in the top 20 bits of each seed.  The
// converter adds them to the 20 significand bits that the code drops (of a
// subnormal code, after the significand has been shifted right to it) and
// truncates; |q| <= 448, so nothing reaches beyond 448.
__device__ __forceinline__ uint32_t dithered4(f4 q, const uint32_t (&seed)[4]) {
  int w = 0;
  w = __builtin_amdgcn_cvt_sr_fp8_f32(q.x, (int)seed[0], w, 0);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(q.y, (int)seed[1], w, 1);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(q.z, (int)seed[2], w, 2);
  w = __builtin_amdgcn_cvt_sr_fp8_f32(q.w, (int)seed[3], w, 3);
  return (uint32_t)w;
}

// The codes of values that are not finite become 0x7F.
__device__ __forceinline__ uint32_t mark_not_finite(f4 x, uint32_t w) {
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if (!(fabsf(x[e]) < __builtin_inff())) w = (w & ~(0xFFu << (8 * e))) | (0x7Fu << (8 * e));
  }
  return w;
}

__device__ __forceinline__ uint32_t dither_word(uint32_t x) {
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  return x ^ (x >> 16);
}

// Bound by its reads and writes, 16 bytes a value in 8 streams (with the copy):
// the same kernel with approximate roots and quotients and no dither is 0.3%
// faster.  The arithmetic is near enough to matter, though: 70 vector
// instructions a value, down from over 100, which took the handling of values
// that are not finite out of the common path, one conversion instruction for
// two bfloat16 copies, and the block's part of the dither on the scalar unit.
// One block per wavefront: the largest magnitude takes four row steps and
// four lane reads, no LDS; 2 or 4 blocks with their loads ahead lose 4 and 15%
// (fewer wavefronts), stores without the non-temporal hint 11%.
template <int ET, bool FULL>
__device__ __forceinline__ void adamw_e4m3_block(const OptimTensor& t, const AdamArgs& a, const Rates& r,
                                                 uint32_t key, size_t first) {
  const size_t n = t.n, block = first / kBlock, i = first + threadIdx.x * 4;
  const f4 g = load_grad4<ET, FULL>(t.g, i, n);
  f4 p = load_f4<true, FULL>(t.p, i, n);
  const uint32_t mw = load_codes<FULL>(t.m, i, n), vw = load_codes<FULL>(t.v, i, n);
  // The scales come as vector loads although their address is the same in
  // every lane: 4 bytes a block through the scalar cache made the step 6%
  // slower.  The empty asm keeps the address in vector registers.
  size_t at = block;
  asm("" : "+v"(at));
  f4 m = e4m3_unpack4(mw) * *global_at<float>(t.ms, at);
  f4 u = e4m3_unpack4(vw) * *global_at<float>(t.vs, at);
  f4 v = u * u;
  adamw4(a, r, g, p, m, v, u);

  // What is not finite is rare and handled for the wavefront as a whole: a
  // NaN in m' or u reaches p', an infinity shows in the largest magnitude.
  uint32_t mtop = wave_absmax(m), utop = wave_absmax(u);
  const bool nan = __builtin_isunordered(p.x, p.y) || __builtin_isunordered(p.z, p.w);
  const bool special = mtop >= 0x7F800000u || utop >= 0x7F800000u || __any(nan);
  if (special) {
    p = canon4(p);
    mtop = wave_absmax(finite4(m));
    utop = wave_absmax(finite4(u));
  }
  store_f4<true, FULL>(t.p, i, n, p);
  if (t.copy != nullptr) store_copy4<FULL>(t, i, n, p);

  const int me = scale_exponent(mtop), ue = scale_exponent(utop);
  const f4 mq = m * pow2(-me);
  f4 uq = u * pow2(-ue);
  // a root above 0 keeps a code: at least the smallest, 2^-9
  if (__any(fminf(fminf(uq.x, uq.y), fminf(uq.z, uq.w)) < 0x1p-9f)) {
#pragma unroll
    for (int e = 0; e < 4; e++) uq[e] = u[e] > 0.0f ? fmaxf(uq[e], 0x1p-9f) : uq[e];
  }
  const uint32_t base = (t.first_block * 128u + (uint32_t)(first / 2)) * 0x9E3779B9u + key;  // of the block's first pair
  const uint32_t x = base + threadIdx.x * (2 * 0x9E3779B9u);
  const uint32_t x0 = dither_word(x), x1 = dither_word(x + 0x9E3779B9u);
  const uint32_t seed[4] = {x0, x0 << 16, x1, x1 << 16};
  uint32_t mc = dithered4(mq, seed), uc = dithered4(uq, seed);
  if (special) {
    mc = mark_not_finite(m, mc);
    uc = mark_not_finite(u, uc);
  }
  store_codes<FULL>(t.m, i, n, mc);
  store_codes<FULL>(t.v, i, n, uc);
  if (threadIdx.x == 0) {
    *global_at<float>(t.ms, block) = pow2(me);
    *global_at<float>(t.vs, block) = pow2(ue);
  }
}

template <int ET>
__global__ __launch_bounds__(kWave) void adamw_e4m3_kernel(const OptimTensor* tensors, const OptimChunk* chunks,
                                                           const gb_optim_control* control, AdamArgs a) {
  const Piece w = step_piece(tensors, chunks);
  // one test, so that the control block's line and the tables' are on their
  // way together
  if ((control->skip != 0) | (w.first >= w.t.n)) return;
  const Rates r = tensor_rates(control, w.t);
  if (w.first + kBlock <= w.t.n) adamw_e4m3_block<ET, true>(w.t, a, r, control->key, w.first);
  else adamw_e4m3_block<ET, false>(w.t, a, r, control->key, w.first);
}

StepArgs step_args(const OptimPlan& plan, double max_norm, double inv_scale) {
  return StepArgs{plan.beta1, plan.beta2, max_norm, inv_scale, plan.seed};
}

}  // namespace

hipError_t launch_optim_upload(OptimTensor* tensors, OptimChunk* chunks, const OptimUpload& up, hipStream_t stream) {
  (void)hipGetLastError();
  optim_upload_kernel<<<dim3(up.count, 8), kThreads, 0, stream>>>(tensors, chunks, up);
  return hipGetLastError();
}

hipError_t launch_optim_begin(const OptimPlan& plan, gb_optim_control* control, double inv_scale,
                              hipStream_t stream) {
  (void)hipGetLastError();
  optim_begin_kernel<<<1, 2, 0, stream>>>(control, step_args(plan, 0.0, inv_scale));
  return hipGetLastError();
}

hipError_t launch_optim_begin_clip(const OptimPlan& plan, gb_optim_control* control, double max_norm,
                                   double inv_scale, hipStream_t stream) {
  const uint32_t count = plan.first[kOptimKinds];
  const StepArgs a = step_args(plan, max_norm, inv_scale);
  (void)hipGetLastError();
  if (count <= kNormSmall) {
    optim_norm_small_kernel<<<1, kSmallThreads, 0, stream>>>(plan.tensors, plan.chunks, count, control, a);
    return hipGetLastError();
  }
  const uint32_t groups = (count + kWaves - 1) / kWaves < kNormGroups ? (count + kWaves - 1) / kWaves : kNormGroups;
  const auto kernel = plan.grad_bytes <= kNormKeepBytes ? optim_norm_kernel<true> : optim_norm_kernel<false>;
  kernel<<<groups, kThreads, 0, stream>>>(plan.tensors, plan.chunks, count, plan.partials);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  optim_close_kernel<<<1, kThreads, 0, stream>>>(plan.partials, groups, control, a);
  return hipGetLastError();
}

hipError_t launch_adamw(const OptimPlan& plan, const gb_optim_control* control, hipStream_t stream) {
  using Kernel = void (*)(const OptimTensor*, const OptimChunk*, const gb_optim_control*, AdamArgs);
  static const Kernel kernels[kOptimKinds] = {
      adamw_f32_kernel<GB_DTYPE_F32>,  adamw_f32_kernel<GB_DTYPE_F16>,  adamw_f32_kernel<GB_DTYPE_BF16>,
      adamw_e4m3_kernel<GB_DTYPE_F32>, adamw_e4m3_kernel<GB_DTYPE_F16>, adamw_e4m3_kernel<GB_DTYPE_BF16>};
  const AdamArgs a = {(float)plan.beta1, (float)(1.0 - plan.beta1), (float)plan.beta2, (float)(1.0 - plan.beta2),
                      plan.eps};
  (void)hipGetLastError();
  for (int k = 0; k < kOptimKinds; k++) {
    for (uint32_t c = plan.first[k]; c < plan.first[k + 1]; c += kLaunchChunks) {
      const uint32_t left = plan.first[k + 1] - c, count = left < kLaunchChunks ? left : kLaunchChunks;
      const unsigned lds = k >= 3 ? 0 : count < kElevenFromChunks ? kFourteenPerCuLds : kElevenPerCuLds;
      kernels[k]<<<count * kPerChunk, kWave, lds, stream>>>(plan.tensors, plan.chunks + c, control, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace gb
