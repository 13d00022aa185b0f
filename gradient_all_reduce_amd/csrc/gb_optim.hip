// gb_optim.hip — the optimizer step: the global gradient norm with clipping,
// and AdamW over the tensors of a plan with float32 or 8-bit moments.  The
// formulas stand in include/gbreduce.h.
#include "gb_device.h"
#include "gb_optim.h"

namespace gb {
namespace {

// A wavefront's block of 256 values, 4 consecutive ones per lane.
constexpr int kWave = 64;
constexpr int kWaves = kThreads / kWave;
static_assert(kOptimChunk == (size_t)kThreads * 4, "a chunk is one vector per lane of a workgroup");

// ---------------------------------------------------------------------------
// Access at the alignment of the element: parameters, gradients and copies
// may be views into a bucket that start at any value.
// ---------------------------------------------------------------------------
typedef f4 f4_any __attribute__((aligned(4)));
typedef u2 u2_any __attribute__((aligned(2)));

template <bool FULL>
__device__ __forceinline__ f4 load_f4(const float* p, size_t i, size_t n) {
  if (FULL || i + 4 <= n) return __builtin_nontemporal_load(reinterpret_cast<const f4_any*>(p + i));
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i < n) v.x = p[i];
  if (i + 1 < n) v.y = p[i + 1];
  if (i + 2 < n) v.z = p[i + 2];
  return v;
}
template <bool FULL>
__device__ __forceinline__ void store_f4(float* p, size_t i, size_t n, f4 v) {
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(v, reinterpret_cast<f4_any*>(p + i));
    return;
  }
  if (i < n) p[i] = v.x;
  if (i + 1 < n) p[i + 1] = v.y;
  if (i + 2 < n) p[i + 2] = v.z;
}
template <bool FULL>
__device__ __forceinline__ u2 load_half4(const uint16_t* p, size_t i, size_t n) {
  if (FULL || i + 4 <= n) return __builtin_nontemporal_load(reinterpret_cast<const u2_any*>(p + i));
  uint32_t w[2] = {0u, 0u};
  for (int e = 0; e < 3; e++) {
    if (i + e < n) w[e >> 1] |= (uint32_t)p[i + e] << (16 * (e & 1));
  }
  return u2{w[0], w[1]};
}
template <bool FULL>
__device__ __forceinline__ void store_half4(uint16_t* p, size_t i, size_t n, u2 w) {
  if (FULL || i + 4 <= n) {
    __builtin_nontemporal_store(w, reinterpret_cast<u2_any*>(p + i));
    return;
  }
  const uint32_t ws[2] = {w.x, w.y};
  for (int e = 0; e < 3; e++) {
    if (i + e < n) p[i + e] = (uint16_t)(ws[e >> 1] >> (16 * (e & 1)));
  }
}
// Values [i, i + 4) of a gradient as binary32 (exact), zero at and beyond n.
template <int ET, bool FULL>
__device__ __forceinline__ f4 load_grad4(const void* p, size_t i, size_t n) {
  if constexpr (ET == GB_DTYPE_F32) {
    return load_f4<FULL>(static_cast<const float*>(p), i, n);
  } else {
    const u2 w = load_half4<FULL>(static_cast<const uint16_t*>(p), i, n);
    if constexpr (ET == GB_DTYPE_BF16) return bf16_unpack4(w);
    const h4 h = __builtin_bit_cast(h4, w);
    return f4{(float)h.x, (float)h.y, (float)h.z, (float)h.w};
  }
}
template <int ET, bool FULL>
__device__ __forceinline__ void store_copy4(void* p, size_t i, size_t n, f4 v) {
  static_assert(ET != GB_DTYPE_F32, "a copy is of a 2-byte type");
  if constexpr (ET == GB_DTYPE_BF16) {
    store_half4<FULL>(static_cast<uint16_t*>(p), i, n, bf16_pack4(v));
  } else {
    asm volatile("" : "+v"(v));  // binary32 first, then its rounding to float16 (gb_device.h, store_vals4_at)
    const h4 h = {(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
    store_half4<FULL>(static_cast<uint16_t*>(p), i, n, __builtin_bit_cast(u2, h));
  }
}

// ---------------------------------------------------------------------------
// The plan's tables
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void optim_upload_kernel(OptimTensor* tensors, OptimChunk* chunks,
                                                                uint32_t* counter, OptimUpload up) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *counter = 0;
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

__device__ void open_step(gb_optim_control* c, const StepArgs& a, float coef) {
  const int64_t t = c->step + 1;
  c->step = t;
  c->skip = 0;
  c->coef = coef;
  c->rate1 = (float)(1.0 / (1.0 - power(a.beta1, t)));
  c->rate2 = (float)(1.0 / sqrt(1.0 - power(a.beta2, t)));
  constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
  uint64_t z = a.seed + (uint64_t)t * kGolden;
  for (int i = 0; i < 3; i++) z = (z ^ (z >> 32)) * kGolden;
  c->key = (uint32_t)(z >> 32);
}

__global__ void optim_begin_kernel(gb_optim_control* c, StepArgs a) { open_step(c, a, (float)a.inv_scale); }

__device__ void close_norm(gb_optim_control* c, const StepArgs& a, double sum) {
  const double norm = a.inv_scale * sqrt(sum);
  c->norm = (float)norm;
  if (!(fabsf((float)norm) < __builtin_inff())) {
    c->coef = 0.0f;
    c->skip = 1;
    c->skipped += 1;
    return;
  }
  open_step(c, a, (float)(norm > a.max_norm ? a.inv_scale * a.max_norm / norm : a.inv_scale));
}

// Sum over the workgroup, in an order fixed by the lane numbers; thread 0
// holds it.
__device__ double group_sum(double s) {
  __shared__ double part[kWaves];
  for (int d = kWave / 2; d > 0; d >>= 1) s += __shfl_xor(s, d);
  __syncthreads();  // `part` may still be read from an earlier call
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = s;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

template <int ET>
__device__ __forceinline__ double square4(const void* g, size_t i, size_t n, double s) {
  const f4 x = i + 4 <= n ? load_grad4<ET, true>(g, i, n) : load_grad4<ET, false>(g, i, n);
#pragma unroll
  for (int e = 0; e < 4; e++) s = fma((double)x[e], (double)x[e], s);  // the product is exact
  return s;
}

// Every workgroup sums the squares of its chunks (b, b + grid, ...) and
// leaves one partial sum; the workgroup that counts last adds the partials
// in order and opens the step.
__global__ __launch_bounds__(kThreads) void optim_norm_kernel(const OptimTensor* tensors, const OptimChunk* chunks,
                                                              uint32_t count, double* partials, uint32_t* counter,
                                                              gb_optim_control* control, StepArgs a) {
  double s = 0.0;
  for (uint32_t b = blockIdx.x; b < count; b += gridDim.x) {
    const OptimChunk c = chunks[b];
    const OptimTensor t = tensors[c.tensor];
    const size_t i = (size_t)c.chunk * kOptimChunk + threadIdx.x * 4;
    if (t.dtype == GB_DTYPE_F32) s = square4<GB_DTYPE_F32>(t.g, i, t.n, s);
    else if (t.dtype == GB_DTYPE_F16) s = square4<GB_DTYPE_F16>(t.g, i, t.n, s);
    else s = square4<GB_DTYPE_BF16>(t.g, i, t.n, s);
  }
  s = group_sum(s);
  __shared__ bool last;
  if (threadIdx.x == 0) {
    __hip_atomic_store(partials + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  double sum = 0.0;
  for (uint32_t b = threadIdx.x; b < gridDim.x; b += kThreads) {
    sum += __hip_atomic_load(partials + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  sum = group_sum(sum);
  if (threadIdx.x == 0) {
    *counter = 0;
    close_norm(control, a, sum);
  }
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
    p[e] = canon(p[e] * r.decay - r.step * (m[e] / d));
  }
}

template <int ET, bool FULL>
__device__ __forceinline__ void adamw_f32_chunk(const OptimTensor& t, const AdamArgs& a, const Rates& r, size_t i) {
  const size_t n = t.n;
  const f4 g = load_grad4<ET, FULL>(t.g, i, n);
  f4 p = load_f4<FULL>(t.p, i, n);
  f4 m = load4_at<FULL>(static_cast<const float*>(t.m), i, n);
  f4 v = load4_at<FULL>(static_cast<const float*>(t.v), i, n);
  f4 u;
  adamw4(a, r, g, p, m, v, u);
  store_f4<FULL>(t.p, i, n, p);
  store4_at<FULL>(static_cast<float*>(t.m), i, n, canon4(m));
  store4_at<FULL>(static_cast<float*>(t.v), i, n, canon4(v));
  if constexpr (ET != GB_DTYPE_F32) {
    if (t.copy != nullptr) store_copy4<ET, FULL>(t.copy, i, n, p);
  }
}

template <int ET>
__global__ __launch_bounds__(kThreads) void adamw_f32_kernel(const OptimTensor* tensors, const OptimChunk* chunks,
                                                             const gb_optim_control* control, AdamArgs a) {
  if (control->skip != 0) return;
  const OptimChunk c = chunks[blockIdx.x];
  const OptimTensor t = tensors[c.tensor];
  const Rates r = tensor_rates(control, t);
  const size_t first = (size_t)c.chunk * kOptimChunk, i = first + threadIdx.x * 4;
  if (first + kOptimChunk <= t.n) adamw_f32_chunk<ET, true>(t, a, r, i);
  else adamw_f32_chunk<ET, false>(t, a, r, i);
}

// The largest finite magnitude of the wavefront's values, as a bit pattern,
// the same in every lane; the values that are not finite count as 0.
__device__ __forceinline__ uint32_t wave_absmax(f4 x) {
  uint32_t b[4], top = 0u;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    b[e] = fbits(x[e]) & 0x7FFFFFFFu;
    top = max(top, b[e]);
  }
  if (top >= 0x7F800000u) {
    top = 0u;
#pragma unroll
    for (int e = 0; e < 4; e++) top = max(top, b[e] >= 0x7F800000u ? 0u : b[e]);
  }
  top = row_max16(top);
  const uint32_t r0 = (uint32_t)__builtin_amdgcn_readlane((int)top, 0);
  const uint32_t r1 = (uint32_t)__builtin_amdgcn_readlane((int)top, 16);
  const uint32_t r2 = (uint32_t)__builtin_amdgcn_readlane((int)top, 32);
  const uint32_t r3 = (uint32_t)__builtin_amdgcn_readlane((int)top, 48);
  return max(max(r0, r1), max(r2, r3));
}

// Exponent e of a block's scale 2^e: the smallest, at least -126, with
// a <= 448 * 2^e = 1.75 * 2^(e + 8); 0 for a = 0.  A finite a gives e <= 120.
__device__ __forceinline__ int scale_exponent(uint32_t abits) {
  if (abits == 0u) return 0;
  const int e = (int)(abits >> 23) - 127 - 8 + ((abits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, -126);
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
    if ((fbits(x[e]) & 0x7FFFFFFFu) >= 0x7F800000u) w = (w & ~(0xFFu << (8 * e))) | (0x7Fu << (8 * e));
  }
  return w;
}

__device__ __forceinline__ uint32_t dither_word(uint32_t x) {
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  return x ^ (x >> 16);
}

template <int ET, bool FULL>
__device__ __forceinline__ void adamw_e4m3_block(const OptimTensor& t, const AdamArgs& a, const Rates& r,
                                                 uint32_t key, size_t block, size_t i) {
  const size_t n = t.n;
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  const f4 g = load_grad4<ET, FULL>(t.g, i, n);
  f4 p = load_f4<FULL>(t.p, i, n);
  const uint32_t mw = load_codes4_at<FULL>(mc, i, n), vw = load_codes4_at<FULL>(vc, i, n);
  f4 m = e4m3_unpack4(mw) * t.ms[block];
  f4 u = e4m3_unpack4(vw) * t.vs[block];
  f4 v = u * u;
  adamw4(a, r, g, p, m, v, u);
  store_f4<FULL>(t.p, i, n, p);
  if constexpr (ET != GB_DTYPE_F32) {
    if (t.copy != nullptr) store_copy4<ET, FULL>(t.copy, i, n, p);
  }
  const int me = scale_exponent(wave_absmax(m)), ue = scale_exponent(wave_absmax(u));
  const f4 mq = m * pow2(-me);
  f4 uq = u * pow2(-ue);
#pragma unroll
  for (int e = 0; e < 4; e++) uq[e] = u[e] > 0.0f ? fmaxf(uq[e], 0x1p-9f) : uq[e];  // a root above 0 keeps a code
  const uint32_t pair = (t.first_block * 128u) + (uint32_t)(i / 2);
  const uint32_t x0 = dither_word(pair * 0x9E3779B9u + key), x1 = dither_word((pair + 1) * 0x9E3779B9u + key);
  const uint32_t seed[4] = {x0, x0 << 16, x1, x1 << 16};
  store_codes4_at<FULL>(mc, i, n, mark_not_finite(m, dithered4(mq, seed)));
  store_codes4_at<FULL>(vc, i, n, mark_not_finite(u, dithered4(uq, seed)));
  if (threadIdx.x % kWave == 0) {
    t.ms[block] = pow2(me);
    t.vs[block] = pow2(ue);
  }
}

template <int ET>
__global__ __launch_bounds__(kThreads) void adamw_e4m3_kernel(const OptimTensor* tensors, const OptimChunk* chunks,
                                                              const gb_optim_control* control, AdamArgs a) {
  if (control->skip != 0) return;
  const OptimChunk c = chunks[blockIdx.x];
  const OptimTensor t = tensors[c.tensor];
  const Rates r = tensor_rates(control, t);
  const size_t first = (size_t)c.chunk * kOptimChunk, i = first + threadIdx.x * 4;
  // one block per wavefront: the last chunk's wavefronts beyond n leave whole
  const size_t block = first / kBlock + threadIdx.x / kWave;
  if (block * kBlock >= t.n) return;
  if (first + kOptimChunk <= t.n) adamw_e4m3_block<ET, true>(t, a, r, control->key, block, i);
  else adamw_e4m3_block<ET, false>(t, a, r, control->key, block, i);
}

StepArgs step_args(const OptimPlan& plan, double max_norm, double inv_scale) {
  return StepArgs{plan.beta1, plan.beta2, max_norm, inv_scale, plan.seed};
}

}  // namespace

hipError_t launch_optim_upload(OptimTensor* tensors, OptimChunk* chunks, uint32_t* counter, const OptimUpload& up,
                               hipStream_t stream) {
  (void)hipGetLastError();
  optim_upload_kernel<<<dim3(up.count > 0 ? up.count : 1, 8), kThreads, 0, stream>>>(tensors, chunks, counter, up);
  return hipGetLastError();
}

hipError_t launch_optim_begin(const OptimPlan& plan, gb_optim_control* control, double inv_scale,
                              hipStream_t stream) {
  (void)hipGetLastError();
  optim_begin_kernel<<<1, 1, 0, stream>>>(control, step_args(plan, 0.0, inv_scale));
  return hipGetLastError();
}

hipError_t launch_optim_begin_clip(const OptimPlan& plan, gb_optim_control* control, double max_norm,
                                   double inv_scale, hipStream_t stream) {
  const uint32_t count = plan.first[kOptimKinds];
  const uint32_t groups = count < 1 ? 1 : count < kNormGroups ? count : kNormGroups;
  (void)hipGetLastError();
  optim_norm_kernel<<<groups, kThreads, 0, stream>>>(plan.tensors, plan.chunks, count, plan.partials, plan.counter,
                                                     control, step_args(plan, max_norm, inv_scale));
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
    const uint32_t count = plan.first[k + 1] - plan.first[k];
    if (count == 0) continue;
    kernels[k]<<<count, kThreads, 0, stream>>>(plan.tensors, plan.chunks + plan.first[k], control, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gb
