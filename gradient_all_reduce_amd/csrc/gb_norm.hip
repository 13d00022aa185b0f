// gb_norm.hip — layer norm over the rows of a 2-D array, forward and backward
// with the weight's and the bias' gradients.  The formulas stand in
// include/gbreduce.h.
#include "gb_rows.h"

namespace gb {
namespace {

// ---------------------------------------------------------------------------
// A team of lanes per row.  L lanes of W wavefronts (W = 1 where L < 64) hold
// a row in registers, K vectors of 16 bytes in each lane: vector k of lane t
// begins at column (k * L * W + t) * V, so a load instruction covers one
// contiguous run.  Each value is read from memory once; mean and variance are
// two passes over registers, so the variance is a sum of squared deviations
// and loses nothing to cancellation.
// ---------------------------------------------------------------------------
template <int ET, int L, int W, int K>
struct Team {
  static constexpr int kV = Type<ET>::kVec, kLanes = L * W, kCols = kLanes * K * kV;
};

// Sum over the team: over the lanes of a wavefront in registers, over
// wavefronts through LDS.  part: W floats of this team.  One barrier if W > 1.
template <int L, int W>
__device__ __forceinline__ float team_sum(float v, float* part) {
  v = lanes_sum<L>(v);
  if constexpr (W > 1) {
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave % W] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; w++) v += part[w];
  }
  return v;
}

template <int ET, int L, int W, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a) {
  using T = Team<ET, L, W, K>;
  constexpr int V = T::kV, kTeams = THREADS / T::kLanes;
  __shared__ float part[W > 1 ? 2 : 1][W > 1 ? kTeams * W : 1];
  const uint32_t lane = threadIdx.x % T::kLanes, team = threadIdx.x / T::kLanes;
  float* const sum_part = &part[0][W > 1 ? team * W : 0];
  float* const var_part = &part[W > 1 ? 1 : 0][W > 1 ? team * W : 0];
  const float n = (float)a.cols;

  float w[K][V], b[K][V];
  auto param = [&](float (&to)[K][V], const void* p, float none) {
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t col = (k * T::kLanes + lane) * V;
#pragma unroll
      for (int e = 0; e < V; e++) to[k][e] = p != nullptr && col + e < a.cols ? load_any(p, a.param_dtype, col + e) : none;
    }
  };
  param(w, a.w, 1.0f);
  param(b, a.b, 0.0f);

  Raw<ET, V> x[K];
  auto load_row = [&](size_t r) {
    const size_t at = r * a.x.stride;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t col = (k * T::kLanes + lane) * V;
      x[k] = r < a.rows ? load_raw<ET, V, true>(a.x.p, at + col, left_of(col, a.cols)) : zero_raw<ET, V>();
    }
  };
  const size_t step = (size_t)gridDim.x * kTeams;
  // the same number of rounds in every team of the workgroup: they meet at barriers
  const size_t first = (size_t)blockIdx.x * kTeams;
  load_row(first + team);
  for (size_t base = first; base < a.rows; base += step) {
    const size_t r = base + team;
    float v[K][V], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) {
#pragma unroll
      for (int e = 0; e < V; e++) {
        v[k][e] = raw_value<ET, V>(x[k], e);  // zeros beyond the row
        sum += v[k][e];
      }
    }
    if (base + step < a.rows) load_row(r + step);
    const float mean = team_sum<L, W>(sum, sum_part) / n;
    float square = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t left = left_of((k * T::kLanes + lane) * V, a.cols);
#pragma unroll
      for (int e = 0; e < V; e++) {
        v[k][e] = left >= V || e < (int)left ? v[k][e] - mean : 0.0f;
        square = fmaf(v[k][e], v[k][e], square);
      }
    }
    const float rstd = 1.0f / sqrtf(team_sum<L, W>(square, var_part) / n + a.eps);
    if (r < a.rows) {
      const size_t at = r * a.y.stride;
#pragma unroll
      for (int k = 0; k < K; k++) {
        const uint32_t col = (k * T::kLanes + lane) * V;
        float y[V];
#pragma unroll
        for (int e = 0; e < V; e++) y[e] = canon(fmaf(v[k][e] * rstd, w[k][e], b[k][e]));
        store_vals<ET, V, true>(a.y.p, at + col, left_of(col, a.cols), y);
      }
      if (lane == 0) {
        if (a.mean != nullptr) a.mean[r] = canon(mean);
        if (a.rstd != nullptr) a.rstd[r] = canon(rstd);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  A workgroup walks over rows with its teams side by side; each
// lane keeps its columns' sums of dy * h and dy in registers from the first
// row to the last, so the weight's gradient costs no traffic until the end,
// when the workgroup leaves one row of partial sums for each.
// ---------------------------------------------------------------------------
template <int ET, int L, int W, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(NormGradArgs a) {
  using T = Team<ET, L, W, K>;
  constexpr int V = T::kV, kTeams = THREADS / T::kLanes;
  __shared__ float part[2][2][W > 1 ? kTeams * W : 1];
  const uint32_t lane = threadIdx.x % T::kLanes, team = threadIdx.x / T::kLanes;
  const float inv_n = 1.0f / (float)a.cols;

  float w[K][V], dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; k++) {
    const uint32_t col = (k * T::kLanes + lane) * V;
#pragma unroll
    for (int e = 0; e < V; e++) {
      w[k][e] = a.w != nullptr && col + e < a.cols ? load_any(a.w, a.param_dtype, col + e) : 1.0f;
      dw[k][e] = db[k][e] = 0.0f;
    }
  }
  Raw<ET, V> x[K], dy[K];
  float mean, rstd;
  auto load_row = [&](size_t r) {
    const bool in = r < a.rows;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t col = (k * T::kLanes + lane) * V;
      x[k] = in ? load_raw<ET, V, true>(a.x.p, r * a.x.stride + col, left_of(col, a.cols)) : zero_raw<ET, V>();
      dy[k] = in ? load_raw<ET, V, true>(a.dy.p, r * a.dy.stride + col, left_of(col, a.cols)) : zero_raw<ET, V>();
    }
    mean = in ? a.mean[r] : 0.0f;
    rstd = in ? a.rstd[r] : 0.0f;
  };
  const size_t step = (size_t)gridDim.x * kTeams, first = (size_t)blockIdx.x * kTeams;
  load_row(first + team);
  int parity = 0;
  for (size_t base = first; base < a.rows; base += step, parity ^= 1) {
    const size_t r = base + team;
    float h[K][V], g[K][V], c1 = 0.0f, c2 = 0.0f;
    const float m = mean, s = rstd;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t left = left_of((k * T::kLanes + lane) * V, a.cols);
#pragma unroll
      for (int e = 0; e < V; e++) {
        const float d = raw_value<ET, V>(dy[k], e);
        // beyond the row d is 0 but the mean need not be, and 0 * Inf is NaN
        h[k][e] = left >= V || e < (int)left ? (raw_value<ET, V>(x[k], e) - m) * s : 0.0f;
        g[k][e] = d * w[k][e];
        c1 += g[k][e];
        c2 = fmaf(g[k][e], h[k][e], c2);
        dw[k][e] = fmaf(d, h[k][e], dw[k][e]);
        db[k][e] += d;
      }
    }
    if (base + step < a.rows) load_row(r + step);
    if (a.dx.p == nullptr) continue;
    c1 = lanes_sum<L>(c1);
    c2 = lanes_sum<L>(c2);
    if constexpr (W > 1) {
      float* const p1 = &part[parity][0][team * W];
      float* const p2 = &part[parity][1][team * W];
      if (threadIdx.x % kWave == 0) {
        p1[threadIdx.x / kWave % W] = c1;
        p2[threadIdx.x / kWave % W] = c2;
      }
      // one barrier a row: the next row writes the other half, and the row
      // after it comes past that row's barrier, which every reader of this
      // half has reached
      __syncthreads();
      c1 = p1[0], c2 = p2[0];
#pragma unroll
      for (int i = 1; i < W; i++) c1 += p1[i], c2 += p2[i];
    }
    c1 *= inv_n * s;
    c2 *= inv_n * s;
    if (r < a.rows) {
      const size_t at = r * a.dx.stride;
#pragma unroll
      for (int k = 0; k < K; k++) {
        const uint32_t col = (k * T::kLanes + lane) * V;
        float dx[V];
#pragma unroll
        for (int e = 0; e < V; e++) dx[e] = canon(fmaf(-h[k][e], c2, fmaf(g[k][e], s, -c1)));
        store_vals<ET, V, true>(a.dx.p, at + col, left_of(col, a.cols), dx);
      }
    }
  }
  if (a.dw == nullptr && a.db == nullptr) return;

  // the teams' sums, joined in the order of the teams
  if constexpr (L < kWave) {
#pragma unroll
    for (int k = 0; k < K; k++) {
#pragma unroll
      for (int e = 0; e < V; e++) {
#pragma unroll
        for (int d = L; d < kWave; d *= 2) {
          dw[k][e] += __shfl_xor(dw[k][e], d);
          db[k][e] += __shfl_xor(db[k][e], d);
        }
      }
    }
  }
  const size_t stride = a.partial_stride;
  float* const out = a.partials + (size_t)blockIdx.x * 2 * stride;
  constexpr int kJoin = L < kWave ? THREADS / kWave : kTeams;  // sums left to join
  if constexpr (kJoin > 1) {
    __shared__ float joined[2][T::kCols];
    const uint32_t mine = L < kWave ? threadIdx.x / kWave : team;
    for (uint32_t j = 0; j < kJoin; j++) {
      if (mine == j && (L == kWave || threadIdx.x % kWave < L)) {
#pragma unroll
        for (int k = 0; k < K; k++) {
          const uint32_t col = (k * T::kLanes + lane) * V;
#pragma unroll
          for (int e = 0; e < V; e++) {
            joined[0][col + e] = j == 0 ? dw[k][e] : joined[0][col + e] + dw[k][e];
            joined[1][col + e] = j == 0 ? db[k][e] : joined[1][col + e] + db[k][e];
          }
        }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < a.cols; c += THREADS) {
      if (a.dw != nullptr) out[c] = joined[0][c];
      if (a.db != nullptr) out[stride + c] = joined[1][c];
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t col = (k * T::kLanes + lane) * V, left = left_of(col, a.cols);
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const uint32_t l = left > (uint32_t)j ? left - j : 0u;
        const float pw[4] = {dw[k][j], dw[k][j + 1], dw[k][j + 2], dw[k][j + 3]};
        const float pb[4] = {db[k][j], db[k][j + 1], db[k][j + 2], db[k][j + 3]};
        if (a.dw != nullptr) store_vals<GB_DTYPE_F32, 4, false>(out, col + j, l, pw);
        if (a.db != nullptr) store_vals<GB_DTYPE_F32, 4, false>(out, stride + col + j, l, pb);
      }
    }
  }
}

// dw and db from the workgroups' partial sums: 4 columns a lane, 16 lanes side
// by side, and 16 (kSlices) of those take every 16th partial each; their sums
// are joined in order.  blockIdx.y: dw or db.
constexpr int kJoinLanes = 16, kSlices = 16;
__global__ __launch_bounds__(kJoinLanes* kSlices) void norm_join_kernel(NormGradArgs a, uint32_t groups) {
  __shared__ f4 slice[kSlices][kJoinLanes];
  void* const out = blockIdx.y == 0 ? a.dw : a.db;
  if (out == nullptr) return;
  const uint32_t l = threadIdx.x % kJoinLanes, s = threadIdx.x / kJoinLanes;
  const uint32_t col = (blockIdx.x * kJoinLanes + l) * 4;
  const size_t stride = a.partial_stride;
  const float* const p = a.partials + blockIdx.y * stride + col;
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < a.cols) {
#pragma unroll 8
    for (uint32_t g = s; g < groups; g += kSlices) v += *(const f4*)(p + (size_t)g * 2 * stride);
  }
  slice[s][l] = v;
  __syncthreads();
  if (s != 0 || col >= a.cols) return;
#pragma unroll
  for (int i = 1; i < kSlices; i++) v += slice[i][l];
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if (col + e >= a.cols) break;
    float t = v[e];
    if (a.accumulate) t = load_any(out, a.grad_dtype, col + e) + t;
    t = canon(t);
    if (a.grad_dtype == GB_DTYPE_F32) store_one<GB_DTYPE_F32>(out, col + e, t);
    else if (a.grad_dtype == GB_DTYPE_F16) store_one<GB_DTYPE_F16>(out, col + e, t);
    else store_one<GB_DTYPE_BF16>(out, col + e, t);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int ET, int L, int W, int K>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int kThreads = W > 4 ? W * kWave : 256;
  constexpr size_t kTeams = kThreads / (L * W);
  size_t grid = (a.rows + kTeams - 1) / kTeams;
  if (grid > 2048) grid = 2048;
  norm_kernel<ET, L, W, K, kThreads><<<dim3((unsigned)grid), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}
template <int ET>
hipError_t pick_norm(const NormArgs& a, hipStream_t stream) {
  const uint32_t v = (a.cols + Type<ET>::kVec - 1) / Type<ET>::kVec;
  if (v <= 8) return run_norm<ET, 8, 1, 1>(a, stream);
  if (v <= 16) return run_norm<ET, 16, 1, 1>(a, stream);
  if (v <= 32) return run_norm<ET, 32, 1, 1>(a, stream);
  if (v <= 64) return run_norm<ET, 64, 1, 1>(a, stream);
  if (v <= 128) return run_norm<ET, 64, 1, 2>(a, stream);
  if (v <= 256) return run_norm<ET, 64, 2, 2>(a, stream);
  if (v <= 512) return run_norm<ET, 64, 4, 2>(a, stream);
  if (v <= 1024) return run_norm<ET, 64, 4, 4>(a, stream);
  if (v <= 2048) return run_norm<ET, 64, 8, 4>(a, stream);
  if constexpr (ET == GB_DTYPE_F32) {
    if (v > 4096) return run_norm<ET, 64, 16, 8>(a, stream);
  }
  return run_norm<ET, 64, 16, 4>(a, stream);
}

template <int ET, int L, int W, int K>
struct NormGrad {
  static constexpr int kThreads = W > 4 ? W * kWave : 256;
  static constexpr size_t kTeams = kThreads / (L * W);
  static uint32_t groups(size_t rows, size_t) {
    const size_t g = (rows + kTeams - 1) / kTeams;
    return (uint32_t)(g < 512 ? g : 512);
  }
  static hipError_t run(const NormGradArgs& a, hipStream_t stream) {
    const uint32_t g = groups(a.rows, a.cols);
    if (g > 0) norm_grad_kernel<ET, L, W, K, kThreads><<<dim3(g), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
  }
};
// Calls f with the NormGrad of a row of cols values.
template <int ET, class F>
auto with_norm_grad(size_t cols, F&& f) {
  const size_t v = (cols + Type<ET>::kVec - 1) / Type<ET>::kVec;
  if (v <= 8) return f(NormGrad<ET, 8, 1, 1>());
  if (v <= 16) return f(NormGrad<ET, 16, 1, 1>());
  if (v <= 32) return f(NormGrad<ET, 32, 1, 1>());
  if (v <= 64) return f(NormGrad<ET, 64, 1, 1>());
  if (v <= 128) return f(NormGrad<ET, 64, 1, 2>());
  if (v <= 256) return f(NormGrad<ET, 64, 2, 2>());
  if (v <= 512) return f(NormGrad<ET, 64, 4, 2>());
  if (v <= 1024) return f(NormGrad<ET, 64, 4, 4>());
  if (v <= 2048) return f(NormGrad<ET, 64, 8, 4>());
  if constexpr (ET == GB_DTYPE_F32) {
    if (v > 4096) return f(NormGrad<ET, 64, 8, 16>());
  }
  return f(NormGrad<ET, 64, 8, 8>());
}
template <class F>
auto with_norm_grad(int dtype, size_t cols, F&& f) {
  if (dtype == GB_DTYPE_F32) return with_norm_grad<GB_DTYPE_F32>(cols, f);
  if (dtype == GB_DTYPE_F16) return with_norm_grad<GB_DTYPE_F16>(cols, f);
  return with_norm_grad<GB_DTYPE_BF16>(cols, f);
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream) {
  if (a.dtype == GB_DTYPE_F32) return pick_norm<GB_DTYPE_F32>(a, stream);
  if (a.dtype == GB_DTYPE_F16) return pick_norm<GB_DTYPE_F16>(a, stream);
  return pick_norm<GB_DTYPE_BF16>(a, stream);
}

uint32_t norm_grad_groups(size_t rows, size_t cols, int dtype) {
  return with_norm_grad(dtype, cols, [&](auto g) { return g.groups(rows, cols); });
}

hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t stream) {
  hipError_t e = with_norm_grad(a.dtype, a.cols, [&](auto g) { return g.run(a, stream); });
  if (e != hipSuccess || (a.dw == nullptr && a.db == nullptr)) return e;
  const uint32_t blocks = (a.cols + 4 * kJoinLanes - 1) / (4 * kJoinLanes);
  norm_join_kernel<<<dim3(blocks, 2), dim3(kJoinLanes * kSlices), 0, stream>>>(
      a, norm_grad_groups(a.rows, a.cols, a.dtype));
  return hipGetLastError();
}

}  // namespace gb
