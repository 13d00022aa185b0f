// gb_norm.hip — layer norm over the rows of a 2-D array, forward and backward
// with the weight's and the bias' gradients.  The formulas stand in
// include/gbreduce.h.
//
// Both passes stream HBM (8 and 16 operations a value, no contraction, so no
// MFMA): forward each value is read and written once, backward x and dy are
// read and dx written once, and the sums over the rows stay in registers.
// Measured on MI355X, algorithmic bytes over kernel time, where the best plain
// copy moves 6.65 TB/s: forward over 16,384 x 8192 bfloat16 values 89.7 us (6.0
// TB/s), over 65,536 x 128 float16 out of wider rows 9.1 us (3.7); backward over
// 16,384 x 4096 bfloat16 71.0 us and 4.8 for the join (5.3 TB/s together), over
// 5003 x 12,289 float16 97.5 and 5.2 us (3.6: rows of odd length start off 16
// bytes and leave a quarter of the lanes idle), over 512 x 771 float32 6.2 and
// 3.9 us.  Counted traffic over algorithmic bytes: 1.003 forward (16,384 x 8192),
// 1.02 backward (16,384 x 4096: the partial sums), 1.07 over 5003 x 12,289.
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
//
// A vector that would pass the row's end is moved back to end with the row:
// every load and store is a whole vector without a branch, the values it
// shares with its neighbour (skip of them, all V in a lane beyond the row)
// count in the neighbour's sums alone, and both store the same bits.  Rows
// shorter than a vector (SHORT) are read value by value.
// ---------------------------------------------------------------------------
template <int ET, int L, int W, int K, bool SHORT>
struct Team {
  static constexpr int V = Type<ET>::kVec, kLanes = L * W, kCols = kLanes * K * V;
  uint32_t lane, at[K], skip[K], cols;
  uint32_t last;  // of the wavefront's lanes in the team

  __device__ __forceinline__ explicit Team(uint32_t n) : lane(threadIdx.x % kLanes), cols(n) {
    last = L < kWave ? L - 1 : __builtin_amdgcn_readfirstlane(lane / kWave) * kWave + kWave - 1;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const uint32_t col = (k * kLanes + lane) * V;
      at[k] = SHORT ? 0 : col + V <= n ? col : n - V;
      skip[k] = SHORT ? (lane == 0 ? V - n : V) : col - at[k] < V ? col - at[k] : V;
    }
  }
  // Whether vector k of some lane of the wavefront is not its own throughout.
  __device__ __forceinline__ bool ragged(int k) const { return SHORT || (k * kLanes + last + 1) * V > cols; }
  __device__ __forceinline__ bool mine(int k, int e) const {
    return SHORT ? lane == 0 && e < (int)cols : e >= (int)skip[k];
  }
  // The lane's offset, made anew for each access: hoisted out of a loop, its
  // widening would take two registers and an addition of 64 bits an access,
  // where the instruction adds 32 bits to a scalar by itself.
  __device__ __forceinline__ uint32_t offset(int k) {
    asm volatile("" : "+v"(at[k]));
    return at[k];
  }
  __device__ __forceinline__ Raw<ET, V> load(const void* row, int k) {
    if constexpr (SHORT) return load_raw<ET, V, true>(row, 0u, lane == 0 ? cols : 0u);
    else return load_full<ET, V, true>(row, offset(k));
  }
  __device__ __forceinline__ void store(void* row, int k, const float (&v)[V]) {
    if constexpr (SHORT) store_vals<ET, V, true>(row, 0u, lane == 0 ? cols : 0u, v);
    else if (!ragged(k) || skip[k] < V) store_vals<ET, V, true>(row, offset(k), V, v);
  }
  template <int PT>
  __device__ __forceinline__ void param_of(float (&to)[V], const void* p, int k) const {
    constexpr int P = Type<PT>::kVec < V ? Type<PT>::kVec : V;
#pragma unroll
    for (int j = 0; j < V; j += P) {
      Raw<PT, P> r;
      if constexpr (SHORT) r = load_raw<PT, P, false>(p, (uint32_t)j, lane == 0 && (int)cols > j ? cols - j : 0u);
      else r = load_full<PT, P, false>(p, at[k] + j);
#pragma unroll
      for (int e = 0; e < P; e++) to[j + e] = raw_value<PT, P>(r, e);
    }
  }
  // A parameter's values at the lane's columns; none where there is no array.
  __device__ __forceinline__ void param(float (&to)[K][V], const void* p, int dtype, float none) const {
    if (p == nullptr) {
#pragma unroll
      for (int k = 0; k < K; k++) {
#pragma unroll
        for (int e = 0; e < V; e++) to[k][e] = none;
      }
    } else if (dtype == GB_DTYPE_F32) {
#pragma unroll
      for (int k = 0; k < K; k++) param_of<GB_DTYPE_F32>(to[k], p, k);
    } else if (dtype == GB_DTYPE_F16) {
#pragma unroll
      for (int k = 0; k < K; k++) param_of<GB_DTYPE_F16>(to[k], p, k);
    } else {
#pragma unroll
      for (int k = 0; k < K; k++) param_of<GB_DTYPE_BF16>(to[k], p, k);
    }
  }
};

// Row r of an array.
template <int ET>
__device__ __forceinline__ char* row_at(const Rows& a, size_t r) {
  return static_cast<char*>(a.p) + r * a.stride * Type<ET>::kSize;
}
// The team's number in the workgroup: a scalar where a wavefront belongs to
// one team, and so are its rows' addresses.
template <int L, int LANES>
__device__ __forceinline__ uint32_t team_number() {
  const uint32_t t = threadIdx.x / LANES;
  return L < kWave ? t : __builtin_amdgcn_readfirstlane(t);
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

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

template <int ET, int L, int W, int K, int THREADS, bool SHORT>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a) {
  using T = Team<ET, L, W, K, SHORT>;
  constexpr int V = T::V, kTeams = THREADS / T::kLanes;
  __shared__ float part[W > 1 ? 2 : 1][W > 1 ? kTeams * W : 1];
  T t(a.cols);
  const uint32_t team = team_number<L, T::kLanes>();
  float* const sum_part = &part[0][W > 1 ? team * W : 0];
  float* const var_part = &part[W > 1 ? 1 : 0][W > 1 ? team * W : 0];
  const float inv_n = 1.0f / (float)a.cols;

  Raw<ET, V> x[K];
  auto load_row = [&](size_t r) {
    const void* const row = row_at<ET>(a.x, r < a.rows ? r : a.rows - 1);
#pragma unroll
    for (int k = 0; k < K; k++) x[k] = t.load(row, k);
  };
  const size_t step = (size_t)gridDim.x * kTeams, first = (size_t)blockIdx.x * kTeams;
  load_row(first + team);
  float w[K][V], b[K][V];
  t.param(w, a.w, a.param_dtype, 1.0f);
  t.param(b, a.b, a.param_dtype, 0.0f);
  bool plain = true;  // the lane's parameters are finite
#pragma unroll
  for (int k = 0; k < K; k++) {
#pragma unroll
    for (int e = 0; e < V; e++) plain = plain && finite(w[k][e]) && finite(b[k][e]);
  }
  // the same number of rounds in every team of the workgroup: they meet at barriers
  for (size_t base = first; base < a.rows; base += step) {
    const size_t r = base + team;
    float v[K][V], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) {
#pragma unroll
      for (int e = 0; e < V; e++) v[k][e] = raw_value<ET, V>(x[k], e);
      if (t.ragged(k)) {
#pragma unroll
        for (int e = 0; e < V; e++) sum += t.mine(k, e) ? v[k][e] : 0.0f;
      } else {
#pragma unroll
        for (int e = 0; e < V; e++) sum += v[k][e];
      }
    }
    if (base + step < a.rows) load_row(r + step);
    const float mean = team_sum<L, W>(sum, sum_part) * inv_n;
    float square = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) {
#pragma unroll
      for (int e = 0; e < V; e++) v[k][e] -= mean;
      if (t.ragged(k)) {
#pragma unroll
        for (int e = 0; e < V; e++) square = t.mine(k, e) ? fmaf(v[k][e], v[k][e], square) : square;
      } else {
#pragma unroll
        for (int e = 0; e < V; e++) square = fmaf(v[k][e], v[k][e], square);
      }
    }
    const float rstd = 1.0f / sqrtf(team_sum<L, W>(square, var_part) * inv_n + a.eps);
    if (r < a.rows) {
      void* const row = row_at<ET>(a.y, r);
      // With mean, weight and bias finite and rstd finite and above 0 no value
      // is NaN: rstd is above 0 only if the sum of the squares is finite, so no
      // deviation is infinite (one of a row of finite values may be: of 3.4e38
      // and twice -3.4e38 the mean is -1.1e38).  A deviation times rstd is then
      // at most the root of cols, and a fused product and sum of finite numbers
      // may overflow but has a sign.
      if (__all(plain && finite(mean) && finite(rstd) && rstd > 0.0f)) {
#pragma unroll
        for (int k = 0; k < K; k++) {
          float y[V];
#pragma unroll
          for (int e = 0; e < V; e++) y[e] = fmaf(v[k][e] * rstd, w[k][e], b[k][e]);
          t.store(row, k, y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; k++) {
          float y[V];
#pragma unroll
          for (int e = 0; e < V; e++) y[e] = canon(fmaf(v[k][e] * rstd, w[k][e], b[k][e]));
          t.store(row, k, y);
        }
      }
      if (t.lane == 0) {
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
template <int ET, int L, int W, int K, int THREADS, bool SHORT>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(NormGradArgs a) {
  using T = Team<ET, L, W, K, SHORT>;
  constexpr int V = T::V, kTeams = THREADS / T::kLanes;
  // h and g stay in registers between the two passes over a row, or are
  // worked out again from the row's values
  constexpr bool kKeep = K * V <= 8;
  // rows read ahead, as many as the registers hold
  constexpr int D = K == 1 ? 2 : K == 2 ? 1 : 0;
  // a lane's weights lie in its registers, or in LDS
  constexpr bool kWeightsInLds = K * V >= 16;
  __shared__ f4 lds_w[kWeightsInLds ? K * V / 4 : 1][kWeightsInLds ? THREADS : 1];
  __shared__ float part[2][2][W > 1 ? kTeams * W : 1];
  T t(a.cols);
  const uint32_t team = team_number<L, T::kLanes>();
  const float inv_n = 1.0f / (float)a.cols;

  struct Row {
    Raw<ET, V> x[K], dy[K];
    float mean, rstd;
  };
  auto load_row = [&](Row& row, size_t r) {
    r = r < a.rows ? r : a.rows - 1;
    const void *const x_row = row_at<ET>(a.x, r), *const dy_row = row_at<ET>(a.dy, r);
#pragma unroll
    for (int k = 0; k < K; k++) {
      row.x[k] = t.load(x_row, k);
      row.dy[k] = t.load(dy_row, k);
    }
    row.mean = a.mean[r];
    row.rstd = a.rstd[r];
  };
  Row ahead[D > 0 ? D : 1];
  const size_t step = (size_t)gridDim.x * kTeams, first = (size_t)blockIdx.x * kTeams;
#pragma unroll
  for (int j = 0; j < D; j++) load_row(ahead[j], first + j * step + team);
  float w[K][V], dw[K][V], db[K][V];
  t.param(w, a.w, a.param_dtype, 1.0f);
#pragma unroll
  for (int k = 0; k < K; k++) {
#pragma unroll
    for (int e = 0; e < V; e++) {
      if constexpr (kWeightsInLds) lds_w[(k * V + e) / 4][threadIdx.x][e % 4] = w[k][e];  // read by this lane alone
      dw[k][e] = db[k][e] = 0.0f;
    }
  }
  int parity = 0;
  auto round = [&](Row& row, size_t base) {
    const size_t r = base + team;
    if (D == 0) load_row(row, r);
    parity ^= 1;
    if (base + kTeams > a.rows && r >= a.rows) {  // a team without a row adds nothing
#pragma unroll
      for (int k = 0; k < K; k++) row.x[k] = row.dy[k] = zero_raw<ET, V>();
      row.mean = row.rstd = 0.0f;
    }
    float h[kKeep ? K : 1][V], g[kKeep ? K : 1][V], c1 = 0.0f, c2 = 0.0f;
    const float m = row.mean, s = row.rstd;
    Row now;
#pragma unroll
    for (int k = 0; k < K; k++) {
      now.x[k] = row.x[k];
      now.dy[k] = row.dy[k];
    }
    auto terms = [&](int k, float (&hk)[V], float (&gk)[V]) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        f4 wj = {w[k][j], w[k][j + 1], w[k][j + 2], w[k][j + 3]};
        if constexpr (kWeightsInLds) wj = lds_w[(k * V + j) / 4][threadIdx.x];
#pragma unroll
        for (int e = j; e < j + 4; e++) {
          hk[e] = (raw_value<ET, V>(now.x[k], e) - m) * s;
          gk[e] = raw_value<ET, V>(now.dy[k], e) * wj[e - j];
        }
      }
    };
#pragma unroll
    for (int k = 0; k < K; k++) {
      float(&hk)[V] = h[kKeep ? k : 0];
      float(&gk)[V] = g[kKeep ? k : 0];
      if constexpr (!kKeep) __builtin_amdgcn_sched_barrier(0);
      terms(k, hk, gk);
#pragma unroll
      for (int e = 0; e < V; e++) {
        const float d = raw_value<ET, V>(now.dy[k], e);
        dw[k][e] = fmaf(d, hk[e], dw[k][e]);
        db[k][e] += d;
      }
      if (t.ragged(k)) {
#pragma unroll
        for (int e = 0; e < V; e++) {
          c1 += t.mine(k, e) ? gk[e] : 0.0f;
          c2 = t.mine(k, e) ? fmaf(gk[e], hk[e], c2) : c2;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; e++) {
          c1 += gk[e];
          c2 = fmaf(gk[e], hk[e], c2);
        }
      }
    }
    if (D > 0 && base + D * step < a.rows) load_row(row, r + D * step);
    if (a.dx.p == nullptr) return;
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
    if constexpr (!kKeep) {
      // or the compiler keeps h and g after all, and spills them
#pragma unroll
      for (int k = 0; k < K; k++) {
#pragma unroll
        for (int j = 0; j < 4; j++) asm volatile("" : "+v"(now.x[k].w[j]), "+v"(now.dy[k].w[j]));
      }
    }
    if (r < a.rows) {
      void* const to = row_at<ET>(a.dx, r);
      // With both sums and rstd finite so are all g and h (an infinite one
      // would show in a sum), and fused products and sums of finite numbers
      // may overflow but have a sign: no value is NaN.
      const bool plain = __all(finite(c1) && finite(c2) && finite(s));
#pragma unroll
      for (int k = 0; k < K; k++) {
        float(&hk)[V] = h[kKeep ? k : 0];
        float(&gk)[V] = g[kKeep ? k : 0];
        if constexpr (!kKeep) {
          __builtin_amdgcn_sched_barrier(0);
          terms(k, hk, gk);
        }
        float dx[V];
#pragma unroll
        for (int e = 0; e < V; e++) dx[e] = fmaf(-hk[e], c2, fmaf(gk[e], s, -c1));
        if (!plain) {
#pragma unroll
          for (int e = 0; e < V; e++) dx[e] = canon(dx[e]);
        }
        t.store(to, k, dx);
      }
    }
  };
  for (size_t base = first; base < a.rows; base += (D > 0 ? D : 1) * step) {
#pragma unroll
    for (int j = 0; j < (D > 0 ? D : 1); j++) {
      if (base + j * step < a.rows) round(ahead[j], base + j * step);
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
  float* const out = a.partials + (size_t)blockIdx.x * 2 * a.partial_stride;
  constexpr int kJoin = L < kWave ? THREADS / kWave : kTeams;  // sums left to join
  if constexpr (kJoin > 1 || SHORT) {
    __shared__ float joined[2][T::kCols];
    const uint32_t mine = L < kWave ? threadIdx.x / kWave : team;
    for (uint32_t j = 0; j < kJoin; j++) {
      if (mine == j && (L == kWave || threadIdx.x % kWave < L)) {
#pragma unroll
        for (int k = 0; k < K; k++) {
#pragma unroll
          for (int e = 0; e < V; e++) {
            if (!t.mine(k, e)) continue;
            const uint32_t c = t.at[k] + e;
            joined[0][c] = j == 0 ? dw[k][e] : joined[0][c] + dw[k][e];
            joined[1][c] = j == 0 ? db[k][e] : joined[1][c] + db[k][e];
          }
        }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < a.cols; c += THREADS) {
      if (a.dw != nullptr) out[c] = joined[0][c];
      if (a.db != nullptr) out[a.partial_stride + c] = joined[1][c];
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; k++) {
      if (t.skip[k] >= V) continue;
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float pw[4] = {dw[k][j], dw[k][j + 1], dw[k][j + 2], dw[k][j + 3]};
        const float pb[4] = {db[k][j], db[k][j + 1], db[k][j + 2], db[k][j + 3]};
        if (a.dw != nullptr) store_vals<GB_DTYPE_F32, 4, false>(out, t.at[k] + j, 4, pw);
        if (a.db != nullptr) store_vals<GB_DTYPE_F32, 4, false>(out, a.partial_stride + t.at[k] + j, 4, pb);
      }
    }
  }
}

// dw and db from the workgroups' partial sums: 4 columns a lane, 16 lanes side
// by side, and 64 (kSlices) of those take every 64th partial each; their sums
// are joined in order, by eights.  blockIdx.y: dw or db.
constexpr int kJoinLanes = 16, kSlices = 64;
__global__ __launch_bounds__(kJoinLanes* kSlices) void norm_join_kernel(NormGradArgs a, uint32_t groups) {
  __shared__ f4 slice[kSlices][kJoinLanes];
  void* const out = blockIdx.y == 0 ? a.dw : a.db;
  if (out == nullptr) return;
  const uint32_t l = threadIdx.x % kJoinLanes, s = threadIdx.x / kJoinLanes;
  const uint32_t col = (blockIdx.x * kJoinLanes + l) * 4;
  const float* const p = a.partials + blockIdx.y * a.partial_stride + col;
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < a.cols) {
    for (uint32_t first = s; first < groups; first += 4 * kSlices) {
      f4 x[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; i++) {
        const uint32_t g = first + i * kSlices;
        x[i] = *(const f4*)(p + (size_t)(g < groups ? g : s) * 2 * a.partial_stride);
      }
#pragma unroll
      for (uint32_t i = 0; i < 4; i++) {
        if (first + i * kSlices < groups) v += x[i];
      }
    }
  }
  slice[s][l] = v;
  __syncthreads();
  if (s % 8 == 0) {
#pragma unroll
    for (int i = 1; i < 8; i++) v += slice[s + i][l];
    slice[s][l] = v;
  }
  __syncthreads();
  if (s != 0 || col >= a.cols) return;
#pragma unroll
  for (int i = 8; i < kSlices; i += 8) v += slice[i][l];
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
// Forward a workgroup is 512 lanes from 1025 columns of 2 bytes on (513 of 4),
// and 512 workgroups walk over the rows, two to a CU, with the parameters in
// registers and the next row on its way; beyond 8192 columns (4096 of 4 bytes)
// 256 workgroups of 1024 lanes.  16,384 x 8192 bfloat16: 512 workgroups 88.7 us,
// 1024 96.9, 4096 92.5, one row each 121.  Eight wavefronts to a row rather than four (91.5 us)
// or sixteen (90.8); over 4096 columns 46.5 us in eight, 47.4 in four, 52 in
// one.  Up to 1024 columns 2048 workgroups of 256 lanes: 14.7 us over 16,384 x
// 1024, 19.5 with 512 workgroups.  Two rows ahead instead of one: 17.5 there,
// level over longer rows.
//
// Beyond 16,384 columns a lane holds 32 columns, and its parameters, its row and
// the next one no longer fit 128 registers: 120 (bfloat16) to 217 (float32)
// spill.  8192 x 32,768 takes 230 us in bfloat16, 321 in float16 (161 at the
// copy's rate) and 490 in float32 (323).
template <int ET, int L, int W, int K, int THREADS, bool SHORT = false>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
  constexpr size_t kTeams = THREADS / (L * W), kMost = 512 * 512 / THREADS * (W > 2 ? 1 : 2);
  size_t grid = (a.rows + kTeams - 1) / kTeams;
  if (grid > kMost) grid = kMost;
  norm_kernel<ET, L, W, K, THREADS, SHORT><<<dim3((unsigned)grid), dim3(THREADS), 0, stream>>>(a);
  return hipGetLastError();
}
template <int ET>
hipError_t pick_norm(const NormArgs& a, hipStream_t stream) {
  const uint32_t v = (a.cols + Type<ET>::kVec - 1) / Type<ET>::kVec;
  if (a.cols < Type<ET>::kVec) return run_norm<ET, 8, 1, 1, 256, true>(a, stream);
  if (v <= 8) return run_norm<ET, 8, 1, 1, 256>(a, stream);
  if (v <= 16) return run_norm<ET, 16, 1, 1, 256>(a, stream);
  if (v <= 32) return run_norm<ET, 32, 1, 1, 256>(a, stream);
  if (v <= 64) return run_norm<ET, 64, 1, 1, 256>(a, stream);
  if (v <= 128) return run_norm<ET, 64, 2, 1, 256>(a, stream);
  if (v <= 256) return run_norm<ET, 64, 4, 1, 512>(a, stream);
  if (v <= 512) return run_norm<ET, 64, 8, 1, 512>(a, stream);
  if (v <= 1024) return run_norm<ET, 64, 8, 2, 512>(a, stream);
  if (v <= 2048) return run_norm<ET, 64, 16, 2, 1024>(a, stream);
  if constexpr (ET == GB_DTYPE_F32) {
    if (v > 4096) return run_norm<ET, 64, 16, 8, 1024>(a, stream);
  }
  return run_norm<ET, 64, 16, 4, 1024>(a, stream);
}

// Backward 256 workgroups of 1024 lanes, one to a CU, as many teams in each as
// fit: half the partial sums of 512 workgroups of 512 lanes.  16,384 rows of
// bfloat16, both kernels: 4096 columns 74.9 against 77.2 us, 8192 142 against
// 147, 2048 43.2 against 46.6.  Two rows ahead rather than one: 75.7 against
// 79.1 us over 4096 columns.  A lane holds 8 columns of 2 bytes where 16
// wavefronts suffice: with 16 columns h and g no longer fit beside the sums and
// spill (5003 x 12,289 float16 255 us), so they are worked out again from the row
// and the weights lie in LDS (103 us), which leaves 2 or 3 registers to spill.
// Beyond 16,384 columns the sums alone take half the registers and 86 to 152
// spill: 8192 x 32,768 takes 1.1 ms in 2 bytes a value, 2.1 in 4.
template <int ET, int L, int W, int K, int THREADS, bool SHORT = false>
struct NormGrad {
  static constexpr size_t kTeams = THREADS / (L * W), kMost = 256 * 1024 / THREADS;
  static uint32_t groups(size_t rows, size_t) {
    const size_t g = (rows + kTeams - 1) / kTeams;
    return (uint32_t)(g < kMost ? g : kMost);
  }
  static hipError_t run(const NormGradArgs& a, hipStream_t stream) {
    const uint32_t g = groups(a.rows, a.cols);
    if (g > 0) norm_grad_kernel<ET, L, W, K, THREADS, SHORT><<<dim3(g), dim3(THREADS), 0, stream>>>(a);
    return hipGetLastError();
  }
};
// Calls f with the NormGrad of a row of cols values.
template <int ET, class F>
auto with_norm_grad(size_t cols, F&& f) {
  const size_t v = (cols + Type<ET>::kVec - 1) / Type<ET>::kVec;
  if (cols < Type<ET>::kVec) return f(NormGrad<ET, 8, 1, 1, 256, true>());
  if (v <= 8) return f(NormGrad<ET, 8, 1, 1, 1024>());
  if (v <= 16) return f(NormGrad<ET, 16, 1, 1, 1024>());
  if (v <= 32) return f(NormGrad<ET, 32, 1, 1, 1024>());
  if (v <= 64) return f(NormGrad<ET, 64, 1, 1, 1024>());
  if (v <= 128) return f(NormGrad<ET, 64, 2, 1, 1024>());
  if (v <= 256) return f(NormGrad<ET, 64, 4, 1, 1024>());
  if (v <= 512) return f(NormGrad<ET, 64, 8, 1, 1024>());
  if (v <= 1024) return f(NormGrad<ET, 64, 16, 1, 1024>());
  if (v <= 2048) return f(NormGrad<ET, 64, 16, 2, 1024>());
  if constexpr (ET == GB_DTYPE_F32) {
    if (v > 4096) return f(NormGrad<ET, 64, 16, 8, 1024>());
  }
  return f(NormGrad<ET, 64, 16, 4, 1024>());
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
