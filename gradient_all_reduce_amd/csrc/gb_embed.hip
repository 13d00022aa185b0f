// gb_embed.hip — embedding lookup with scaling, and the table's gradient by
// sorted tokens.  The formulas and the order of the gradient's sums stand in
// include/gbreduce.h.
#include "gb_rows.h"

namespace gb {
namespace {

__device__ __forceinline__ int64_t load_id(const void* ids, int dtype, size_t t) {
  return dtype == GB_DTYPE_I64 ? *((const GB_GLOBAL int64_t*)ids + t) : (int64_t) * ((const GB_GLOBAL int32_t*)ids + t);
}
// The row of an id, or a number of vocab or more for an id outside the table:
// the difference without a sign, which is at least 2^64 - 2^63 - first > vocab
// for an id below first.
__device__ __forceinline__ uint64_t row_of(int64_t id, int64_t first) { return (uint64_t)id - (uint64_t)first; }

// ---------------------------------------------------------------------------
// Lookup: the output is cut into vectors of V values, and a lane copies U of
// them, 256 apart, all ids and then all rows in flight at once.
// ---------------------------------------------------------------------------
constexpr int kLookThreads = 256;
template <int TT, int OT, int U>
__global__ __launch_bounds__(kLookThreads) void embedding_kernel(LookArgs a, uint32_t row_vecs, size_t vecs) {
  constexpr int V = Type<TT>::kVec < Type<OT>::kVec ? Type<TT>::kVec : Type<OT>::kVec;
  const size_t base = (size_t)blockIdx.x * (kLookThreads * U) + threadIdx.x;
  size_t token[U];
  uint64_t row[U];
  uint32_t col[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const size_t v = base + (size_t)u * kLookThreads;
    token[u] = v / row_vecs;
    col[u] = (uint32_t)(v - token[u] * row_vecs) * V;
    row[u] = v < vecs ? row_of(load_id(a.ids, a.id_dtype, token[u]), a.first) : a.vocab;
  }
  Raw<TT, V> x[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    x[u] = row[u] < a.vocab ? load_raw<TT, V, false>(a.table.p, row[u] * a.table.stride + col[u],
                                                     left_of(col[u], (uint32_t)a.dim))
                            : zero_raw<TT, V>();
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    if (base + (size_t)u * kLookThreads >= vecs) break;
    float y[V];
#pragma unroll
    for (int e = 0; e < V; e++) y[e] = row[u] < a.vocab ? canon(raw_value<TT, V>(x[u], e) * a.scale) : 0.0f;
    store_vals<OT, V, true>(a.out.p, token[u] * a.out.stride + col[u], left_of(col[u], (uint32_t)a.dim), y);
  }
}

// ---------------------------------------------------------------------------
// The tokens in the order of their rows, those of a row in their own order: a
// stable radix sort.  Tokens that name no row of the table, or the padding
// row, are left out by the first digit's pass.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = kSortThreads / kWave;
constexpr uint32_t kBins = 1u << kSortDigitBits;
static_assert(kBins == kSortThreads, "a lane for each bin");

struct Digits {
  uint32_t bits, passes;  // passes * bits cover vocab - 1
};

__device__ __forceinline__ bool token_row(const LookGradArgs& a, size_t t, uint32_t& row) {
  const int64_t id = load_id(a.ids, a.id_dtype, t);
  const uint64_t r = row_of(id, a.first);
  row = (uint32_t)r;
  return r < a.vocab && id != a.padding;
}

// Lanes of the wavefront whose digit is this lane's, among the valid ones.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool valid, uint32_t bits) {
  uint64_t same = __ballot(valid);
  for (uint32_t b = 0; b < bits; b++) {
    const uint64_t set = __ballot((digit >> b) & 1u);
    same &= (digit >> b) & 1u ? set : ~set;
  }
  return same;
}
__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// Ranks I digits a lane within the wavefront, item i of the lanes before item
// i + 1: rank[i] counts the equal digits before it, and counts[digit] ends as
// their number.  counts: zeroed, this wavefront's own.
template <int I>
__device__ __forceinline__ void rank_wave(const uint32_t (&digit)[I], const bool (&valid)[I], uint32_t bits,
                                          volatile uint16_t* counts, uint32_t (&rank)[I]) {
#pragma unroll
  for (int i = 0; i < I; i++) {
    const uint64_t same = same_digit(digit[i], valid[i], bits);
    const uint32_t below = lanes_below(same);
    if (valid[i]) {
      const uint32_t before = counts[digit[i]];
      rank[i] = before + below;
      // LDS instructions of a wavefront keep their order: all lanes have read
      // before the first lane of each digit writes
      __builtin_amdgcn_wave_barrier();
      if (below == 0) counts[digit[i]] = (uint16_t)(before + __popcll(same));
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Exclusive sum over the workgroup's lanes; *total receives the sum.
__device__ __forceinline__ uint32_t scan_lanes(uint32_t v, uint32_t* waves, uint32_t* total) {
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t s = v;
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t o = __shfl_up(s, d);
    if ((int)lane >= d) s += o;
  }
  if (lane == kWave - 1) waves[wave] = s;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kSortWaves; w++) {
    if (w < (int)wave) before += waves[w];
    all += waves[w];
  }
  *total = all;
  return before + s - v;
}

// One workgroup sorts up to kSortSmall tokens, in LDS between the passes.
constexpr int kSmallItems = kSortSmall / kSortThreads;
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(LookGradArgs a, Digits d, uint32_t* count,
                                                                  uint32_t* keys, uint32_t* tokens) {
  __shared__ uint32_t row_of_slot[kSortSmall], token_of_slot[kSortSmall];
  __shared__ uint16_t counts[kSortWaves][kBins];
  __shared__ uint32_t start[kBins], waves[kSortWaves];
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  // items a lane takes: only as many rounds as the tokens need
  const uint32_t rounds = ((uint32_t)a.tokens + kSortThreads - 1) / kSortThreads;
  uint32_t key[kSmallItems], token[kSmallItems], digit[kSmallItems], rank[kSmallItems];
  bool valid[kSmallItems];
  const uint32_t first = wave * rounds * kWave + lane;
#pragma unroll
  for (int i = 0; i < kSmallItems; i++) {
    token[i] = first + i * kWave;
    key[i] = 0;
    valid[i] = i < (int)rounds && token[i] < a.tokens && token_row(a, token[i], key[i]);
  }
  uint32_t n = 0;
  for (uint32_t pass = 0; pass < d.passes; pass++) {
    for (uint32_t i = threadIdx.x; i < kSortWaves * kBins / 2; i += kSortThreads) ((uint32_t*)counts)[i] = 0u;
    if (pass > 0) {
#pragma unroll
      for (int i = 0; i < kSmallItems; i++) {
        const uint32_t at = first + i * kWave;
        valid[i] = i < (int)rounds && at < n;
        if (valid[i]) key[i] = row_of_slot[at], token[i] = token_of_slot[at];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSmallItems; i++) digit[i] = (key[i] >> (pass * d.bits)) & ((1u << d.bits) - 1u);
    rank_wave<kSmallItems>(digit, valid, d.bits, counts[wave], rank);
    __syncthreads();
    uint32_t sum = 0;
    for (int w = 0; w < kSortWaves; w++) {
      const uint32_t c = counts[w][threadIdx.x];
      counts[w][threadIdx.x] = (uint16_t)sum;
      sum += c;
    }
    const uint32_t before = scan_lanes(sum, waves, &n);
    start[threadIdx.x] = before;
    __syncthreads();
    const bool last = pass + 1 == d.passes;
#pragma unroll
    for (int i = 0; i < kSmallItems; i++) {
      if (!valid[i]) continue;
      const uint32_t to = start[digit[i]] + counts[wave][digit[i]] + rank[i];
      if (last) {
        keys[to] = key[i];
        tokens[to] = token[i];
      } else {
        row_of_slot[to] = key[i];
        token_of_slot[to] = token[i];
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = n;
}

// A digit pass over more tokens: workgroup b of gridDim.x takes a run of whole
// tiles.  The first pass reads the ids.
struct DigitPass {
  const uint32_t* keys;    // NULL in the first pass
  const uint32_t* tokens;
  const uint32_t* count;   // tokens in them
  uint32_t* hist;          // [workgroups][bins]
  uint32_t shift, bits;
};
__device__ __forceinline__ size_t block_tokens(size_t tokens) {
  const size_t tiles = (tokens + kSortTile - 1) / kSortTile;
  return (tiles + gridDim.x - 1) / gridDim.x * kSortTile;
}
__device__ __forceinline__ bool pass_item(const LookGradArgs& a, const DigitPass& p, size_t at, size_t n,
                                          uint32_t& key, uint32_t& token) {
  if (at >= n) return false;
  if (p.keys == nullptr) {
    token = (uint32_t)at;
    return token_row(a, at, key);
  }
  key = p.keys[at];
  token = p.tokens[at];
  return true;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(LookGradArgs a, DigitPass p) {
  __shared__ uint32_t bins[kBins];
  bins[threadIdx.x] = 0u;
  __syncthreads();
  const size_t n = p.keys == nullptr ? a.tokens : *p.count, each = block_tokens(a.tokens);
  const size_t from = blockIdx.x * each, to = from + each < n ? from + each : n;
  for (size_t at = from + threadIdx.x; at < to; at += kSortThreads) {
    uint32_t key, token;
    if (pass_item(a, p, at, n, key, token)) atomicAdd(&bins[(key >> p.shift) & ((1u << p.bits) - 1u)], 1u);
  }
  __syncthreads();
  p.hist[(size_t)blockIdx.x * kBins + threadIdx.x] = bins[threadIdx.x];
}

constexpr int kTileItems = kSortTile / kSortThreads;
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(LookGradArgs a, DigitPass p, uint32_t* keys,
                                                                    uint32_t* tokens, uint32_t* count) {
  __shared__ uint16_t counts[kSortWaves][kBins];
  __shared__ uint32_t start[kBins], waves[kSortWaves];
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  // where this workgroup's tokens of each bin begin: after all smaller bins,
  // and after the earlier workgroups' tokens of the same bin
  uint32_t mine = 0, sum = 0;
#pragma unroll 8
  for (uint32_t b = 0; b < gridDim.x; b++) {
    const uint32_t c = p.hist[(size_t)b * kBins + threadIdx.x];
    if (b < blockIdx.x) mine += c;
    sum += c;
  }
  uint32_t total;
  uint32_t begin = scan_lanes(sum, waves, &total) + mine;
  const size_t n = p.keys == nullptr ? a.tokens : *p.count, each = block_tokens(a.tokens);
  const size_t from = blockIdx.x * each, to = from + each < n ? from + each : n;
  for (size_t tile = from; tile < to; tile += kSortTile) {
    for (uint32_t i = threadIdx.x; i < kSortWaves * kBins / 2; i += kSortThreads) ((uint32_t*)counts)[i] = 0u;
    start[threadIdx.x] = begin;
    uint32_t key[kTileItems], token[kTileItems], digit[kTileItems], rank[kTileItems];
    bool valid[kTileItems];
#pragma unroll
    for (int i = 0; i < kTileItems; i++) {
      key[i] = 0;
      valid[i] = pass_item(a, p, tile + (wave * kTileItems + i) * kWave + lane, n, key[i], token[i]);
      digit[i] = (key[i] >> p.shift) & ((1u << p.bits) - 1u);
    }
    __syncthreads();
    rank_wave<kTileItems>(digit, valid, p.bits, counts[wave], rank);
    __syncthreads();
    uint32_t in_tile = 0;
    for (int w = 0; w < kSortWaves; w++) {
      const uint32_t c = counts[w][threadIdx.x];
      counts[w][threadIdx.x] = (uint16_t)in_tile;
      in_tile += c;
    }
    begin += in_tile;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileItems; i++) {
      if (!valid[i]) continue;
      const uint32_t at = start[digit[i]] + counts[wave][digit[i]] + rank[i];
      keys[at] = key[i];
      tokens[at] = token[i];
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *count = total;
}

// ---------------------------------------------------------------------------
// The sums.  A run is the sorted tokens of one row; its folds begin at every
// kFold-th token from its start.  A wavefront takes the folds that begin in a
// window of kFold sorted tokens, for a slab of columns: the sum of a run of
// one fold goes to the table, any other fold's to the partials, where the join
// finds it.  Of two folds of longer runs that begin in one window, one ends a
// run (it is not that run's first) and one begins a run, since the folds of a
// run lie exactly a window apart and a run of one fold leaves no partial.
// ---------------------------------------------------------------------------
struct Sorted {
  const uint32_t* count;  // NULL: no tokens
  const uint32_t* keys;
  const uint32_t* tokens;
  float* partials;
  size_t stride;  // of the partials
};
__device__ __forceinline__ size_t partial_slot(uint32_t fold_start, bool begins_run) {
  return 2 * (size_t)(fold_start / kFold) + (begins_run ? 1 : 0);
}

// First position in [0, n) whose key is at least key (n if none).
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t n, uint32_t key) {
  uint32_t lo = 0, hi = n;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (keys[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// A row of the table from its sum.
template <int GT, int V>
__device__ __forceinline__ void store_row(const LookGradArgs& a, uint32_t row, uint32_t col, uint32_t left,
                                          const float (&sum)[V]) {
  const size_t at = (size_t)row * a.dtable.stride + col;
  float v[V];
  constexpr int kPart = Type<GT>::kVec < V ? Type<GT>::kVec : V;
  Raw<GT, kPart> old[V / kPart];
  if (a.accumulate) {
#pragma unroll
    for (int j = 0; j < V / kPart; j++) {
      old[j] = load_raw<GT, kPart, false>(a.dtable.p, at + j * kPart,
                                          left > (uint32_t)(j * kPart) ? left - j * kPart : 0u);
    }
  }
#pragma unroll
  for (int e = 0; e < V; e++) {
    v[e] = sum[e] * a.scale;
    if (a.accumulate) v[e] = raw_value<GT, kPart>(old[e / kPart], e % kPart) + v[e];
    v[e] = canon(v[e]);
  }
  store_vals<GT, V, true>(a.dtable.p, at, left, v);
}

constexpr int kSumWaves = 4;
template <int ET, int GT>
__device__ __forceinline__ void sum_window(const LookGradArgs& a, const Sorted& s, uint32_t window, uint32_t slab) {
  constexpr int V = Type<ET>::kVec, U = 4;
  const uint32_t n = *s.count, p0 = window * kFold, lane = threadIdx.x % kWave;
  if (p0 >= n) return;
  const uint32_t col = (slab * kWave + lane) * V, left = left_of(col, (uint32_t)a.dim);
  const uint32_t pa = p0 + lane, pb = p0 + kFold + lane;
  const uint32_t key_a = pa < n ? s.keys[pa] : ~0u, key_b = pb < n ? s.keys[pb] : ~0u;
  const uint32_t token_a = pa < n ? s.tokens[pa] : 0u, token_b = pb < n ? s.tokens[pb] : 0u;
  const uint32_t before = pa > 0 && pa < n ? s.keys[pa - 1] : ~0u;
  // where runs begin in the window, and whether one goes on into it
  uint64_t starts = __ballot(pa < n && (pa == 0 || before != key_a));
  uint64_t heads = starts;
  if (!(starts & 1u)) {
    const uint32_t key = __builtin_amdgcn_readfirstlane(key_a);
    const uint32_t offset = (lower_bound(s.keys, n, key) - p0) % kFold;  // of its fold in this window
    const uint64_t same = __ballot(pa < n && key_a == key);
    if ((same >> offset) & 1u) heads |= (uint64_t)1 << offset;
  }
  if (heads == 0) return;
  // the last fold may end beyond the window
  const uint32_t last = 63 - __clzll(heads);
  const uint32_t last_key = __builtin_amdgcn_readlane(key_a, last);
  const uint64_t tail_a = __ballot(pa < n && key_a == last_key) >> last;
  const uint64_t tail_b = __ballot(pb < n && key_b == last_key && lane < last);
  const uint32_t end = last + __popcll(tail_a) + __popcll(tail_b);
  // runs of more than one fold
  const uint64_t more = __ballot(pb < n && key_b == key_a);

  float acc[V];
  uint32_t at = __ffsll((unsigned long long)heads) - 1;
  uint32_t head = at;
  while (at < end) {
    Raw<ET, V> x[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t i = at + u;
      if (i < end) {
        const uint32_t t = i < 64 ? __builtin_amdgcn_readlane(token_a, i) : __builtin_amdgcn_readlane(token_b, i - 64);
        x[u] = load_raw<ET, V, true>(a.dout.p, (size_t)t * a.dout.stride + col, left);
      } else {
        x[u] = zero_raw<ET, V>();
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t i = at + u;
      if (i >= end) break;
      const bool begins = i < 64 && ((heads >> i) & 1u);
      if (begins) head = i;
#pragma unroll
      for (int e = 0; e < V; e++) {
        const float v = raw_value<ET, V>(x[u], e);
        acc[e] = begins ? v : acc[e] + v;
      }
      if (i + 1 == end || (i + 1 < 64 && ((heads >> (i + 1)) & 1u))) {
        const bool first = (starts >> head) & 1u;
        if (first && !((more >> head) & 1u)) {
          store_row<GT, V>(a, __builtin_amdgcn_readlane(key_a, head), col, left, acc);
        } else {
          float* const out = s.partials + partial_slot(p0 + head, first) * s.stride;
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float v[4] = {acc[j], acc[j + 1], acc[j + 2], acc[j + 3]};
            store_vals<GB_DTYPE_F32, 4, false>(out, col + j, left > (uint32_t)j ? left - j : 0u, v);
          }
        }
      }
    }
    at += U;
  }
}

// Zeros in the rows that no token names: rows [row, row + rows), rows <= 64.
template <int GT>
__device__ __forceinline__ void zero_rows(const LookGradArgs& a, const Sorted& s, size_t row, uint32_t rows) {
  const uint32_t lane = threadIdx.x % kWave;
  const uint32_t n = s.count != nullptr ? *s.count : 0u;
  const bool mine = lane < rows && row + lane < a.vocab;
  const uint32_t r = (uint32_t)(row + lane);
  bool empty = mine;
  if (mine && n > 0) {
    const uint32_t at = lower_bound(s.keys, n, r);
    empty = at == n || s.keys[at] != r;
  }
  const uint64_t todo = __ballot(empty);
  constexpr int V = Type<GT>::kVec;
  float zero[V];
#pragma unroll
  for (int e = 0; e < V; e++) zero[e] = 0.0f;
  for (uint32_t i = threadIdx.x / kWave; i < rows; i += kSumWaves) {
    if (!((todo >> i) & 1u)) continue;
    const size_t at = (row + i) * a.dtable.stride;
    for (size_t c = lane * V; c < a.dim; c += kWave * V) {
      store_vals<GT, V, true>(a.dtable.p, at + c, left_of((uint32_t)c, (uint32_t)a.dim), zero);
    }
  }
}

// Workgroups [0, sums) take windows and slabs, the rest rows without a token.
template <int ET, int GT>
__global__ __launch_bounds__(kSumWaves* kWave) void embedding_sum_kernel(LookGradArgs a, Sorted s, uint32_t sums,
                                                                        uint32_t slabs, size_t units,
                                                                        uint32_t zero_each) {
  if (blockIdx.x < sums) {
    const size_t unit = (size_t)blockIdx.x * kSumWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (unit < units) sum_window<ET, GT>(a, s, (uint32_t)(unit / slabs), (uint32_t)(unit % slabs));
  } else {
    zero_rows<GT>(a, s, (size_t)(blockIdx.x - sums) * zero_each, zero_each);
  }
}

// The sums of runs of several folds: a workgroup takes the run that begins in
// its window, if it is such a run (two of them begin more than a window
// apart), for a slab of 256 columns.  Level by level kFold sums are added in
// order, each wavefront taking every kJoinWaves-th of a level's groups.
constexpr int kJoinWaves = 4;
template <int GT>
__global__ __launch_bounds__(kJoinWaves* kWave) void embedding_join_kernel(LookGradArgs a, Sorted s) {
  const uint32_t n = *s.count, p0 = blockIdx.x * kFold, lane = threadIdx.x % kWave;
  if (p0 >= n) return;
  const uint32_t p = p0 + lane, key = p < n ? s.keys[p] : 0u;
  const bool head = p + kFold < n && s.keys[p + kFold] == key && (p == 0 || s.keys[p - 1] != key);
  const uint64_t heads = __ballot(head);
  if (heads == 0) return;
  const uint32_t at = __ffsll((unsigned long long)heads) - 1, start = p0 + at;
  const uint32_t row = __builtin_amdgcn_readlane(key, at);
  const uint32_t length = (row == ~0u ? n : lower_bound(s.keys, n, row + 1)) - start;
  const uint32_t col = (blockIdx.y * kWave + lane) * 4, left = left_of(col, (uint32_t)a.dim);
  const uint32_t wave = threadIdx.x / kWave;
  auto slot = [&](uint32_t fold) {
    return s.partials + partial_slot(start + fold * kFold, fold == 0) * s.stride + col;
  };
  uint32_t level = 1;  // a level's sums stand in every level-th fold's slot
  for (uint32_t sums = (length + kFold - 1) / kFold; sums > 1; sums = (sums + kFold - 1) / kFold) {
    for (uint32_t g = wave; g * kFold < sums; g += kJoinWaves) {
      const uint32_t from = g * kFold, to = from + kFold < sums ? from + kFold : sums;
      if (left > 0) {
        f4 v = *(const f4*)slot(from * level);
#pragma unroll 8
        for (uint32_t i = from + 1; i < to; i++) v += *(const f4*)slot(i * level);
        *(f4*)slot(from * level) = v;
      }
    }
    level *= kFold;
    __syncthreads();
  }
  if (wave != 0 || left == 0) return;
  const f4 v = *(const f4*)slot(0);
  const float sum[4] = {v.x, v.y, v.z, v.w};
  store_row<GT, 4>(a, row, col, left, sum);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int TT, int OT>
hipError_t run_look(const LookArgs& a, hipStream_t stream) {
  constexpr int V = Type<TT>::kVec < Type<OT>::kVec ? Type<TT>::kVec : Type<OT>::kVec, U = 4;
  const size_t row_vecs = (a.dim + V - 1) / V, vecs = a.tokens * row_vecs;
  const size_t grid = (vecs + kLookThreads * U - 1) / (kLookThreads * U);
  embedding_kernel<TT, OT, U><<<dim3((unsigned)grid), dim3(kLookThreads), 0, stream>>>(a, (uint32_t)row_vecs, vecs);
  return hipGetLastError();
}
template <int TT>
hipError_t pick_look(const LookArgs& a, hipStream_t stream) {
  if (a.out_dtype == GB_DTYPE_F32) return run_look<TT, GB_DTYPE_F32>(a, stream);
  if (a.out_dtype == GB_DTYPE_F16) return run_look<TT, GB_DTYPE_F16>(a, stream);
  return run_look<TT, GB_DTYPE_BF16>(a, stream);
}

hipError_t sort_tokens(const LookGradArgs& a, const LookGradLayout& l, Sorted* s, hipStream_t stream) {
  uint32_t bits = 1;
  while (bits < 32 && ((a.vocab - 1) >> bits) != 0) bits++;
  Digits d;
  d.passes = (bits + kSortDigitBits - 1) / kSortDigitBits;
  d.bits = (bits + d.passes - 1) / d.passes;
  uint32_t* const count = (uint32_t*)(a.workspace + l.count);
  uint32_t *keys[2], *tokens[2];
  for (int i = 0; i < 2; i++) {
    keys[i] = (uint32_t*)(a.workspace + l.keys[i]);
    tokens[i] = (uint32_t*)(a.workspace + l.tokens[i]);
  }
  s->count = count;
  if (a.tokens <= kSortSmall) {
    s->keys = keys[0], s->tokens = tokens[0];
    sort_small_kernel<<<dim3(1), dim3(kSortThreads), 0, stream>>>(a, d, count, keys[0], tokens[0]);
    return hipGetLastError();
  }
  const dim3 grid(sort_blocks(a.tokens));
  for (uint32_t pass = 0; pass < d.passes; pass++) {
    const int from = (pass + 1) % 2, to = pass % 2;
    DigitPass p = {pass == 0 ? nullptr : keys[from], tokens[from], count, (uint32_t*)(a.workspace + l.hist),
                   pass * d.bits, d.bits};
    sort_count_kernel<<<grid, dim3(kSortThreads), 0, stream>>>(a, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sort_scatter_kernel<<<grid, dim3(kSortThreads), 0, stream>>>(a, p, keys[to], tokens[to], count);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    s->keys = keys[to], s->tokens = tokens[to];
  }
  return hipSuccess;
}

template <int ET, int GT>
hipError_t run_sums(const LookGradArgs& a, const Sorted& s, hipStream_t stream) {
  constexpr size_t kCols = (size_t)kWave * Type<ET>::kVec;
  const size_t slabs = (a.dim + kCols - 1) / kCols, units = look_windows(a.tokens) * slabs;
  const size_t sums = (units + kSumWaves - 1) / kSumWaves;
  // rows a workgroup looks after: about 256 KiB of the table, 64 at most
  size_t each = ((size_t)256 << 10) / (a.dim * Type<GT>::kSize);
  each = each < 1 ? 1 : each > 64 ? 64 : each;
  const size_t zeros = a.accumulate ? 0 : (a.vocab + each - 1) / each;
  if (sums + zeros > 0) {
    embedding_sum_kernel<ET, GT><<<dim3((unsigned)(sums + zeros)), dim3(kSumWaves * kWave), 0, stream>>>(
        a, s, (uint32_t)sums, (uint32_t)slabs, units, (uint32_t)each);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.tokens <= kFold) return e;
  const dim3 grid((unsigned)look_windows(a.tokens), (unsigned)((a.dim + 4 * kWave - 1) / (4 * kWave)));
  embedding_join_kernel<GT><<<grid, dim3(kJoinWaves * kWave), 0, stream>>>(a, s);
  return hipGetLastError();
}
template <int ET>
hipError_t pick_sums(const LookGradArgs& a, const Sorted& s, hipStream_t stream) {
  if (a.grad_dtype == GB_DTYPE_F32) return run_sums<ET, GB_DTYPE_F32>(a, s, stream);
  if (a.grad_dtype == GB_DTYPE_F16) return run_sums<ET, GB_DTYPE_F16>(a, s, stream);
  return run_sums<ET, GB_DTYPE_BF16>(a, s, stream);
}

}  // namespace

hipError_t launch_embedding(const LookArgs& a, hipStream_t stream) {
  if (a.table_dtype == GB_DTYPE_F32) return pick_look<GB_DTYPE_F32>(a, stream);
  if (a.table_dtype == GB_DTYPE_F16) return pick_look<GB_DTYPE_F16>(a, stream);
  return pick_look<GB_DTYPE_BF16>(a, stream);
}

hipError_t launch_embedding_grad(const LookGradArgs& a, hipStream_t stream) {
  Sorted s = {};
  if (a.tokens > 0) {
    const LookGradLayout l = look_grad_layout(a.tokens, a.dim);
    hipError_t e = sort_tokens(a, l, &s, stream);
    if (e != hipSuccess) return e;
    s.partials = (float*)(a.workspace + l.partials);
    s.stride = look_partial_stride(a.dim);
  }
  if (a.dtype == GB_DTYPE_F32) return pick_sums<GB_DTYPE_F32>(a, s, stream);
  if (a.dtype == GB_DTYPE_F16) return pick_sums<GB_DTYPE_F16>(a, s, stream);
  return pick_sums<GB_DTYPE_BF16>(a, s, stream);
}

}  // namespace gb
