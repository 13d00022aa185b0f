// gb_embed.hip — embedding lookup with scaling, and the table's gradient by
// sorted tokens.  The formulas and the order of the gradient's sums stand in
// include/gbreduce.h.
//
// All of it moves rows and adds them: one multiplication or addition a value.
// Measured on MI355X, where the best plain copy moves 6.65 TB/s and a plain write
// 6.69: 32,768 tokens out of a 131,072 x 4096 float32 table into bfloat16 95 us
// (4.9 TB/s by the bytes of the different rows, 197 MB; rows are read again for each
// of their tokens, 537 MB, and 367 MB of that pass the L2s); the gradient of 16,384 bfloat16
// tokens written over all of a 131,072 x 4096 float32 table 413 to 436 us (5.2 to
// 5.5 TB/s: the sums and zeros 375 to 405 us, the sort 26, the join 6), of 98,304
// tokens added into 50,003 x 1024 105 to 122 us (3.0 to 3.5 TB/s: the sums 72 to 82,
// the sort 25, the join 6 to 10), of 512 tokens over 2000 x 257 float32 values 9 us
// the sort, 8 the sums and 2 to 4 the join.
#include "gb_rows.h"

#define GB_LDS __attribute__((address_space(3)))

namespace gb {
namespace {

// The ids of N tokens, one type test for all of them: a load inside a branch
// would be waited for there.
template <int N>
__device__ __forceinline__ void load_ids(const void* ids, int dtype, const uint32_t (&token)[N], int64_t (&id)[N]) {
  if (dtype == GB_DTYPE_I64) {
#pragma unroll
    for (int i = 0; i < N; i++) id[i] = ((const GB_GLOBAL int64_t*)ids)[token[i]];
  } else {
    int32_t narrow[N];
#pragma unroll
    for (int i = 0; i < N; i++) narrow[i] = ((const GB_GLOBAL int32_t*)ids)[token[i]];
#pragma unroll
    for (int i = 0; i < N; i++) id[i] = narrow[i];
  }
}
// The row of an id, or a number of vocab or more for an id outside the table:
// the difference without a sign, which is at least 2^64 - 2^63 - first > vocab
// for an id below first.
__device__ __forceinline__ uint64_t row_of(int64_t id, int64_t first) { return (uint64_t)id - (uint64_t)first; }

// ---------------------------------------------------------------------------
// Lookup: the output is cut into vectors of V values, and a lane copies U of
// them, 256 apart, all ids and then all rows in flight at once: nothing is
// read inside a branch, where it would be waited for (as it first was, with
// each id and row guarded: 32,768 tokens of 4096 float32 values 131 us).  The
// last vector of a row is moved back to end with the row, a token that names
// no row reads the first one and stores zeros.  Rows shorter than a vector,
// and a table without rows, take the guarded form.
// ---------------------------------------------------------------------------
constexpr int kLookThreads = 256;
struct LookCut {
  uint32_t vecs;      // of this launch, 2^30 at most
  uint32_t row_vecs;  // of a row
  uint64_t inverse;   // 2^64 / row_vecs rounded up; 0 for row_vecs = 1
};
template <int TT, int OT, bool GUARDED>
__global__ __launch_bounds__(kLookThreads) void embedding_kernel(LookArgs a, LookCut c) {
  constexpr int V = Type<TT>::kVec < Type<OT>::kVec ? Type<TT>::kVec : Type<OT>::kVec, U = GUARDED ? 1 : 4;
  const uint32_t dim = (uint32_t)a.dim, base = blockIdx.x * (kLookThreads * U) + threadIdx.x;
  uint32_t token[U], col[U];
  int64_t id[U];
  bool in[U];
  Raw<TT, V> x[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t v = min(base + u * kLookThreads, c.vecs - 1);
    // v / row_vecs: exact, as both are below 2^32
    token[u] = c.inverse == 0 ? v : (uint32_t)__umul64hi(v, c.inverse);
    col[u] = (v - token[u] * c.row_vecs) * V;
    if constexpr (!GUARDED) col[u] = min(col[u], dim - V);
  }
  load_ids<U>(a.ids, a.id_dtype, token, id);
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint64_t row = row_of(id[u], a.first);
    in[u] = row < a.vocab;
    const size_t at = (in[u] ? row : 0) * a.table.stride + col[u];
    if constexpr (GUARDED) x[u] = load_raw<TT, V, false>(a.table.p, at, in[u] ? dim - col[u] : 0u);
    else x[u] = load_full<TT, V, false>(a.table.p, at);
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    if (base + u * kLookThreads >= c.vecs) break;
    float y[V];
#pragma unroll
    for (int e = 0; e < V; e++) y[e] = in[u] ? canon(raw_value<TT, V>(x[u], e) * a.scale) : 0.0f;
    store_vals<OT, V, true>(a.out.p, (size_t)token[u] * a.out.stride + col[u], GUARDED ? dim - col[u] : V, y);
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

// The rows of N tokens, those below `to` of them that name one marked valid.
template <int N>
__device__ __forceinline__ void token_rows(const LookGradArgs& a, const uint32_t (&token)[N], uint32_t to,
                                           uint32_t (&key)[N], bool (&valid)[N]) {
  uint32_t at[N];
  int64_t id[N];
#pragma unroll
  for (int i = 0; i < N; i++) at[i] = min(token[i], (uint32_t)a.tokens - 1);
  load_ids<N>(a.ids, a.id_dtype, at, id);
#pragma unroll
  for (int i = 0; i < N; i++) {
    const uint64_t row = row_of(id[i], a.first);
    valid[i] = token[i] < to && row < a.vocab && id[i] != a.padding;
    key[i] = valid[i] ? (uint32_t)row : 0u;
  }
}

// Lanes of the wavefront whose digit is this lane's, among the valid ones.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool valid, uint32_t bits) {
  const uint64_t all = __ballot(valid);
  uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
  for (uint32_t b = 0; b < bits; b++) {
    const uint32_t mine = 0u - ((digit >> b) & 1u);  // all ones, or zeros
    const uint64_t set = __ballot(mine != 0u);
    lo &= ~((uint32_t)set ^ mine);
    hi &= ~((uint32_t)(set >> 32) ^ mine);
  }
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// Ranks `items` (I at most) digits a lane within the wavefront, item i of the
// lanes before item i + 1: rank[i] counts the equal digits before it, and
// counts[digit] ends as their number.  counts: zeroed, this wavefront's own, in
// LDS by its type: through a pointer of no address space volatile accesses are
// flat ones, each of which waits for all of the wavefront's accesses to memory.
template <int I>
__device__ __forceinline__ void rank_wave(const uint32_t (&digit)[I], const bool (&valid)[I], uint32_t items,
                                          uint32_t bits, volatile GB_LDS uint16_t* counts, uint32_t (&rank)[I]) {
#pragma unroll
  for (int i = 0; i < I; i++) {
    if (i >= (int)items) break;
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

// Clears the flags of the rows: part of parts.  (An array of whole 256 bytes.)
__device__ __forceinline__ void clear_named(const LookGradArgs& a, uint8_t* named, uint32_t part, uint32_t parts) {
  const size_t words = (a.vocab + 15) / 16;
  for (size_t i = (size_t)part * kSortThreads + threadIdx.x; i < words; i += (size_t)parts * kSortThreads) {
    ((u4*)named)[i] = u4{0u, 0u, 0u, 0u};
  }
}

// One workgroup sorts up to kSortSmall tokens, in LDS between the passes: one
// launch of 9 us instead of four of 5 to 9 us each.  Whole gradients, us, sorted
// this way and by digit passes: into 32,000 rows of 16 float32 values, added,
// 1025 tokens 26.3 and 30.7, 4096 34.3 and 38.8, 6144 37.8 and 40.2, 8192 42.1
// and 41.7; written, 8192 tokens 42.4 and 40.2.  With 10^6 rows, whose flags one
// workgroup clears here, written, 1025 tokens 165 and 174, 8192 184 and 177.
constexpr int kSmallItems = kSortSmall / kSortThreads;
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(LookGradArgs a, Digits d, uint32_t* count,
                                                                  uint32_t* keys, uint32_t* tokens, uint8_t* named) {
  __shared__ uint32_t row_of_slot[kSortSmall], token_of_slot[kSortSmall];
  __shared__ uint16_t counts[kSortWaves][kBins];
  __shared__ uint32_t start[kBins], waves[kSortWaves];
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  // items a lane takes: only as many rounds as the tokens need
  const uint32_t rounds = ((uint32_t)a.tokens + kSortThreads - 1) / kSortThreads;
  uint32_t key[kSmallItems], token[kSmallItems], digit[kSmallItems], rank[kSmallItems];
  bool valid[kSmallItems];
  const uint32_t first = wave * rounds * kWave + lane;
  // a wavefront's tokens end where the next one's begin
  const uint32_t own_end = min((wave + 1) * rounds * kWave, (uint32_t)a.tokens);
#pragma unroll
  for (int i = 0; i < kSmallItems; i++) token[i] = first + i * kWave;
  token_rows<kSmallItems>(a, token, own_end, key, valid);
  uint32_t n = 0;
  if (named != nullptr) clear_named(a, named, 0, 1);
  for (uint32_t pass = 0; pass < d.passes; pass++) {
    for (uint32_t w = 0; w < kSortWaves; w++) counts[w][threadIdx.x] = 0;
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
    rank_wave<kSmallItems>(digit, valid, rounds, d.bits, (GB_LDS uint16_t*)counts[wave], rank);
    __syncthreads();
    uint32_t sum = 0, c[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) c[w] = counts[w][threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) {
      counts[w][threadIdx.x] = (uint16_t)sum;
      sum += c[w];
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
        if (named != nullptr) named[key[i]] = 1;
      } else {
        row_of_slot[to] = key[i];
        token_of_slot[to] = token[i];
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    count[0] = n;
    count[1] = 0u;  // long runs, which the sums count
  }
}

// A digit pass over more tokens: workgroup b of gridDim.x takes a run of whole
// tiles.  The first pass reads the ids.
struct DigitPass {
  const uint32_t* keys;    // NULL in the first pass
  const uint32_t* tokens;
  const uint32_t* count;   // tokens in them
  uint32_t* hist;          // [workgroups][bins]
  uint8_t* named;          // flags of the rows that the first pass sets, or NULL
  uint32_t shift, bits;
};
__device__ __forceinline__ size_t block_tokens(size_t tokens) {
  const size_t tiles = (tokens + kSortTile - 1) / kSortTile;
  return (tiles + gridDim.x - 1) / gridDim.x * kSortTile;
}
// N items of a pass, those below `to` that name a row marked valid.
template <int N>
__device__ __forceinline__ void pass_items(const LookGradArgs& a, const DigitPass& p, const uint32_t (&at)[N],
                                           uint32_t to, uint32_t (&key)[N], uint32_t (&token)[N], bool (&valid)[N]) {
  if (p.keys == nullptr) {
    token_rows<N>(a, at, to, key, valid);
#pragma unroll
    for (int i = 0; i < N; i++) token[i] = at[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    const uint32_t j = min(at[i], (uint32_t)a.tokens - 1);
    key[i] = p.keys[j];
    token[i] = p.tokens[j];
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    valid[i] = at[i] < to;
    key[i] = valid[i] ? key[i] : 0u;
  }
}
constexpr int kTileItems = kSortTile / kSortThreads;

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(LookGradArgs a, DigitPass p) {
  __shared__ uint32_t bins[kBins];
  bins[threadIdx.x] = 0u;
  if (p.keys == nullptr && p.named != nullptr) clear_named(a, p.named, blockIdx.x, gridDim.x);
  __syncthreads();
  const size_t n = p.keys == nullptr ? a.tokens : *p.count, each = block_tokens(a.tokens);
  const size_t from = blockIdx.x * each, to = from + each < n ? from + each : n;
  for (size_t tile = from; tile < to; tile += kSortTile) {
    uint32_t at[kTileItems], key[kTileItems], token[kTileItems];
    bool valid[kTileItems];
#pragma unroll
    for (int i = 0; i < kTileItems; i++) at[i] = (uint32_t)tile + i * kSortThreads + threadIdx.x;
    pass_items<kTileItems>(a, p, at, (uint32_t)to, key, token, valid);
#pragma unroll
    for (int i = 0; i < kTileItems; i++) {
      if (valid[i]) atomicAdd(&bins[(key[i] >> p.shift) & ((1u << p.bits) - 1u)], 1u);
    }
  }
  __syncthreads();
  if (threadIdx.x >> p.bits == 0) p.hist[((size_t)blockIdx.x << p.bits) + threadIdx.x] = bins[threadIdx.x];
}

__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(LookGradArgs a, DigitPass p, uint32_t* keys,
                                                                    uint32_t* tokens, uint32_t* count) {
  __shared__ uint16_t counts[kSortWaves][kBins];
  __shared__ uint32_t start[kBins], waves[kSortWaves], sums[2][kSortThreads];
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const uint32_t bin = threadIdx.x & ((1u << p.bits) - 1u);
  const bool owner = threadIdx.x >> p.bits == 0;  // of the bin
  const size_t n = p.keys == nullptr ? a.tokens : *p.count, each = block_tokens(a.tokens);
  const size_t from = blockIdx.x * each, to = from + each < n ? from + each : n;
  uint32_t key[kTileItems], token[kTileItems], digit[kTileItems], rank[kTileItems];
  bool valid[kTileItems];
  auto load_tile = [&](size_t tile) {
    uint32_t at[kTileItems];
#pragma unroll
    for (int i = 0; i < kTileItems; i++) at[i] = (uint32_t)tile + (wave * kTileItems + i) * kWave + lane;
    pass_items<kTileItems>(a, p, at, (uint32_t)to, key, token, valid);
#pragma unroll
    for (int i = 0; i < kTileItems; i++) digit[i] = (key[i] >> p.shift) & ((1u << p.bits) - 1u);
  };
  load_tile(from);
  // where this workgroup's tokens of each bin begin: after all smaller bins,
  // and after the earlier workgroups' tokens of the same bin.  With fewer bins
  // than lanes several lanes share the workgroups of a bin.
  uint32_t mine = 0, sum = 0;
  const uint32_t sharers = kSortThreads >> p.bits;
  for (uint32_t first = threadIdx.x >> p.bits; first < gridDim.x; first += 16 * sharers) {
    uint32_t c[16];
#pragma unroll
    for (uint32_t i = 0; i < 16; i++) {
      const uint32_t b = first + i * sharers;
      c[i] = p.hist[((size_t)(b < gridDim.x ? b : 0) << p.bits) + bin];
    }
#pragma unroll
    for (uint32_t i = 0; i < 16; i++) {
      const uint32_t b = first + i * sharers;
      if (b < blockIdx.x) mine += c[i];
      if (b < gridDim.x) sum += c[i];
    }
  }
  sums[0][threadIdx.x] = sum;
  sums[1][threadIdx.x] = mine;
  __syncthreads();
  if (owner) {
    for (uint32_t i = threadIdx.x + (1u << p.bits); i < kSortThreads; i += 1u << p.bits) {
      sum += sums[0][i];
      mine += sums[1][i];
    }
  } else {
    sum = mine = 0;
  }
  uint32_t total;
  uint32_t begin = scan_lanes(sum, waves, &total) + mine;
  for (size_t tile = from; tile < to; tile += kSortTile) {
    if (tile != from) load_tile(tile);
    if (owner) {
      for (uint32_t w = 0; w < kSortWaves; w++) counts[w][bin] = 0;
      start[bin] = begin;
    }
    __syncthreads();
    rank_wave<kTileItems>(digit, valid, kTileItems, p.bits, (GB_LDS uint16_t*)counts[wave], rank);
    __syncthreads();
    if (owner) {
      uint32_t in_tile = 0, c[kSortWaves];
#pragma unroll
      for (int w = 0; w < kSortWaves; w++) c[w] = counts[w][bin];
#pragma unroll
      for (int w = 0; w < kSortWaves; w++) {
        counts[w][bin] = (uint16_t)in_tile;
        in_tile += c[w];
      }
      begin += in_tile;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileItems; i++) {
      if (!valid[i]) continue;
      const uint32_t at = start[digit[i]] + counts[wave][digit[i]] + rank[i];
      keys[at] = key[i];
      tokens[at] = token[i];
      if (p.keys == nullptr && p.named != nullptr) p.named[key[i]] = 1;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    count[0] = total;
    count[1] = 0u;  // long runs, which the sums count
  }
}

// ---------------------------------------------------------------------------
// The sums.  A run is the sorted tokens of one row; its folds begin at every
// kFold-th token from its start.  A wavefront takes the folds that begin in a
// window of kWindow sorted tokens, for a slab of columns: the sum of a run of
// one fold goes to the table, any other fold's to the partials, where the join
// finds it.  Two folds of longer runs that begin among the same kFold tokens:
// one ends a run (it is not that run's first) and one begins a run, since the
// folds of a run lie kFold apart and a run of one fold leaves no partial.
// ---------------------------------------------------------------------------
// 98,304 tokens of 1024 columns added: windows of 8, 16, 32 and 64 tokens 122, 112,
// 113 and 114 us; 16,384 of 4096: 100, 94, 101 and 98.
constexpr uint32_t kWindow = 16;
static_assert(kFold % kWindow == 0 && kFold == kWave, "a fold is a lane each");

struct LongRun {
  uint32_t start, length, row;
};
static_assert(sizeof(LongRun) == kLongRunBytes, "the workspace has room for them");
struct Sorted {
  uint32_t* count;       // tokens that name a row; NULL: no tokens
  uint32_t* long_count;  // runs of more than one fold
  LongRun* long_runs;
  const uint32_t* keys;
  const uint32_t* tokens;
  float* partials;
  size_t stride;   // of the partials
  uint8_t* named;  // whether a token names a row; NULL where no row needs zeros, or none has a token
};
__device__ __forceinline__ size_t partial_slot(uint32_t fold_start, bool begins_run) {
  return 2 * (size_t)(fold_start / kFold) + (begins_run ? 1 : 0);
}

// First position in [0, n) whose key is at least key (n if none): all lanes
// look at once, so a step divides the range by 65.  key is the same in all.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t n, uint32_t key) {
  const uint32_t lane = threadIdx.x % kWave;
  uint32_t lo = 0, hi = n;
  while (hi - lo > 0) {
    // lanes look at 64 places that cut [lo, hi) into 65 pieces, the first at lo + each
    const uint32_t each = (hi - lo) / (kWave + 1);
    const uint32_t at = lo + each + lane * (each + 1);
    const uint32_t less = __popcll(__ballot(at < hi && keys[at] < key));
    const uint32_t next = lo + each + less * (each + 1);  // the first place not below key
    lo = less == 0 ? lo : next - (each + 1) + 1;
    hi = next < hi ? next : hi;
  }
  return lo;
}

// A wavefront's slab is a vector in each lane, the shorter one of the two
// types, so that every access of an instruction is one contiguous run (two
// 16-byte halves of a lane's 8 float32 values would each touch every line,
// and the non-temporal hint lets a line go after the first: 16,384 tokens of
// 4096 columns added into float32 rows 108 us with 8 columns a lane, 94 with 4).
template <int ET, int GT>
struct Slab {
  static constexpr int V = Type<ET>::kVec < Type<GT>::kVec ? Type<ET>::kVec : Type<GT>::kVec;
  static constexpr uint32_t kCols = kWave * V;
};

// A row of the table from its sum and, with ADD, what it held.
template <int GT, int V, bool ADD>
__device__ __forceinline__ void store_row(const LookGradArgs& a, uint32_t row, uint32_t col, uint32_t left,
                                          const float (&sum)[V], const Raw<GT, V>& old) {
  char* const to = (char*)a.dtable.p + (size_t)row * a.dtable.stride * Type<GT>::kSize;
  float v[V];
#pragma unroll
  for (int e = 0; e < V; e++) {
    v[e] = sum[e] * a.scale;
    if constexpr (ADD) v[e] = raw_value<GT, V>(old, e) + v[e];
    v[e] = canon(v[e]);
  }
  store_vals<GT, V, true>(to, col, left, v);
}

constexpr int kSumWaves = 4;
constexpr uint32_t kXcds = 8;
static_assert(kSumLaunch % kXcds == 0 && (uint64_t)kSumLaunch * kSumWaves * kWave < (uint64_t)1 << 32,
              "a launch's lanes, and whole rounds of the XCDs");
template <int ET, int GT, bool ADD, bool FULL>
__device__ __forceinline__ void sum_window(const LookGradArgs& a, const Sorted& s, uint32_t window, uint32_t slab) {
  constexpr int V = Slab<ET, GT>::V, U = 8;
  const uint32_t p0 = window * kWindow, lane = threadIdx.x % kWave;
  const uint32_t pa = p0 + lane, pb = p0 + kFold + lane, tokens = (uint32_t)a.tokens;
  // read before their number is known: what lies beyond it is not looked at
  uint32_t key_a = s.keys[pa < tokens ? pa : 0], key_b = s.keys[pb < tokens ? pb : 0];
  const uint32_t before = s.keys[pa > 0 && pa < tokens ? pa - 1 : 0];
  const uint32_t token_a = s.tokens[pa < tokens ? pa : 0], token_b = s.tokens[pb < tokens ? pb : 0];
  const uint32_t n = *s.count;
  if (p0 >= n) return;
  key_a = pa < n ? key_a : ~0u;
  key_b = pb < n ? key_b : ~0u;
  uint32_t col = (slab * kWave + lane) * V;
  const uint32_t left = FULL ? V : left_of(col, (uint32_t)a.dim);
  // where runs begin in the lanes' tokens, and whether one goes on into them
  const uint64_t starts = __ballot(pa < n && (pa == 0 || before != key_a));
  uint64_t heads = starts;
  // runs of more than one fold from here on
  const uint64_t more = __ballot(pb < n && key_b == key_a);
  if (!(starts & 1u)) {
    const uint32_t key = __builtin_amdgcn_readfirstlane(key_a);
    const uint32_t start = lower_bound(s.keys, p0, key), offset = (start - p0) % kFold;  // of its next fold from here
    const uint64_t same = __ballot(pa < n && key_a == key), rest = __ballot(pb < n && key_b == key);
    if ((same >> offset) & 1u) {
      heads |= (uint64_t)1 << offset;
      if (slab == 0 && lane == 0 && offset < kWindow && !((more >> offset) & 1u)) {
        // the run's last fold: the run goes to the join's work list, whose order changes no result
        const uint32_t end = p0 + __popcll(same) + (same == ~(uint64_t)0 ? __popcll(rest) : 0);
        s.long_runs[atomicAdd(s.long_count, 1u)] = LongRun{start, end - start, key};
      }
    }
  }
  heads &= ((uint64_t)1 << kWindow) - 1;
  if (heads == 0) return;
  // the last fold may end beyond the window
  const uint32_t last = 63 - __clzll(heads);
  const uint32_t last_key = __builtin_amdgcn_readlane(key_a, last);
  const uint64_t tail_a = __ballot(pa < n && key_a == last_key) >> last;
  const uint64_t tail_b = __ballot(pb < n && key_b == last_key && lane < last);
  const uint32_t end = last + __popcll(tail_a) + __popcll(tail_b);
  const uint64_t whole = starts & ~more;  // runs of one fold: their sums are the table's

  float acc[V];
  Raw<ET, V> x[U];
  Raw<GT, V> old[ADD ? U : 1], now;
  uint32_t head = __ffsll((unsigned long long)heads) - 1;
  for (uint32_t at = head; at < end; at += U) {
    asm volatile("" : "+v"(col));  // a lane's offset of 32 bits, not widened ahead of the loop
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t i = at + u < end ? at + u : end - 1;
      const uint32_t ta = __builtin_amdgcn_readlane(token_a, i % 64), tb = __builtin_amdgcn_readlane(token_b, i % 64);
      const size_t t = i < 64 ? ta : tb;
      x[u] = load_raw<ET, V, true>((const char*)a.dout.p + t * a.dout.stride * Type<ET>::kSize, col, left);
    }
    if constexpr (ADD) {
#pragma unroll
      for (int u = 0; u < U; u++) {
        const uint32_t i = at + u;
        if (i < 64 && ((whole >> i) & 1u) && i < end) {
          const size_t row = __builtin_amdgcn_readlane(key_a, i);
          old[u] = load_raw<GT, V, true>((const char*)a.dtable.p + row * a.dtable.stride * Type<GT>::kSize, col, left);
        }
      }
    }
    // the sum of the fold that ends before token i, to where it belongs
    auto ends_before = [&](uint32_t i) { return i == end || (i < kWindow && ((heads >> i) & 1u)); };
    auto store_fold = [&]() {
      if ((whole >> head) & 1u) {
        store_row<GT, V, ADD>(a, __builtin_amdgcn_readlane(key_a, head), col, left, acc, now);
      } else {
        float* const out = s.partials + partial_slot(p0 + head, (starts >> head) & 1u) * s.stride;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const float v[4] = {acc[j], acc[j + 1], acc[j + 2], acc[j + 3]};
          store_vals<GB_DTYPE_F32, 4, false>(out, col + j, left > (uint32_t)j ? left - j : 0u, v);
        }
      }
    };
    if (at + U <= end && (at >= kWindow || ((heads >> at) & ((1u << U) - 1u)) == 0)) {
      // within a fold: nothing but additions
#pragma unroll
      for (int u = 0; u < U; u++) {
#pragma unroll
        for (int e = 0; e < V; e++) acc[e] += raw_value<ET, V>(x[u], e);
      }
      if (ends_before(at + U)) store_fold();
      continue;
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t i = at + u;
      if (i >= end) break;
      const bool begins = i < kWindow && ((heads >> i) & 1u);
      if (begins) {
        head = i;
        if constexpr (ADD) now = old[u];
      }
#pragma unroll
      for (int e = 0; e < V; e++) {
        const float v = raw_value<ET, V>(x[u], e);
        acc[e] = begins ? v : acc[e] + v;
      }
      if (ends_before(i + 1)) store_fold();
    }
  }
}

// Zeros in the rows that no token names: rows [row, row + rows), rows <= 64.
// Stored without the non-temporal hint (131,072 x 4096 float32: 357 us, with it
// 375), by workgroups that take about 16 KiB each and whose XCD's rows lie
// together (327 us; in the order of the workgroups 383).
template <int GT>
__device__ __forceinline__ void zero_rows(const LookGradArgs& a, const Sorted& s, size_t row, uint32_t rows) {
  const uint32_t lane = threadIdx.x % kWave;
  if (row >= a.vocab) return;
  const bool mine = lane < rows && row + lane < a.vocab;
  const uint64_t todo = __ballot(mine && (s.named == nullptr || s.named[row + lane] == 0));
  constexpr uint32_t V = Type<GT>::kVec;
  const float zero[V] = {};
  const uint32_t dim = (uint32_t)a.dim;
  for (uint32_t i = 0; i < rows; i++) {
    if (!((todo >> i) & 1u)) continue;
    char* const to = (char*)a.dtable.p + (row + i) * a.dtable.stride * Type<GT>::kSize;
    uint32_t c = threadIdx.x * V;
    for (; c + V <= dim; c += kSumWaves * kWave * V) store_vals<GT, (int)V, false>(to, c, V, zero);
    if (c < dim) store_vals<GT, (int)V, false>(to, c, dim - c, zero);
  }
}

// Workgroups [0, sums) take windows and slabs, the rest rows without a token.
template <int ET, int GT, bool ADD>
__global__ __launch_bounds__(kSumWaves* kWave) void embedding_sum_kernel(LookGradArgs a, Sorted s, SumGrid g) {
  const uint32_t group = g.base + blockIdx.x;
  if (ADD || group < g.sums) {
    const size_t unit = (size_t)group * kSumWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (unit >= g.units) return;
    const uint32_t window = (uint32_t)(unit / g.slabs), slab = (uint32_t)(unit % g.slabs);
    if ((slab + 1) * Slab<ET, GT>::kCols <= a.dim) sum_window<ET, GT, ADD, true>(a, s, window, slab);
    else sum_window<ET, GT, ADD, false>(a, s, window, slab);
  } else {
    // workgroups go to the 8 XCDs in turn: each XCD's rows lie together
    const uint32_t z = group - g.sums, per_xcd = g.zeros / kXcds;
    zero_rows<GT>(a, s, ((size_t)(z % kXcds) * per_xcd + z / kXcds) * g.zero_each, g.zero_each);
  }
}

// The sums of runs of several folds (a grid over all windows instead of the work
// list takes 22 us where this takes 6 to 10): a workgroup takes a run of the work list
// for a slab of 64 columns at a time.  Level by level kFold sums are added in
// order, each wavefront taking every kJoinWaves-th of a level's groups, all of
// a group's loads in flight at once.  Their addresses and conditions are the
// same in all lanes and take more scalar registers than there are: 133 spill to
// vector registers (79 with addresses a step apart, at level times).
constexpr int kJoinWaves = 4;
template <int GT>
__global__ __launch_bounds__(kJoinWaves* kWave) void embedding_join_kernel(LookGradArgs a, Sorted s, uint32_t slabs) {
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t items = *s.long_count * slabs;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const LongRun run = s.long_runs[item / slabs];
    const uint32_t start = run.start, length = run.length, row = run.row;
    const uint32_t col = item % slabs * kWave + lane;
    const bool in = col < a.dim;
    // the first fold's sum lies apart from the others', which stand two slots apart
    float* const first = s.partials + partial_slot(start, true) * s.stride + col;
    float* const rest = s.partials + partial_slot(start, false) * s.stride + col;
    auto slot = [&](uint32_t fold) { return fold == 0 ? first : rest + 2 * (size_t)fold * s.stride; };
    uint32_t level = 1;  // a level's sums stand in every level-th fold's slot
    for (uint32_t sums = (length + kFold - 1) / kFold; sums > 1; sums = (sums + kFold - 1) / kFold) {
      for (uint32_t g = wave; g * kFold < sums; g += kJoinWaves) {
        const uint32_t from = g * kFold, count = sums - from < kFold ? sums - from : kFold;
        if (in) {
          float x[kFold];
#pragma unroll
          for (uint32_t i = 0; i < kFold; i++) x[i] = i < count ? *slot((from + i) * level) : 0.0f;
          float v = x[0];
#pragma unroll
          for (uint32_t i = 1; i < kFold; i++) v = i < count ? v + x[i] : v;
          *slot(from * level) = v;
        }
      }
      level *= kFold;
      __syncthreads();
    }
    if (wave == 0 && in) {
      float v = *slot(0) * a.scale;
      const size_t at = (size_t)row * a.dtable.stride + col;
      if (a.accumulate) v = load_one<GT>(a.dtable.p, at) + v;
      store_one<GT>(a.dtable.p, at, canon(v));
    }
    // a wavefront may go on to the next run: its sums lie elsewhere
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int TT, int OT>
hipError_t run_look(LookArgs a, hipStream_t stream) {
  constexpr int V = Type<TT>::kVec < Type<OT>::kVec ? Type<TT>::kVec : Type<OT>::kVec;
  const bool guarded = a.dim < V || a.vocab == 0;
  LookCut c;
  c.row_vecs = (uint32_t)((a.dim + V - 1) / V);
  c.inverse = c.row_vecs == 1 ? 0 : ~(uint64_t)0 / c.row_vecs + 1;
  // a launch takes as many tokens as 2^30 vectors hold
  const size_t most = ((size_t)1 << 30) / c.row_vecs, tokens = a.tokens, each = kLookThreads * (guarded ? 1 : 4);
  for (size_t t = 0; t < tokens; t += most) {
    const size_t now = tokens - t < most ? tokens - t : most;
    c.vecs = (uint32_t)(now * c.row_vecs);
    const dim3 grid((unsigned)((c.vecs + each - 1) / each));
    if (guarded) embedding_kernel<TT, OT, true><<<grid, dim3(kLookThreads), 0, stream>>>(a, c);
    else embedding_kernel<TT, OT, false><<<grid, dim3(kLookThreads), 0, stream>>>(a, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.ids = (const char*)a.ids + now * (a.id_dtype == GB_DTYPE_I64 ? 8 : 4);
    a.out.p = (char*)a.out.p + now * a.out.stride * Type<OT>::kSize;
  }
  return hipSuccess;
}
template <int TT>
hipError_t pick_look(const LookArgs& a, hipStream_t stream) {
  if (a.out_dtype == GB_DTYPE_F32) return run_look<TT, GB_DTYPE_F32>(a, stream);
  if (a.out_dtype == GB_DTYPE_F16) return run_look<TT, GB_DTYPE_F16>(a, stream);
  return run_look<TT, GB_DTYPE_BF16>(a, stream);
}

hipError_t sort_tokens(const LookGradArgs& a, const LookGradLayout& l, Sorted* s, hipStream_t stream) {
  s->named = a.accumulate ? nullptr : (uint8_t*)(a.workspace + l.named);
  uint32_t bits = 1;
  while (bits < 32 && ((a.vocab - 1) >> bits) != 0) bits++;
  Digits d;
  d.passes = (bits + kSortDigitBits - 1) / kSortDigitBits;
  d.bits = (bits + d.passes - 1) / d.passes;
  if (d.bits < kSortLeastBits) d.bits = kSortLeastBits;
  uint32_t* const count = (uint32_t*)(a.workspace + l.count);
  uint32_t *keys[2], *tokens[2];
  for (int i = 0; i < 2; i++) {
    keys[i] = (uint32_t*)(a.workspace + l.keys[i]);
    tokens[i] = (uint32_t*)(a.workspace + l.tokens[i]);
  }
  s->count = count;
  s->long_count = count + 1;
  s->long_runs = (LongRun*)(a.workspace + l.long_runs);
  if (a.tokens <= kSortSmall) {
    s->keys = keys[0], s->tokens = tokens[0];
    sort_small_kernel<<<dim3(1), dim3(kSortThreads), 0, stream>>>(a, d, count, keys[0], tokens[0], s->named);
    return hipGetLastError();
  }
  const dim3 grid(sort_blocks(a.tokens));
  for (uint32_t pass = 0; pass < d.passes; pass++) {
    const int from = (pass + 1) % 2, to = pass % 2;
    DigitPass p = {pass == 0 ? nullptr : keys[from], tokens[from], count, (uint32_t*)(a.workspace + l.hist),
                   s->named, pass * d.bits, d.bits};
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
  constexpr size_t kCols = Slab<ET, GT>::kCols;
  SumGrid g = {};
  g.slabs = (uint32_t)((a.dim + kCols - 1) / kCols);
  g.units = (a.tokens + kWindow - 1) / kWindow * g.slabs;
  g.sums = (uint32_t)(((g.units + kSumWaves - 1) / kSumWaves + kXcds - 1) / kXcds * kXcds);
  // rows a workgroup looks after (zero_rows): about 16 KiB of the table, 64 at most
  const size_t each = ((size_t)16 << 10) / (a.dim * Type<GT>::kSize);
  g.zero_each = each < 1 ? 1 : each > 64 ? 64 : (uint32_t)each;
  if (!a.accumulate) g.zeros = (uint32_t)(((a.vocab + g.zero_each - 1) / g.zero_each + kXcds - 1) / kXcds * kXcds);
  for (const uint32_t all = g.sums + g.zeros; g.base < all; g.base += kSumLaunch) {
    const dim3 grid(all - g.base < kSumLaunch ? all - g.base : kSumLaunch), block(kSumWaves * kWave);
    if (a.accumulate) embedding_sum_kernel<ET, GT, true><<<grid, block, 0, stream>>>(a, s, g);
    else embedding_sum_kernel<ET, GT, false><<<grid, block, 0, stream>>>(a, s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.tokens <= kFold) return hipSuccess;
  // a long run has more than kFold tokens
  const size_t join_slabs = (a.dim + kWave - 1) / kWave, items = a.tokens / (kFold + 1) * join_slabs;
  embedding_join_kernel<GT><<<dim3((unsigned)(items < 2048 ? items : 2048)), dim3(kJoinWaves * kWave), 0, stream>>>(
      a, s, (uint32_t)join_slabs);
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
    const LookGradLayout l = look_grad_layout(a.tokens, a.vocab, a.dim);
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
