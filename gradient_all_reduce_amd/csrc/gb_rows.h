// gb_rows.h — device helpers shared by the kernels of the token-sum layers
// (gb_norm.hip, gb_embed.hip): 16-byte vectors of one row's values at any
// element alignment, and sums over a group of lanes.  Internal linkage.
#pragma once

#include <hip/hip_runtime.h>

#include "gb_layers.h"

namespace gb {
namespace {

constexpr int kWave = 64;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

#define GB_GLOBAL __attribute__((address_space(1)))
// Rows may be views into a bucket or a wider array, so a vector is aligned to
// its element only.  The under-aligned types are named where the access is
// made: as a template argument a type loses its alignment attribute.
typedef u4 u4_any4 __attribute__((aligned(4)));
typedef u4 u4_any2 __attribute__((aligned(2)));
typedef u2 u2_any2 __attribute__((aligned(2)));

// The canonical quiet NaN, as in every float32 result of the library.
__device__ __forceinline__ float canon(float v) { return v != v ? __uint_as_float(0x7FC00000u) : v; }

template <int ET>
struct Type;
template <>
struct Type<GB_DTYPE_F32> {
  static constexpr int kSize = 4, kVec = 4;  // values of a 16-byte vector
};
template <>
struct Type<GB_DTYPE_F16> {
  static constexpr int kSize = 2, kVec = 8;
};
template <>
struct Type<GB_DTYPE_BF16> {
  static constexpr int kSize = 2, kVec = 8;
};

// ---------------------------------------------------------------------------
// One value
// ---------------------------------------------------------------------------
template <int ET>
__device__ __forceinline__ float half_value(uint32_t h) {
  if constexpr (ET == GB_DTYPE_BF16) return __uint_as_float(h << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
template <int ET>
__device__ __forceinline__ float load_one(const void* p, size_t i) {
  if constexpr (ET == GB_DTYPE_F32) return *((const GB_GLOBAL float*)p + i);
  else return half_value<ET>(*((const GB_GLOBAL uint16_t*)p + i));
}
// v, rounded to nearest even.
template <int ET>
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  if constexpr (ET == GB_DTYPE_BF16) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
  } else {
    // binary32 first, then its rounding: left alone, the compiler may fold the
    // operation that made a value and its conversion into one rounding
    asm volatile("" : "+v"(a), "+v"(b));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
  }
}
template <int ET>
__device__ __forceinline__ void store_one(void* p, size_t i, float v) {
  if constexpr (ET == GB_DTYPE_F32) *((GB_GLOBAL float*)p + i) = v;
  else *((GB_GLOBAL uint16_t*)p + i) = (uint16_t)half_pair<ET>(v, v);
}
__device__ __forceinline__ float load_any(const void* p, int dtype, size_t i) {
  if (dtype == GB_DTYPE_F32) return load_one<GB_DTYPE_F32>(p, i);
  return dtype == GB_DTYPE_F16 ? load_one<GB_DTYPE_F16>(p, i) : load_one<GB_DTYPE_BF16>(p, i);
}

// ---------------------------------------------------------------------------
// V values at p[i], where left of them (1 or more) lie in the row; zeros
// beyond.  V is 16 bytes' worth, or 4 halves (8 bytes).
// ---------------------------------------------------------------------------
template <int ET, int V>
struct Raw {
  static constexpr int kWords = V * Type<ET>::kSize / 4;
  uint32_t w[kWords];
};
// The address of value i.  Of 32 bits, i is a lane's offset from an address
// that the wavefront shares, which the load or store instruction adds itself.
template <int ET, class I>
__device__ __forceinline__ const GB_GLOBAL char* value_at(const void* p, I i) {
  return (const GB_GLOBAL char*)p + (I)(i * Type<ET>::kSize);
}
template <int ET, class I>
__device__ __forceinline__ GB_GLOBAL char* value_at(void* p, I i) {
  return (GB_GLOBAL char*)p + (I)(i * Type<ET>::kSize);
}
template <int ET, int V, bool NT, class I>
__device__ __forceinline__ Raw<ET, V> load_full(const void* p, I i) {
  Raw<ET, V> r;
  if constexpr (Type<ET>::kSize == 4) {
    static_assert(V == 4, "");
    const GB_GLOBAL u4_any4* q = (const GB_GLOBAL u4_any4*)value_at<ET>(p, i);
    u4 v;
    if constexpr (NT) v = __builtin_nontemporal_load(q);
    else v = *q;
#pragma unroll
    for (int j = 0; j < 4; j++) r.w[j] = v[j];
  } else if constexpr (V == 8) {
    const GB_GLOBAL u4_any2* q = (const GB_GLOBAL u4_any2*)value_at<ET>(p, i);
    u4 v;
    if constexpr (NT) v = __builtin_nontemporal_load(q);
    else v = *q;
#pragma unroll
    for (int j = 0; j < 4; j++) r.w[j] = v[j];
  } else {
    static_assert(V == 4, "");
    const GB_GLOBAL u2_any2* q = (const GB_GLOBAL u2_any2*)value_at<ET>(p, i);
    u2 v;
    if constexpr (NT) v = __builtin_nontemporal_load(q);
    else v = *q;
    r.w[0] = v.x, r.w[1] = v.y;
  }
  return r;
}
template <int ET, int V, bool NT, class I>
__device__ __forceinline__ Raw<ET, V> load_raw(const void* p, I i, uint32_t left) {
  if (left >= V) return load_full<ET, V, NT>(p, i);
  Raw<ET, V> r;
#pragma unroll
  for (int j = 0; j < Raw<ET, V>::kWords; j++) r.w[j] = 0u;
#pragma unroll
  for (int e = 0; e < V - 1; e++) {
    if (e < (int)left) {
      if constexpr (Type<ET>::kSize == 4) r.w[e] = *((const GB_GLOBAL uint32_t*)p + i + e);
      else r.w[e / 2] |= (uint32_t)*((const GB_GLOBAL uint16_t*)p + i + e) << (16 * (e & 1));
    }
  }
  return r;
}
template <int ET, int V>
__device__ __forceinline__ Raw<ET, V> zero_raw() {
  Raw<ET, V> r;
#pragma unroll
  for (int j = 0; j < Raw<ET, V>::kWords; j++) r.w[j] = 0u;
  return r;
}
template <int ET, int V>
__device__ __forceinline__ float raw_value(const Raw<ET, V>& r, int e) {
  if constexpr (Type<ET>::kSize == 4) return __uint_as_float(r.w[e]);
  else if constexpr (ET == GB_DTYPE_BF16)
    return __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
  else return (float)__builtin_bit_cast(h2, r.w[e / 2])[e & 1];
}

template <int ET, int V, bool NT, class I>
__device__ __forceinline__ void store_vals(void* p, I i, uint32_t left, const float (&v)[V]) {
  if (left >= V) {
    if constexpr (Type<ET>::kSize == 4) {
      static_assert(V % 4 == 0, "");
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const u4 w = {__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                      __float_as_uint(v[j + 3])};
        GB_GLOBAL u4_any4* q = (GB_GLOBAL u4_any4*)value_at<ET>(p, (I)(i + j));
        if constexpr (NT) __builtin_nontemporal_store(w, q);
        else *q = w;
      }
    } else if constexpr (V == 8) {
      const u4 w = {half_pair<ET>(v[0], v[1]), half_pair<ET>(v[2], v[3]), half_pair<ET>(v[4], v[5]),
                    half_pair<ET>(v[6], v[7])};
      GB_GLOBAL u4_any2* q = (GB_GLOBAL u4_any2*)value_at<ET>(p, i);
      if constexpr (NT) __builtin_nontemporal_store(w, q);
      else *q = w;
    } else {
      const u2 w = {half_pair<ET>(v[0], v[1]), half_pair<ET>(v[2], v[3])};
      GB_GLOBAL u2_any2* q = (GB_GLOBAL u2_any2*)value_at<ET>(p, i);
      if constexpr (NT) __builtin_nontemporal_store(w, q);
      else *q = w;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < V - 1; e++) {
    if (e < (int)left) store_one<ET>(p, i + e, v[e]);
  }
}

// Values of col within a row of cols that a vector starting there covers.
__device__ __forceinline__ uint32_t left_of(uint32_t col, uint32_t cols) { return col < cols ? cols - col : 0u; }

// ---------------------------------------------------------------------------
// Sum over aligned groups of L lanes, the same bits in each of them (a
// butterfly: at every step both partners add the same two numbers).  All
// lanes of the wavefront must be active.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v += dpp<0xB1>(v);   // quad_perm 1,0,3,2
  if constexpr (L >= 4) v += dpp<0x4E>(v);   // quad_perm 2,3,0,1
  if constexpr (L >= 8) v += dpp<0x141>(v);  // row_half_mirror
  if constexpr (L >= 16) v += dpp<0x140>(v); // row_mirror
  if constexpr (L >= 32) {
    // swaps the odd rows of 16 lanes of one operand with the even rows of the other
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

}  // namespace
}  // namespace gb
