// Device helpers of the dense side's kernels: element types, vectors of eight, sums over lanes.
#pragma once

#include <hip/hip_runtime.h>

#include "dense_internal.h"

namespace emb {

// Data of a call beyond this, the size of the cache in front of HBM, is read and written past the
// caches (ONCE below): nothing of it would be found there again.  Backward of the norms, 20011 x 2048 in
// bf16, 492 MB: 100 -> 94 us; 5003 x 333 in fp32, 53 MB: 19 -> 24 us.
constexpr int64_t kOnceBytes = 256ll << 20;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <typename T> struct Vec8;
template <> struct Vec8<float> { typedef f32x8 t; };
template <> struct Vec8<_Float16> { typedef f16x8 t; };
template <> struct Vec8<__bf16> { typedef bf16x8 t; };

template <typename T, int N> using Vec = T __attribute__((ext_vector_type(N)));

// N elements at p as they are.  `n` of them exist; the others are zero and are not read.  p need only be
// aligned to its elements: global memory takes 16-byte accesses at any address.
// ONCE: what nothing reads again soon, and what the caches need not keep (a nontemporal access).
template <int N, typename T, bool ONCE = false>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p, int n) {
  typedef Vec<T, N> V;
  typedef V U __attribute__((aligned(sizeof(T))));
  if (n >= N) {
    if (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const U*>(p));
    return *reinterpret_cast<const U*>(p);
  }
  V v = {};
#pragma unroll
  for (int i = 0; i < N - 1; ++i)
    if (i < n) v[i] = p[i];
  return v;
}
// Rounds N values to T (nearest even) and writes the first n.
template <int N, typename T, bool ONCE = false>
__device__ __forceinline__ void store_vec(T* p, Vec<float, N> x, int n) {
  typedef Vec<T, N> V;
  typedef V U __attribute__((aligned(sizeof(T))));
  const V v = __builtin_convertvector(x, V);
  if (n >= N) {
    if (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<U*>(p));
    else *reinterpret_cast<U*>(p) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < N - 1; ++i)
    if (i < n) p[i] = v[i];
}
template <typename T, bool ONCE = false>
__device__ __forceinline__ typename Vec8<T>::t load8(const T* p, int n) {
  return load_vec<8, T, ONCE>(p, n);
}
template <typename T, bool ONCE = false>
__device__ __forceinline__ void store8(T* p, f32x8 x, int n) {
  store_vec<8, T, ONCE>(p, x, n);
}

template <typename T, bool ONCE>
__device__ __forceinline__ f32x4 load4(const T* p, int n) {
  return __builtin_convertvector((load_vec<4, T, ONCE>(p, n)), f32x4);
}
template <typename T, bool ONCE>
__device__ __forceinline__ void store4(T* p, f32x4 x, int n) {
  store_vec<4, T, ONCE>(p, x, n);
}

template <typename V>
__device__ __forceinline__ f32x8 widen(V v) {
  return __builtin_convertvector(v, f32x8);
}

// ---------------------------------------------------------------- sums over lanes
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float swap16_sum(float x) {  // with the neighbouring row of 16 lanes
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_int(x), __float_as_int(x), false, false);
  return __int_as_float(r[0]) + __int_as_float(r[1]);
}
__device__ __forceinline__ float swap32_sum(float x) {  // with the other half of the wave
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_int(x), __float_as_int(x), false, false);
  return __int_as_float(r[0]) + __int_as_float(r[1]);
}
__device__ __forceinline__ float swap32_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_int(x), __float_as_int(x), false, false);
  return fmaxf(__int_as_float(r[0]), __int_as_float(r[1]));
}
// The sum over each group of N lanes (8, 16, 32 or 64), in every lane of it and the same bits there:
// exchanges within rows of 16 lanes on the vector unit, then swaps of rows and halves; no LDS.
template <int N>
__device__ __forceinline__ float lanes_sum(float x) {
  if (N == 8) {
    x += dpp<0x141>(x);  // row_half_mirror: with lane 7 - i of the eight
    x += dpp<0xB1>(x);   // quad_perm: with lane i ^ 1
    return x + dpp<0x4E>(x);  // i ^ 2
  }
  x += dpp<0x128>(x);  // row_ror:8
  x += dpp<0x124>(x);
  x += dpp<0x122>(x);
  x += dpp<0x121>(x);
  if (N >= 32) x = swap16_sum(x);
  if (N >= 64) x = swap32_sum(x);
  return x;
}

}  // namespace emb
