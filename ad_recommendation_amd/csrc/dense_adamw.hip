// AdamW over many weight tensors in one launch, with states in 32 bits or in 8.
//
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   w = w - lr (m / c1 / (sqrt(v) / sqrt(c2) + eps) + wd w)
// Bound by HBM: everything is read and written once a step, past the caches where it is more than they
// hold (an fp32 step over 96 tensors of 21M elements: 123 -> 114 us; by now 97, 6.0 TB/s).
//
// In 8 bits the states are m and s = sqrt(v), each an e4m3 code times a power of two shared by a block
// of 128: the root halves the exponent range that v needs.  A code is within 1/16 of its value, while
// b2 = 0.999 moves s by at most 0.05 % a step when g falls to zero, so rounding to the nearest would
// leave s where it is for good; both states are rounded up or down at random, in proportion, so that
// their means move as the formula says.  335.6M weights in 64 tensors with bf16 gradients and copies: 994
// us, 5.4 TB/s.
#include <algorithm>

#include "dense_device.h"

// Products and sums round one by one, as the formula is written: the vector path, the element path
// and a program that does the same steps give the same bits.
#pragma clang fp contract(off)

namespace emb {

namespace {

constexpr int kThreads = 256;
static_assert(kAdamChunk == kThreads * 8, "eight elements a thread");

__device__ __forceinline__ uint32_t mix32(uint32_t x) {  // the finaliser of MurmurHash3
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ uint32_t row_max(uint32_t x) {  // over 16 lanes
#define STEP(C) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, C, 0xF, 0xF, false))
  STEP(0x128);
  STEP(0x124);
  STEP(0x122);
  STEP(0x121);
#undef STEP
  return x;
}

// Eight codes as values.
__device__ __forceinline__ f32x8 decode8(uint2 c, int exp) {
  const f32x2 p0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false);
  const f32x2 p1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
  const f32x2 p2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false);
  const f32x2 p3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
  f32x8 x = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = ldexpf(x[i], exp - 127);
  return x;
}

// Eight values of a block, its 16 lanes' 128 in all, as codes; returns the block's exponent + 127.
// `down`: for each value a number in (0, 1), a multiple of 2^-17.  KEEP: a value that is not zero gets a code that
// is not.
template <bool KEEP>
__device__ __forceinline__ int encode8(const f32x8& x, const f32x8& down, uint2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = (uint32_t)__float_as_int(x[i]) & 0x7FFFFFFFu;
    top = max(top, b < 0x7F800000u ? b : 0u);
  }
  top = row_max(top);
  // floor(log2(top)) - 7, within the exponents that a byte holds
  const int k = top ? max(__builtin_amdgcn_frexp_expf(__int_as_float((int)top)) - 8, -127) : -127;
  f32x8 c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = ldexpf(fabsf(x[i]), -k);
    const int e = max(__builtin_amdgcn_frexp_expf(y) - 1, -6);
    // The upper of two codes where the place between them is past `down`.  Both are exact in fp32; a sum with
    // 1 - down would be rounded, onto the border now and then.  On the border itself, which keeps the mean as well
    // either way, the lower.
    const float t = ldexpf(y, 3 - e);
    float q = floorf(t);
    q += t - q > down[i] ? 1.f : 0.f;
    if (KEEP && y > 0.f) q = fmaxf(q, 1.f);
    c[i] = copysignf(ldexpf(q, e - 3), x[i]);
    // infinities and NaN: the one code that e4m3 has for them
    if (!(y < __builtin_huge_valf())) c[i] = __builtin_nanf("");
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  codes = make_uint2((uint32_t)lo, (uint32_t)hi);
  return k + 127;
}

// One element's new m, v (both zero where `in` is false) and weight; returns the root of v.
__device__ __forceinline__ float update(const AdamArgs& a, float g, float wd, bool in, float& m, float& v, float& w) {
  m = m * a.b1 + g * a.omb1;
  v = v * a.b2 + g * g * a.omb2;
  if (!in) m = v = 0.f;
  const float root = sqrtf(v);
  w = w - a.lr * (m * a.inv_c1 / (root * a.inv_c2 + a.eps) + wd * w);
  return root;
}

// One workgroup takes one chunk of one tensor.  The state arrays hold whole blocks of 128, so only w, g
// and the copy have a ragged end.
template <typename G, typename C, bool COPY, bool Q8, bool ONCE>
__global__ void __launch_bounds__(kThreads) adamw(const AdamArgs a) {
  uint32_t lo = 0, hi = a.n_tensors;  // the last tensor whose first chunk is not past this one
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (a.t[mid].chunk0 <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const AdamTensor& t = a.t[lo];
  float* const w = t.w;
  const G* const g = static_cast<const G*>(t.g);
  C* const copy = static_cast<C*>(t.copy);
  const int64_t n = t.n;
  const int64_t n_pad = (n + EMB_ADAMW_BLOCK - 1) & ~(int64_t)(EMB_ADAMW_BLOCK - 1);
  const int64_t s0 = (int64_t)t.block0 * EMB_ADAMW_BLOCK;
  const float wd = t.wd;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int64_t e0 = (int64_t)(blockIdx.x - t.chunk0) * kAdamChunk;

  if constexpr (!Q8) {
    // two vectors of four a thread, each next to its neighbours' in memory
    f32x4 wv[2] = {}, gv[2] = {}, m[2] = {}, v[2] = {};
    int left[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t e = e0 + k * (kAdamChunk / 2) + threadIdx.x * 4;
      left[k] = (int)min(max(n - e, (int64_t)0), (int64_t)4);
      if (left[k] > 0) {
        wv[k] = load4<float, ONCE>(w + e, left[k]);
        gv[k] = load4<G, ONCE>(g + e, left[k]);
        m[k] = load4<float, ONCE>(a.m + s0 + e, 4);
        v[k] = load4<float, ONCE>(a.v + s0 + e, 4);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t e = e0 + k * (kAdamChunk / 2) + threadIdx.x * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mi = m[k][i], vi = v[k][i], wi = wv[k][i];
        update(a, gv[k][i] * gs, wd, i < left[k], mi, vi, wi);
        m[k][i] = mi;
        v[k][i] = vi;
        wv[k][i] = wi;
      }
      if (left[k] > 0) {
        store4<float, ONCE>(w + e, wv[k], left[k]);
        if (COPY) store4<C, ONCE>(copy + e, wv[k], left[k]);
      }
      if (e < n_pad) {
        store4<float, ONCE>(a.m + s0 + e, m[k], 4);
        store4<float, ONCE>(a.v + s0 + e, v[k], 4);
      }
    }
  } else {
    // eight elements a thread: 16 lanes share a block
    const uint32_t seed = mix32(a.seed_lo) ^ a.seed_hi;
    const int64_t e = e0 + threadIdx.x * 8, s = s0 + e;
    const bool in = e < n_pad;  // the same for the 16 lanes
    const int left = (int)min(max(n - e, (int64_t)0), (int64_t)8);
    f32x8 wv = {}, gv = {}, m = {}, v = {}, root;
    if (left > 0) {
      wv = load8<float, ONCE>(w + e, left);
      gv = widen(load8<G, ONCE>(g + e, left));
    }
    if (in) {
      m = decode8(*reinterpret_cast<const uint2*>(a.m8 + s), a.m_exp[s / EMB_ADAMW_BLOCK]);
      v = decode8(*reinterpret_cast<const uint2*>(a.v8 + s), a.v_exp[s / EMB_ADAMW_BLOCK]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float mi = m[i], vi = v[i] * v[i], wi = wv[i];
      root[i] = update(a, gv[i] * gs, wd, i < left, mi, vi, wi);
      m[i] = mi;
      wv[i] = wi;
    }
    if (left > 0) {
      store8<float, ONCE>(w + e, wv, left);
      if (COPY) store8<C, ONCE>(copy + e, wv, left);
    }
    const uint32_t base = mix32(seed ^ (uint32_t)((uint64_t)s >> 32) * 0x9E3779B1u);
    f32x8 down_m, down_v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t r = mix32((uint32_t)(s + i) + base);
      down_m[i] = (65535.5f - (float)(r & 0xFFFFu)) * (1.f / 65536.f);
      down_v[i] = (65535.5f - (float)(r >> 16)) * (1.f / 65536.f);
    }
    uint2 cm, cv;
    const int em = encode8<false>(m, down_m, cm);
    const int ev = encode8<true>(root, down_v, cv);
    if (in) {
      *reinterpret_cast<uint2*>(a.m8 + s) = cm;
      *reinterpret_cast<uint2*>(a.v8 + s) = cv;
      if ((threadIdx.x & 15) == 0) {
        a.m_exp[s / EMB_ADAMW_BLOCK] = (uint8_t)em;
        a.v_exp[s / EMB_ADAMW_BLOCK] = (uint8_t)ev;
      }
    }
  }
}

// The values of codes, for a look at the states or to store them elsewhere: 335.6M to bf16 in 167 us, 6 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) adamw_values(const uint8_t* codes, const uint8_t* exp,
                                                         int64_t elems, T* out) {
  const int64_t stride = (int64_t)gridDim.x * kAdamChunk;
  for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; e < elems; e += stride)
    store8<T, true>(out + e, decode8(*reinterpret_cast<const uint2*>(codes + e), exp[e / EMB_ADAMW_BLOCK]), 8);
}

template <typename G, typename C, bool COPY, bool Q8>
void go(const AdamArgs& a, uint32_t chunks, hipStream_t st) {
  if (a.once) hipLaunchKernelGGL((adamw<G, C, COPY, Q8, true>), dim3(chunks), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((adamw<G, C, COPY, Q8, false>), dim3(chunks), dim3(kThreads), 0, st, a);
}

template <typename G, bool Q8>
void go_copy(const AdamArgs& a, uint32_t chunks, int copy_dtype, hipStream_t st) {
  if (copy_dtype == EMB_F16) go<G, _Float16, true, Q8>(a, chunks, st);
  else if (copy_dtype == EMB_BF16) go<G, __bf16, true, Q8>(a, chunks, st);
  else go<G, _Float16, false, Q8>(a, chunks, st);
}

template <bool Q8>
void go_type(const AdamArgs& a, uint32_t chunks, int grad_dtype, int copy_dtype, hipStream_t st) {
  if (grad_dtype == EMB_F32) go_copy<float, Q8>(a, chunks, copy_dtype, st);
  else if (grad_dtype == EMB_F16) go_copy<_Float16, Q8>(a, chunks, copy_dtype, st);
  else go_copy<__bf16, Q8>(a, chunks, copy_dtype, st);
}

}  // namespace

hipError_t launch_adamw(AdamArgs& a, int64_t elems, uint32_t n_chunks, bool q8, int grad_dtype,
                        int copy_dtype, hipStream_t st) {
  const int each = 8 + (q8 ? 4 : 16) + (grad_dtype == EMB_F32 ? 4 : 2) + (copy_dtype >= 0 ? 2 : 0);
  a.once = elems * each > kOnceBytes;
  if (q8) go_type<true>(a, n_chunks, grad_dtype, copy_dtype, st);
  else go_type<false>(a, n_chunks, grad_dtype, copy_dtype, st);
  return hipGetLastError();
}

hipError_t launch_adamw_values(const uint8_t* codes, const uint8_t* exp, int64_t elems, void* out,
                               int out_dtype, hipStream_t st) {
  const int64_t blocks = (elems + kAdamChunk - 1) / kAdamChunk;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, kAdamChunks)), block(kThreads);
  if (out_dtype == EMB_BF16)
    hipLaunchKernelGGL((adamw_values<__bf16>), grid, block, 0, st, codes, exp, elems, static_cast<__bf16*>(out));
  else
    hipLaunchKernelGGL((adamw_values<float>), grid, block, 0, st, codes, exp, elems, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace emb
