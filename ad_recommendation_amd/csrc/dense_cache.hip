// Caches of keys and values in 8 bits: written as events come in, and read back.
//
// A row is one token's head: with the exponent k = floor(log2(largest |x|)) - 7 its elements are x 2^-k, the
// largest in [128, 256), rounded to the nearest e4m3 code (ties to even).  Powers of two lose nothing of a
// floating-point code, so which scale a row has decides no rounding, and x 2^-k is exact.
//
// Memory bound: a lane has eight elements, a row up to 16 lanes whose maximum goes round on the vector unit.  With a test
// of every element, a limit and a scaling of its own the vector unit was as busy as memory; the maximum of bits and a
// conversion that scales do without in the common case, and what is rare (numbers that are not finite, exponents at T's
// ends) goes another way: writing and reading back 64 histories of up to 8191 events, 8 heads of 128, bf16, took 745 us,
// and takes 693 at 5.2 TB/s.
#include <type_traits>

#include "dense_shared_device.h"

namespace emb {

namespace {

constexpr int kRowsAtOnce = 4;  // of a lane, all loaded before the first is used

// The largest over each group of N lanes, in every lane of it.  Bits of numbers without their sign: in the order of
// the numbers, with what is not finite above them.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  auto from = [&](auto how) {
    return __builtin_bit_cast(uint32_t, dpp<decltype(how)::value>(__builtin_bit_cast(float, x)));
  };
  if (N >= 16) x = max(x, from(std::integral_constant<int, 0x128>{}));  // row_ror:8
  if (N >= 8) x = max(x, from(std::integral_constant<int, 0x141>{}));   // row_half_mirror: with lane 7 - i of the eight
  if (N >= 2) x = max(x, from(std::integral_constant<int, 0xB1>{}));    // i ^ 1
  if (N >= 4) x = max(x, from(std::integral_constant<int, 0x4E>{}));    // i ^ 2
  return x;
}

// A lane's rows of a workgroup's tokens: heads of keys, heads of values, then the next token's; `step` rows on each
// time, without a division.
struct Walk {
  int t, x;       // token of the workgroup's, row of the token
  int dt, dx, per;
  __device__ __forceinline__ Walk(int row, int step, int heads) {
    per = 2 * heads;
    t = (uint32_t)row / (uint32_t)per;
    x = row - t * per;
    dt = (uint32_t)step / (uint32_t)per;
    dx = step - dt * per;
  }
  __device__ __forceinline__ void next() {
    t += dt;
    x += dx;
    if (x >= per) {
      x -= per;
      ++t;
    }
  }
};

template <typename T> constexpr int kTopExp = std::is_same<T, _Float16>::value ? 8 : 120;

// The largest |x|, as bits of a T.
__device__ __forceinline__ uint32_t largest(f32x8 x) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, fabsf(x[e])));
  return m;
}
template <typename V8>
__device__ __forceinline__ uint32_t largest(V8 x) {
  typedef uint16_t U2 __attribute__((ext_vector_type(2)));
  const u32x4 w = __builtin_bit_cast(u32x4, x);
  U2 m = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(U2, w[e] & 0x7fff7fffu));
  return max(m[0], m[1]);
}
template <typename T>
__device__ __forceinline__ float of_bits(uint32_t x) {
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, x);
  else return (float)__builtin_bit_cast(T, (uint16_t)x);
}

// Codes of x 2^-k; all finite, below 2^(k + 8).
__device__ __forceinline__ u32x2 codes_of(f32x8 x, int k) {
  const float by = __builtin_amdgcn_ldexpf(1.f, -k);
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i] * by, x[4 * i + 1] * by, 0, false);
    c[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2] * by, x[4 * i + 3] * by, lo, true);
  }
  return c;
}
__device__ __forceinline__ u32x2 codes_of(f16x8 x, int k) {
  const float by = __builtin_amdgcn_ldexpf(1.f, k);  // which the conversion divides by
  typedef short S2 __attribute__((ext_vector_type(2)));
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    S2 t = {};
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(t, f16x2{x[4 * i], x[4 * i + 1]}, by, false);
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(t, f16x2{x[4 * i + 2], x[4 * i + 3]}, by, true);
    c[i] = __builtin_bit_cast(uint32_t, t);
  }
  return c;
}
__device__ __forceinline__ u32x2 codes_of(bf16x8 x, int k) {
  const float by = __builtin_amdgcn_ldexpf(1.f, k);  // which the conversion divides by
  typedef short S2 __attribute__((ext_vector_type(2)));
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    S2 t = {};
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(t, bf16x2{x[4 * i], x[4 * i + 1]}, by, false);
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(t, bf16x2{x[4 * i + 2], x[4 * i + 3]}, by, true);
    c[i] = __builtin_bit_cast(uint32_t, t);
  }
  return c;
}

// The same of any numbers, with the row's exponent.
template <typename T, int LANES>
__device__ u32x2 odd_codes(typename Vec8<T>::t x, int& k) {
  f32x8 y = widen(x);
  f32x8 finite = y;
#pragma unroll
  for (int e = 0; e < 8; ++e) finite[e] = fabsf(y[e]) < kInf ? y[e] : 0.f;
  const float top = of_bits<float>(lanes_max<LANES>(largest(finite)));
  k = top > 0.f ? max(__builtin_amdgcn_frexp_expf(top) - 8, -127) : -127;
  // 256 times the largest power is past T's numbers
  const float most = k == kTopExp<T> ? 240.f : 256.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float z = __builtin_amdgcn_ldexpf(y[e], -k);
    y[e] = fabsf(y[e]) < kInf ? fminf(fmaxf(z, -most), most) : __builtin_nanf("");
  }
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
    c[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], lo, true);
  }
  return c;
}

// Tokens of a workgroup: enough rows that finding its sequence costs little.
constexpr int kTokens = 32;

template <typename T, int LANES, bool WRITE, bool ONCE>
__global__ void __launch_bounds__(256) cache_q8(CacheArgs a) {
  typedef typename Vec8<T>::t V8;
  Seq s;
  if (a.off) {
    s = uniform(find_tile(a, blockIdx.x, [](int64_t t, int b) { return t / kTokens + b; }));
    if (s.tile < 0 || (int64_t)s.tile * kTokens >= s.len) return;
  } else {
    s.index = blockIdx.x;
    s.begin = s.index;
    s.len = 1;
    s.tile = 0;
  }
  const int t0 = s.tile * kTokens, tokens = min(kTokens, s.len - t0);
  const int64_t tok0 = s.begin + t0, at0 = (a.start ? uniform(a.start[s.index]) : 0) + (int64_t)t0;
  constexpr int kGroups = 256 / LANES;
  const int col = threadIdx.x % LANES * 8;
  const bool inside = col < a.dim;
  Walk here(threadIdx.x / LANES, kGroups, a.heads);
  auto in_cache = [&](const Walk& w) { return at0 + w.t >= 0 && at0 + w.t < a.capacity; };
  auto value_at = [&](const Walk& w) {
    const bool v = w.x >= a.heads;
    const EmbHeads& h = a.x[v];
    return static_cast<T*>(h.p) + (tok0 + w.t) * h.tok + (w.x - (v ? a.heads : 0)) * h.head + col;
  };
  auto cached = [&](const EmbHeads* c, const Walk& w) {
    const bool v = w.x >= a.heads;
    const EmbHeads& h = c[v];
    return static_cast<uint8_t*>(h.p) + s.index * h.seq + (at0 + w.t) * h.tok + (w.x - (v ? a.heads : 0)) * h.head;
  };
  while (here.t < tokens) {
    Walk w = here;
    if constexpr (WRITE) {
      V8 x[kRowsAtOnce];
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        x[n] = V8{};
        if (w.t < tokens && inside) x[n] = load8<T, ONCE>(value_at(w), 8);
        w.next();
      }
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        const float top = of_bits<T>(lanes_max<LANES>(largest(x[n])));
        int k = top > 0.f ? __builtin_amdgcn_frexp_expf(top) - 8 : -127;
        u32x2 c;
        // most rows are finite, and neither so large that a code may pass T's numbers nor cut off below
        if (__any(!(top < kInf) || k >= kTopExp<T> || (k < -126 && top > 0.f))) c = odd_codes<T, LANES>(x[n], k);
        else c = codes_of(x[n], max(k, -126));
        if (here.t < tokens && in_cache(here)) {
          if (inside) {
            u32x2* to = reinterpret_cast<u32x2*>(cached(a.code, here) + col);
            if (ONCE) __builtin_nontemporal_store(c, to);
            else *to = c;
          }
          if (col == 0) *cached(a.exp, here) = (uint8_t)(k + 127);
        }
        here.next();
      }
    } else {
      u32x2 c[kRowsAtOnce];
      uint32_t ex[kRowsAtOnce];
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        c[n] = u32x2{0, 0};
        ex[n] = 0;
        if (w.t < tokens && inside && in_cache(w)) {
          const u32x2* from = reinterpret_cast<const u32x2*>(cached(a.code, w) + col);
          c[n] = ONCE ? __builtin_nontemporal_load(from) : *from;
          ex[n] = *cached(a.exp, w);
        }
        w.next();
      }
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        V8 y;
        if constexpr (std::is_same<T, float>::value) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x2 u = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[n][i], false);
            const f32x2 v = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[n][i], true);
            y[4 * i] = u[0], y[4 * i + 1] = u[1], y[4 * i + 2] = v[0], y[4 * i + 3] = v[1];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = ex[n] == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(y[e], (int)ex[n] - 127);
        } else {
          y = of_codes<T>(c[n], ex[n]);
        }
        if (here.t < tokens && inside) {
          V8* to = reinterpret_cast<V8*>(value_at(here));
          if (ONCE) __builtin_nontemporal_store(y, to);
          else *to = y;
        }
        here.next();
      }
    }
  }
}

int64_t blocks(const CacheArgs& a) { return a.off ? a.n_tok / kTokens + a.n_seq : a.n_seq; }

}  // namespace

int64_t cache_threads(const CacheArgs& a) { return blocks(a) * 256; }

hipError_t launch_cache(const CacheArgs& a, bool write, hipStream_t st) {
  const dim3 grid((unsigned)blocks(a));
  auto go = [&](auto t, auto lanes) {
    typedef decltype(t) T;
    constexpr int LANES = decltype(lanes)::value;
    const bool once = 2 * a.n_tok * a.heads * a.dim * (int64_t)(sizeof(T) + 1) > kOnceBytes;
    if (write && once) hipLaunchKernelGGL((cache_q8<T, LANES, true, true>), grid, dim3(256), 0, st, a);
    else if (write) hipLaunchKernelGGL((cache_q8<T, LANES, true, false>), grid, dim3(256), 0, st, a);
    else if (once) hipLaunchKernelGGL((cache_q8<T, LANES, false, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((cache_q8<T, LANES, false, false>), grid, dim3(256), 0, st, a);
  };
  auto by_lanes = [&](auto t) {
    if (a.dim <= 8) go(t, std::integral_constant<int, 1>{});
    else if (a.dim <= 16) go(t, std::integral_constant<int, 2>{});
    else if (a.dim <= 32) go(t, std::integral_constant<int, 4>{});
    else if (a.dim <= 64) go(t, std::integral_constant<int, 8>{});
    else go(t, std::integral_constant<int, 16>{});
  };
  if (a.dtype == EMB_F32) by_lanes(float{});
  else if (a.dtype == EMB_F16) by_lanes(_Float16{});
  else by_lanes(__bf16{});
  return hipGetLastError();
}

}  // namespace emb
