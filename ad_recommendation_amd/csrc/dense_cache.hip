// Caches of keys and values in 8 bits: written as events come in, and read back.
//
// A row is one token's head: with the exponent k = floor(log2(largest |x|)) - 7 its elements are x 2^-k, the
// largest in [128, 256), rounded to the nearest e4m3 code (ties to even).  Powers of two lose nothing of a
// floating-point code, so which scale a row has decides no rounding, and x 2^-k is exact.
//
// Memory bound: a lane has eight elements, a row up to 16 lanes whose maximum goes round on the vector unit.
#include <type_traits>

#include "dense_shared_device.h"

namespace emb {

namespace {

constexpr int kRowsAtOnce = 4;  // of a lane, all loaded before the first is used

// The largest over each group of N lanes, in every lane of it.
template <int N>
__device__ __forceinline__ float lanes_max(float x) {
  if (N >= 16) x = fmaxf(x, dpp<0x128>(x));  // row_ror:8
  if (N >= 8) x = fmaxf(x, dpp<0x141>(x));   // row_half_mirror: with lane 7 - i of the eight
  if (N >= 2) x = fmaxf(x, dpp<0xB1>(x));    // i ^ 1
  if (N >= 4) x = fmaxf(x, dpp<0x4E>(x));    // i ^ 2
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
        f32x8 y = widen(x[n]);
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]) < kInf ? fabsf(y[e]) : 0.f);
        top = lanes_max<LANES>(top);
        const int k = top > 0.f ? max(__builtin_amdgcn_frexp_expf(top) - 8, -127) : -127;
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
