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

struct Place {
  int64_t tok;   // packed
  int64_t at;    // in the cache, or -1
  int seq, head, which;
};
// Row `row` of a workgroup's tokens: heads of keys, heads of values, then the next token's.
__device__ __forceinline__ Place place_of(const CacheArgs& a, const Seq& s, int64_t start, int tile, int row) {
  const int per = 2 * a.heads, t = row / per, x = row - t * per;
  Place p;
  p.which = x >= a.heads;
  p.head = x - p.which * a.heads;
  p.seq = s.index;
  const int64_t i = (int64_t)s.tile * tile + t;
  p.tok = s.begin + i;
  p.at = start + i;
  if (p.at < 0 || p.at >= a.capacity) p.at = -1;
  return p;
}

template <typename T> constexpr int kTopExp = std::is_same<T, _Float16>::value ? 8 : 120;

// Tokens of a workgroup: the same for every width and type.
constexpr int kTokens = 8;

template <typename T, int LANES, bool WRITE>
__global__ void __launch_bounds__(256) cache_q8(CacheArgs a) {
  typedef typename Vec8<T>::t V8;
  Seq s;
  if (a.off) {
    s = find_tile(a, blockIdx.x, [](int64_t t, int b) { return t / kTokens + b; });
    if (s.tile < 0 || (int64_t)s.tile * kTokens >= s.len) return;
  } else {
    s.index = blockIdx.x;
    s.begin = s.index;
    s.len = 1;
    s.tile = 0;
  }
  const int64_t start = a.start ? a.start[s.index] : 0;
  const int rows = min(kTokens, s.len - s.tile * kTokens) * 2 * a.heads;
  constexpr int kGroups = 256 / LANES;
  const int group = threadIdx.x / LANES, col = threadIdx.x % LANES * 8;
  const bool inside = col < a.dim;
  for (int row0 = group; row0 < rows; row0 += kGroups * kRowsAtOnce) {
    if constexpr (WRITE) {
      V8 x[kRowsAtOnce];
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        const int row = row0 + n * kGroups;
        x[n] = V8{};
        if (row < rows && inside) {
          const Place p = place_of(a, s, start, kTokens, row);
          const EmbHeads& h = a.x[p.which];
          x[n] = *reinterpret_cast<const V8*>(static_cast<const T*>(h.p) + p.tok * h.tok + p.head * h.head + col);
        }
      }
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        const int row = row0 + n * kGroups;
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
        for (int w = 0; w < 2; ++w) {
          const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w], y[4 * w + 1], 0, false);
          c[w] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w + 2], y[4 * w + 3], lo, true);
        }
        if (row >= rows) continue;
        const Place p = place_of(a, s, start, kTokens, row);
        if (p.at < 0) continue;
        const EmbHeads &h = a.code[p.which], &g = a.exp[p.which];
        if (inside)
          *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(h.p) + p.seq * h.seq + p.at * h.tok + p.head * h.head +
                                    col) = c;
        if (col == 0) static_cast<uint8_t*>(g.p)[p.seq * g.seq + p.at * g.tok + p.head * g.head] = (uint8_t)(k + 127);
      }
    } else {
      u32x2 c[kRowsAtOnce];
      uint32_t ex[kRowsAtOnce];
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        const int row = row0 + n * kGroups;
        c[n] = u32x2{0, 0};
        ex[n] = 0;
        if (row >= rows || !inside) continue;
        const Place p = place_of(a, s, start, kTokens, row);
        if (p.at < 0) continue;
        const EmbHeads &h = a.code[p.which], &g = a.exp[p.which];
        c[n] = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(h.p) + p.seq * h.seq + p.at * h.tok +
                                               p.head * h.head + col);
        ex[n] = static_cast<const uint8_t*>(g.p)[p.seq * g.seq + p.at * g.tok + p.head * g.head];
      }
#pragma unroll
      for (int n = 0; n < kRowsAtOnce; ++n) {
        const int row = row0 + n * kGroups;
        if (row >= rows || !inside) continue;
        const Place p = place_of(a, s, start, kTokens, row);
        V8 y;
        if constexpr (std::is_same<T, float>::value) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const f32x2 u = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[n][w], false);
            const f32x2 v = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[n][w], true);
            y[4 * w] = u[0], y[4 * w + 1] = u[1], y[4 * w + 2] = v[0], y[4 * w + 3] = v[1];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = ex[n] == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(y[e], (int)ex[n] - 127);
        } else {
          y = of_codes<T>(c[n], ex[n]);
        }
        const EmbHeads& h = a.x[p.which];
        *reinterpret_cast<V8*>(static_cast<T*>(h.p) + p.tok * h.tok + p.head * h.head + col) = y;
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
    if (write) hipLaunchKernelGGL((cache_q8<T, LANES, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((cache_q8<T, LANES, false>), grid, dim3(256), 0, st, a);
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
