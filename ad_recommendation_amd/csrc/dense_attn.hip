// Attention of ragged event sequences with a sliding window and a few first keys that stay visible:
// forward, backward and the form for one new event against a cache.
//
//   see(i, j) = j <= i and (i - j < window or j < sinks)
//   s_ij = scale q_i . k_j;  p_ij = exp(s_ij - lse_i);  out_i = sum_j p_ij v_j
//   delta_i = out_i . dout_i;  ds_ij = scale p_ij (dout_i . v_j - delta_i)
//   dq_i = sum_j ds_ij k_j;  dk_j = sum_i ds_ij q_i;  dv_j = sum_i p_ij dout_i
#include "dense_device.h"

namespace emb {

namespace {

// One wave a row; a lane holds two of the row's dimensions.
struct Pair {
  float a, b;
};
template <typename T>
__device__ __forceinline__ Pair get(const EmbHeads& t, int64_t seq, int64_t tok, int h, int D) {
  const int d = (threadIdx.x & 63) * 2;
  if (d >= D) return Pair{0.f, 0.f};
  const T* p = static_cast<const T*>(t.p) + seq * t.seq + tok * t.tok + h * t.head + d;
  return Pair{(float)p[0], (float)p[1]};
}
template <typename T>
__device__ __forceinline__ void put(const EmbHeads& t, int64_t tok, int h, int D, Pair x) {
  const int d = (threadIdx.x & 63) * 2;
  if (d >= D) return;
  T* p = static_cast<T*>(t.p) + tok * t.tok + h * t.head + d;
  p[0] = (T)x.a;
  p[1] = (T)x.b;
}
__device__ __forceinline__ float dot(Pair x, Pair y) { return lanes_sum<64>(x.a * y.a + x.b * y.b); }

// The sequence that token t belongs to, by its offsets clamped to [0, n_tok]; false if none does.
__device__ __forceinline__ bool find_seq(const AttnArgs& a, int64_t t, int64_t& begin, int64_t& len) {
  int lo = 0, hi = a.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.off[mid] <= t) lo = mid;
    else hi = mid;
  }
  begin = min(max((int64_t)a.off[lo], (int64_t)0), a.n_tok);
  const int64_t end = min(max((int64_t)a.off[lo + 1], (int64_t)0), a.n_tok);
  len = end - begin;
  return t >= begin && t < end;
}

// The next key that row i sees after j.
__device__ __forceinline__ int64_t next_key(const AttnArgs& a, int64_t i, int64_t j) {
  ++j;
  return j >= a.sinks && i - j >= a.window ? i - a.window + 1 : j;
}

template <typename T>
__device__ __forceinline__ void row_fwd(const AttnArgs& a, Pair q, int64_t seq, int64_t begin,
                                        int64_t i, int kh, Pair& o, float& m, float& l) {
  o = Pair{0.f, 0.f};
  m = -__builtin_huge_valf();
  l = 0.f;
  for (int64_t j = next_key(a, i, -1); j <= i; j = next_key(a, i, j)) {
    const float s = dot(q, get<T>(a.k, seq, begin + j, kh, a.dim)) * a.scale;
    const Pair v = get<T>(a.v, seq, begin + j, kh, a.dim);
    const float mn = fmaxf(m, s);
    const float c = l > 0.f ? __expf(m - mn) : 0.f, p = __expf(s - mn);
    o.a = o.a * c + p * v.a;
    o.b = o.b * c + p * v.b;
    l = l * c + p;
    m = mn;
  }
  if (l > 0.f) {
    o.a /= l;
    o.b /= l;
  }
}

template <typename T>
__global__ void __launch_bounds__(64) attn_fwd(AttnArgs a) {
  for (int64_t b = blockIdx.x; b < a.n_tok * a.q_heads; b += gridDim.x) {
    const int64_t t = b / a.q_heads;
    const int h = (int)(b % a.q_heads);
    int64_t begin, len;
    if (!find_seq(a, t, begin, len)) continue;
    Pair o;
    float m, l;
    row_fwd<T>(a, get<T>(a.q, 0, t, h, a.dim), 0, begin, t - begin, h / (a.q_heads / a.kv_heads), o, m, l);
    put<T>(a.out, t, h, a.dim, o);
    if (a.lse && threadIdx.x == 0) a.lse[h * a.n_tok + t] = m + __logf(l);
  }
}

template <typename T>
__global__ void __launch_bounds__(64) attn_decode(AttnArgs a) {
  for (int64_t b = blockIdx.x; b < (int64_t)a.n_seq * a.q_heads; b += gridDim.x) {
    const int64_t s = b / a.q_heads;
    const int h = (int)(b % a.q_heads);
    const int64_t len = min(max((int64_t)a.off[s], (int64_t)0), a.n_tok);
    Pair o;
    float m, l;
    row_fwd<T>(a, get<T>(a.q, 0, s, h, a.dim), s, 0, len - 1, h / (a.q_heads / a.kv_heads), o, m, l);
    put<T>(a.out, s, h, a.dim, o);
  }
}

template <typename T>
__global__ void __launch_bounds__(64) attn_dq(AttnArgs a) {
  for (int64_t b = blockIdx.x; b < a.n_tok * a.q_heads; b += gridDim.x) {
    const int64_t t = b / a.q_heads;
    const int h = (int)(b % a.q_heads), kh = h / (a.q_heads / a.kv_heads);
    int64_t begin, len;
    if (!find_seq(a, t, begin, len)) continue;
    const int64_t i = t - begin;
    const Pair q = get<T>(a.q, 0, t, h, a.dim), d = get<T>(a.dout, 0, t, h, a.dim);
    const float delta = dot(d, get<T>(a.out, 0, t, h, a.dim)), lse = a.lse[h * a.n_tok + t];
    if (threadIdx.x == 0) a.delta[h * a.n_tok + t] = delta;
    Pair o{0.f, 0.f};
    for (int64_t j = next_key(a, i, -1); j <= i; j = next_key(a, i, j)) {
      const Pair k = get<T>(a.k, 0, begin + j, kh, a.dim);
      const float p = __expf(dot(q, k) * a.scale - lse);
      const float ds = p * (dot(d, get<T>(a.v, 0, begin + j, kh, a.dim)) - delta) * a.scale;
      o.a += ds * k.a;
      o.b += ds * k.b;
    }
    put<T>(a.dq, t, h, a.dim, o);
  }
}

template <typename T>
__global__ void __launch_bounds__(64) attn_dkv(AttnArgs a) {
  const int group = a.q_heads / a.kv_heads;
  for (int64_t b = blockIdx.x; b < a.n_tok * a.kv_heads; b += gridDim.x) {
    const int64_t t = b / a.kv_heads;
    const int kh = (int)(b % a.kv_heads);
    int64_t begin, len;
    if (!find_seq(a, t, begin, len)) continue;
    const int64_t j = t - begin;
    const Pair k = get<T>(a.k, 0, t, kh, a.dim), v = get<T>(a.v, 0, t, kh, a.dim);
    Pair dk{0.f, 0.f}, dv{0.f, 0.f};
    const int64_t end = j < a.sinks ? len : min(len, j + a.window);
    for (int h = kh * group; h < (kh + 1) * group; ++h) {
      for (int64_t i = j; i < end; ++i) {
        const Pair q = get<T>(a.q, 0, begin + i, h, a.dim), d = get<T>(a.dout, 0, begin + i, h, a.dim);
        const float p = __expf(dot(q, k) * a.scale - a.lse[h * a.n_tok + begin + i]);
        const float ds = p * (dot(d, v) - a.delta[h * a.n_tok + begin + i]) * a.scale;
        dv.a += p * d.a;
        dv.b += p * d.b;
        dk.a += ds * q.a;
        dk.b += ds * q.b;
      }
    }
    put<T>(a.dk, t, kh, a.dim, dk);
    put<T>(a.dv, t, kh, a.dim, dv);
  }
}

dim3 grid_of(int64_t n) { return dim3((unsigned)(n < (1 << 20) ? n : (1 << 20))); }

}  // namespace

AttnBwdPlan plan_attn_bwd(const EmbAttn& a, int64_t n_seq, int64_t n_tok) {
  AttnBwdPlan p{};
  p.off_part = ((size_t)n_tok * a.q_heads * sizeof(float) + 255) & ~(size_t)255;
  p.bytes = p.off_part;
  return p;
}

AttnDecodePlan plan_attn_decode(const EmbAttn& a, int64_t n_seq, int64_t capacity) {
  return AttnDecodePlan{1, 0};
}

#define BY_TYPE(K, GRID)                                                                        \
  do {                                                                                          \
    if (a.dtype == EMB_F16) hipLaunchKernelGGL((K<_Float16>), GRID, dim3(64), 0, st, a);         \
    else hipLaunchKernelGGL((K<__bf16>), GRID, dim3(64), 0, st, a);                              \
  } while (0)

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st) {
  BY_TYPE(attn_fwd, grid_of(a.n_tok * a.q_heads));
  return hipGetLastError();
}
hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st) {
  BY_TYPE(attn_dq, grid_of(a.n_tok * a.q_heads));
  BY_TYPE(attn_dkv, grid_of(a.n_tok * a.kv_heads));
  return hipGetLastError();
}
hipError_t launch_attn_decode(const AttnArgs& a, const AttnDecodePlan&, hipStream_t st) {
  BY_TYPE(attn_decode, grid_of((int64_t)a.n_seq * a.q_heads));
  return hipGetLastError();
}

}  // namespace emb
