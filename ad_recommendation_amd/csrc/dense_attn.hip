// Attention of ragged event sequences with a sliding window and a few first keys that stay visible:
// forward, backward and the form for one new event against a cache.
//
//   see(i, j) = j <= i and (i - j < window or j < sinks)
//   s_ij = scale q_i . k_j;  p_ij = exp(s_ij - lse_i);  out_i = sum_j p_ij v_j
//   delta_i = out_i . dout_i;  ds_ij = scale p_ij (dout_i . v_j - delta_i)
//   dq_i = sum_j ds_ij k_j;  dk_j = sum_i ds_ij q_i;  dv_j = sum_i p_ij dout_i
//
// All products run on the matrix cores as 32x32x16 with fp32 sums.  A product's result has a column
// in a lane and 16 of its 32 rows (8 (r / 4) + 4 (lane / 32) + r % 4 for register r) in that lane's
// registers, and a right operand has a column in a lane and eight consecutive k of 16 there.  The
// kernels put what the softmax runs over into rows (keys where a lane has a query, queries where it
// has a key), so that statistics and rescaling stay within a lane and its partner 32 lanes on, and
// the probabilities become the next product's right operand as they are: which row of the sum
// stands at which k is free as long as the left operand agrees, and the left operand comes out of
// LDS by transposing reads, four rows at any address at a time.
#include <algorithm>
#include <type_traits>

#include "dense_device.h"

namespace emb {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kThreads = 256;
constexpr int kQTile = 128;  // tokens of a workgroup: 32 for each of its four waves
constexpr int kStageRows = 64;  // rows of an LDS tile

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mma(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }
// The row of a result that register r of this lane holds.
__device__ __forceinline__ int row_of(int r) { return 8 * (r >> 2) + 4 * (lane_id() >> 5) + (r & 3); }

// ---------------------------------------------------------------- work items
struct Seq {
  int64_t begin;  // first token
  int len, tile;  // tokens; which tile of the sequence this workgroup has
  int index;
};
// Tile slot s of a ragged batch: sequence b's tiles start at slot off[b] / tile + extra * b, which
// leaves every sequence room for ceil(len / tile) + extra - 1 tiles without a pass over the
// lengths.  64 lanes look for the sequence together.  Offsets are clamped to the tokens.
__device__ __forceinline__ Seq find_tile(const AttnArgs& a, int slot, int tile, int extra) {
  auto start = [&](int b) {
    return min(max((int64_t)a.off[b], (int64_t)0), a.n_tok) / tile + (int64_t)extra * b;
  };
  int lo = 0, n = a.n_seq;
  while (n > 1) {
    const int step = (n + 63) >> 6, k = lane_id() * step;
    const bool at_or_before = k < n && start(lo + k) <= slot;
    const int c = max(__popcll(__ballot(at_or_before)), 1) - 1;
    lo += c * step;
    n = min(step, n - c * step);
    lo = __builtin_amdgcn_readfirstlane(lo);
    n = __builtin_amdgcn_readfirstlane(n);
  }
  Seq s;
  s.index = lo;
  s.begin = min(max((int64_t)a.off[lo], (int64_t)0), a.n_tok);
  const int64_t end = min(max((int64_t)a.off[lo + 1], s.begin), a.n_tok);
  s.len = (int)(end - s.begin);
  s.tile = (int)max((int64_t)slot - (s.begin / tile + (int64_t)extra * lo), (int64_t)-1);
  return s;
}

__device__ __forceinline__ bool sees(const AttnArgs& a, int i, int j) {
  return j <= i && (i - j < a.window || j < a.sinks);
}

// ---------------------------------------------------------------- LDS tiles
// Rows of DH elements in 16-byte pieces, a row's pieces exchanged by its number so that the eight or
// more rows which one read touches lie in different banks.
template <int DH>
struct Tile {
  static constexpr int kPieces = DH / 8;
  static constexpr int kBytes = kStageRows * DH * 2;
  static constexpr int kRegs = kStageRows * kPieces / kThreads;
  __device__ static __forceinline__ int at(int row, int piece) {
    const int x = kPieces >= 8 ? row & 7 : (row >> 1) & 3;
    return (row * kPieces + (piece ^ x)) * 16;
  }
};

template <int DH>
struct Staged {
  u32x4 r[Tile<DH>::kRegs];
  // Rows row0 .. row0 + 63 of a head; zeros past `len` rows and past D columns.
  template <typename T>
  __device__ __forceinline__ void load(const T* base, int64_t stride, int row0, int len, int D) {
#pragma unroll
    for (int n = 0; n < Tile<DH>::kRegs; ++n) {
      const int idx = threadIdx.x + n * kThreads;
      const int row = row0 + idx / Tile<DH>::kPieces, col = idx % Tile<DH>::kPieces * 8;
      r[n] = u32x4{0, 0, 0, 0};
      if (row < len && col < D) r[n] = *reinterpret_cast<const u32x4*>(base + row * stride + col);
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int n = 0; n < Tile<DH>::kRegs; ++n) {
      const int idx = threadIdx.x + n * kThreads;
      *reinterpret_cast<u32x4*>(lds + Tile<DH>::at(idx / Tile<DH>::kPieces, idx % Tile<DH>::kPieces)) = r[n];
    }
  }
};

// Left operand: rows row0 .. row0 + 31, columns 16 ks .. 16 ks + 15 as k.
template <typename T, int DH>
__device__ __forceinline__ typename Vec8<T>::t left(const char* lds, int row0, int ks) {
  const int l = lane_id();
  return *reinterpret_cast<const typename Vec8<T>::t*>(lds + Tile<DH>::at(row0 + (l & 31), 2 * ks + (l >> 5)));
}
// Left operand, transposed: columns 32 db .. 32 db + 31 as rows, rows row0 .. row0 + 15 as k, in the
// order in which a result's registers hold them.
template <typename T, int DH>
__device__ __forceinline__ typename Vec8<T>::t left_t(const char* lds, int row0, int db) {
  const int l = lane_id();
  const int row = row0 + 4 * (l >> 5) + ((l & 15) >> 2);
  const int piece = db * 4 + ((l >> 4) & 1) * 2 + ((l & 3) >> 1);
  typedef __attribute__((address_space(3))) i16x4* Lds;
  const char* p0 = lds + Tile<DH>::at(row, piece) + (l & 1) * 8;
  const char* p1 = lds + Tile<DH>::at(row + 8, piece) + (l & 1) * 8;
  const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p0);
  const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p1);
  const i16x8 v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(typename Vec8<T>::t, v);
}

// Right operands of a token's row, one per 16 columns: a lane's row, columns 16 ks + 8 (lane / 32).
template <typename T, int DH>
__device__ __forceinline__ void right_row(const EmbHeads& t, int64_t tok, int head, bool live, int D,
                                          typename Vec8<T>::t (&f)[DH / 16]) {
  const T* p = static_cast<const T*>(t.p) + tok * t.tok + head * t.head;
#pragma unroll
  for (int ks = 0; ks < DH / 16; ++ks) {
    const int col = ks * 16 + (lane_id() >> 5) * 8;
    f[ks] = typename Vec8<T>::t{};
    if (live && col < D) f[ks] = *reinterpret_cast<const typename Vec8<T>::t*>(p + col);
  }
}
// Eight registers of a result as the right operand of the next product, rounded to T: a product's
// operands have 16 bits, and its sum is fp32 again.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::t right_of(const float* p) {
  const f32x8 x = {p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
  return __builtin_convertvector(x, typename Vec8<T>::t);
}

// Writes a lane's row from results that hold it as a column (one per 32 of its elements).
template <typename T, int DH>
__device__ __forceinline__ void store_row(const EmbHeads& t, int64_t tok, int head, int D,
                                          const f32x16 (&x)[DH / 32], float by) {
  typedef T V __attribute__((ext_vector_type(4)));
  T* p = static_cast<T*>(t.p) + tok * t.tok + head * t.head;
#pragma unroll
  for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = db * 32 + 8 * g + 4 * (lane_id() >> 5);
      const f32x4 v = {x[db][4 * g] * by, x[db][4 * g + 1] * by, x[db][4 * g + 2] * by, x[db][4 * g + 3] * by};
      if (col < D) *reinterpret_cast<V*>(p + col) = __builtin_convertvector(v, V);
    }
  }
}

// ---------------------------------------------------------------- what is not finite
// A product adds 0 * x for a pair that does not see each other, which is NaN where x is not finite.
// A row whose sums come out not finite is therefore computed once more from the pairs that see each
// other alone, by the whole wave, two dimensions a lane: it costs nothing while values are finite.
struct Pair {
  float a, b;
};
template <typename T>
__device__ __forceinline__ Pair get(const EmbHeads& t, int64_t tok, int h, int D) {
  const int d = lane_id() * 2;
  if (d >= D) return Pair{0.f, 0.f};
  const T* p = static_cast<const T*>(t.p) + tok * t.tok + h * t.head + d;
  return Pair{(float)p[0], (float)p[1]};
}
template <typename T>
__device__ __forceinline__ void put(const EmbHeads& t, int64_t tok, int h, int D, Pair x, float by) {
  const int d = lane_id() * 2;
  if (d >= D) return;
  T* p = static_cast<T*>(t.p) + tok * t.tok + h * t.head + d;
  p[0] = (T)(x.a * by);
  p[1] = (T)(x.b * by);
}
__device__ __forceinline__ float dot(Pair x, Pair y) { return lanes_sum<64>(x.a * y.a + x.b * y.b); }

template <int N>
__device__ __forceinline__ bool not_finite(const f32x16 (&x)[N]) {
  float z = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) z = fmaf(x[n][r], 0.f, z);
  return z != 0.f;
}
// Whether a lane or its partner says so: one bit for each of the 32 rows or columns.
__device__ __forceinline__ uint32_t either(bool b) {
  const uint64_t m = __ballot(b);
  return (uint32_t)m | (uint32_t)(m >> 32);
}

// The next key that row i sees after j.
__device__ __forceinline__ int next_key(const AttnArgs& a, int i, int j) {
  ++j;
  return j >= a.sinks && i - j >= a.window ? i - a.window + 1 : j;
}
template <typename T>
__device__ __forceinline__ void again_fwd(const AttnArgs& a, int64_t begin, int i, int h, int kh) {
  const Pair q = get<T>(a.q, begin + i, h, a.dim);
  Pair o{0.f, 0.f};
  float m = -kInf, l = 0.f;
  for (int j = next_key(a, i, -1); j <= i; j = next_key(a, i, j)) {
    const float s = dot(q, get<T>(a.k, begin + j, kh, a.dim)) * a.scale;
    const Pair v = get<T>(a.v, begin + j, kh, a.dim);
    const float mn = fmaxf(m, s);
    const float by = m == -kInf ? 0.f : expf(m - mn), p = expf(s - mn);
    o.a = o.a * by + p * v.a;
    o.b = o.b * by + p * v.b;
    l = l * by + p;
    m = mn;
  }
  put<T>(a.out, begin + i, h, a.dim, o, 1.f / l);
}
template <typename T>
__device__ __forceinline__ void again_dq(const AttnArgs& a, int64_t begin, int i, int h, int kh) {
  const Pair q = get<T>(a.q, begin + i, h, a.dim), d = get<T>(a.dout, begin + i, h, a.dim);
  const int64_t stat = (int64_t)h * a.n_tok + begin + i;
  const float delta = dot(d, get<T>(a.out, begin + i, h, a.dim)), lse = a.lse[stat];
  Pair o{0.f, 0.f};
  for (int j = next_key(a, i, -1); j <= i; j = next_key(a, i, j)) {
    const Pair k = get<T>(a.k, begin + j, kh, a.dim);
    const float p = expf(dot(q, k) * a.scale - lse);
    const float ds = p * (dot(d, get<T>(a.v, begin + j, kh, a.dim)) - delta);
    o.a += ds * k.a;
    o.b += ds * k.b;
  }
  put<T>(a.dq, begin + i, h, a.dim, o, a.scale);
}
// Key j's unscaled sums over rows j .. end - 1, of which it is seen by all.
template <typename T>
__device__ __forceinline__ void again_dkv(const AttnArgs& a, int64_t begin, int j, int end, int kh,
                                          Pair& dk, Pair& dv) {
  const Pair k = get<T>(a.k, begin + j, kh, a.dim), v = get<T>(a.v, begin + j, kh, a.dim);
  const int group = a.q_heads / a.kv_heads;
  dk = dv = Pair{0.f, 0.f};
  for (int h = kh * group; h < (kh + 1) * group; ++h) {
    for (int i = j; i < end; ++i) {
      const Pair q = get<T>(a.q, begin + i, h, a.dim), d = get<T>(a.dout, begin + i, h, a.dim);
      const int64_t stat = (int64_t)h * a.n_tok + begin + i;
      const float p = expf(dot(q, k) * a.scale - a.lse[stat]);
      const float ds = p * (dot(d, v) - a.delta[stat]);
      dv.a += p * d.a;
      dv.b += p * d.b;
      dk.a += ds * q.a;
      dk.b += ds * q.b;
    }
  }
}

// ---------------------------------------------------------------- which keys a query tile meets
// Tiles of 64 keys: the one that holds the sinks where the window does not reach it, then the
// window's.
struct KeyTiles {
  int first, n, sink;
  __device__ __forceinline__ KeyTiles(const AttnArgs& a, int i0, int len) {
    const int end = min(len, i0 + kQTile);
    first = max(i0 - a.window + 1, 0) & ~(kStageRows - 1);
    sink = a.sinks > 0 && first > 0 ? 1 : 0;
    n = (end - first + kStageRows - 1) / kStageRows + sink;
  }
  __device__ __forceinline__ int key0(int it) const {
    return it < sink ? 0 : first + (it - sink) * kStageRows;
  }
};

// ---------------------------------------------------------------- forward
template <typename T, int DH>
__global__ void __launch_bounds__(kThreads, 2) attn_fwd(AttnArgs a) {
  typedef typename Vec8<T>::t V8;
  __shared__ __attribute__((aligned(16))) char lds[2][2][Tile<DH>::kBytes];
  const int group = a.q_heads / a.kv_heads;
  const int kh = blockIdx.x % a.kv_heads;
  const int rest = blockIdx.x / a.kv_heads;
  const int h = kh * group + rest % group;
  const Seq s = find_tile(a, rest / group, kQTile, 1);
  if (s.tile < 0 || (int64_t)s.tile * kQTile >= s.len) return;
  const int i0 = s.tile * kQTile;
  const int iw = __builtin_amdgcn_readfirstlane(i0 + (threadIdx.x >> 6) * 32);
  const int i = iw + (lane_id() & 31);
  const bool live = i < s.len;

  V8 q[DH / 16];
  right_row<T, DH>(a.q, s.begin + i, h, live && a.scale != 0.f, a.dim, q);
  // the running maximum is one of q . k, so a negative scale turns q around and a scale of zero
  // leaves zeros
  if (a.scale < 0.f) {
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) q[ks] = -q[ks];
  }
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;

  const KeyTiles tiles(a, i0, s.len);
  const T* kp = static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head;
  Staged<DH> ks_, vs_;
  ks_.load(kp, a.k.tok, tiles.key0(0), s.len, a.dim);
  vs_.load(vp, a.v.tok, tiles.key0(0), s.len, a.dim);

  f32x16 o[DH / 32] = {};
  float m = -kInf, l = 0.f;  // the maximum that o and l stand at, and this lane's half of the sum
  for (int it = 0; it < tiles.n; ++it) {
    char* kt = lds[it & 1][0];
    char* vt = lds[it & 1][1];
    ks_.store(kt);
    vs_.store(vt);
    if (it + 1 < tiles.n) {
      ks_.load(kp, a.k.tok, tiles.key0(it + 1), s.len, a.dim);
      vs_.load(vp, a.v.tok, tiles.key0(it + 1), s.len, a.dim);
    }
    __syncthreads();
    const int j0 = tiles.key0(it);
    if (iw >= s.len || j0 > iw + 31) continue;
    if (j0 >= a.sinks && j0 + 63 <= iw - a.window) continue;

    f32x16 sc[2] = {};
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) {
      sc[0] = mma(left<T, DH>(kt, 0, ks), q[ks], sc[0]);
      sc[1] = mma(left<T, DH>(kt, 32, ks), q[ks], sc[1]);
    }
    if (j0 + 63 > iw || j0 < iw + 31 - a.window + 1) {
#pragma unroll
      for (int r = 0; r < 32; ++r)
        if (!sees(a, i, j0 + (r >> 4) * 32 + row_of(r & 15))) sc[r >> 4][r & 15] = -kInf;
    }
    float top = sc[0][0];
#pragma unroll
    for (int r = 1; r < 32; ++r) top = fmaxf(top, sc[r >> 4][r & 15]);
    top = swap32_max(top);
    // o and l move to a new maximum only when it is over 2^8 times the old one's exponential: below
    // that the probabilities stay small enough for 16 bits and the sums for 32
    if (__any((top - m) * c > 8.f)) {
      const float mn = fmaxf(m, top);
      const float by = m == -kInf ? 0.f : exp2f((m - mn) * c);
      m = mn;
      l *= by;
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] *= by;
    }
    const float off = m == -kInf ? 0.f : m * c;
    float p[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      p[r] = __builtin_amdgcn_exp2f(fmaf(sc[r >> 4][r & 15], c, -off));
      l += p[r];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const V8 pb = right_of<T>(p + 8 * k);
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T, DH>(vt, 16 * k, db), pb, o[db]);
    }
  }
  l = swap32_sum(l);
  uint32_t again = either(live && not_finite(o));
  if (live && !(again >> (lane_id() & 31) & 1)) store_row<T, DH>(a.out, s.begin + i, h, a.dim, o, 1.f / l);
  if (live && a.lse && lane_id() < 32)
    a.lse[(int64_t)h * a.n_tok + s.begin + i] = m * c * kLn2 + logf(l);
  for (; again; again &= again - 1) again_fwd<T>(a, s.begin, iw + __builtin_ctz(again), h, kh);
}

// ---------------------------------------------------------------- backward: dq
// As the forward, with dout as a second right operand; also writes delta.
template <typename T, int DH>
__global__ void __launch_bounds__(kThreads, 2) attn_dq(AttnArgs a) {
  typedef typename Vec8<T>::t V8;
  __shared__ __attribute__((aligned(16))) char lds[2][2][Tile<DH>::kBytes];
  const int group = a.q_heads / a.kv_heads;
  const int kh = blockIdx.x % a.kv_heads;
  const int rest = blockIdx.x / a.kv_heads;
  const int h = kh * group + rest % group;
  const Seq s = find_tile(a, rest / group, kQTile, 1);
  if (s.tile < 0 || (int64_t)s.tile * kQTile >= s.len) return;
  const int i0 = s.tile * kQTile;
  const int iw = __builtin_amdgcn_readfirstlane(i0 + (threadIdx.x >> 6) * 32);
  const int i = iw + (lane_id() & 31);
  const bool live = i < s.len;

  const KeyTiles tiles(a, i0, s.len);
  const T* kp = static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head;
  Staged<DH> ks_, vs_;
  ks_.load(kp, a.k.tok, tiles.key0(0), s.len, a.dim);
  vs_.load(vp, a.v.tok, tiles.key0(0), s.len, a.dim);

  V8 q[DH / 16], d[DH / 16];
  right_row<T, DH>(a.q, s.begin + i, h, live, a.dim, q);
  right_row<T, DH>(a.dout, s.begin + i, h, live, a.dim, d);
  float delta = 0.f;
  {
    V8 out[DH / 16];
    right_row<T, DH>(a.out, s.begin + i, h, live, a.dim, out);
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta += (float)out[ks][e] * (float)d[ks][e];
    delta = swap32_sum(delta);
  }
  const int64_t stat = (int64_t)h * a.n_tok + s.begin + i;
  if (live && lane_id() < 32) a.delta[stat] = delta;
  const float c = a.scale * kLog2e;
  const float lse = live ? a.lse[stat] * kLog2e : kInf;

  f32x16 dq[DH / 32] = {};
  for (int it = 0; it < tiles.n; ++it) {
    char* kt = lds[it & 1][0];
    char* vt = lds[it & 1][1];
    ks_.store(kt);
    vs_.store(vt);
    if (it + 1 < tiles.n) {
      ks_.load(kp, a.k.tok, tiles.key0(it + 1), s.len, a.dim);
      vs_.load(vp, a.v.tok, tiles.key0(it + 1), s.len, a.dim);
    }
    __syncthreads();
    const int j0 = tiles.key0(it);
    if (iw >= s.len) continue;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int js = j0 + 32 * sub;
      if (js > iw + 31 || (js >= a.sinks && js + 31 <= iw - a.window)) continue;
      f32x16 sc = {}, dp = {};
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks) {
        sc = mma(left<T, DH>(kt, 32 * sub, ks), q[ks], sc);
        dp = mma(left<T, DH>(vt, 32 * sub, ks), d[ks], dp);
      }
      float ds[16];
#pragma unroll
      for (int r = 0; r < 16; ++r)
        ds[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -lse)) * (dp[r] - delta);
      if (js + 31 > iw || js < iw + 31 - a.window + 1) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!sees(a, i, js + row_of(r))) ds[r] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const V8 b = right_of<T>(ds + 8 * k);
#pragma unroll
        for (int db = 0; db < DH / 32; ++db)
          dq[db] = mma(left_t<T, DH>(kt, 32 * sub + 16 * k, db), b, dq[db]);
      }
    }
  }
  uint32_t again = either(live && not_finite(dq));
  if (live && !(again >> (lane_id() & 31) & 1)) store_row<T, DH>(a.dq, s.begin + i, h, a.dim, dq, a.scale);
  for (; again; again &= again - 1) again_dq<T>(a, s.begin, iw + __builtin_ctz(again), h, kh);
}

// ---------------------------------------------------------------- backward: dk, dv
// A workgroup has 128 keys of a key/value head, 32 a wave, and meets the queries of every head of its
// group that see them; sums stay in registers, so nothing is added up in memory.  The sinks are
// seen by every later query of their sequence too: those queries, from `reach` on, are cut into
// chunks, each a workgroup whose four waves take its rows in turn for the first 32 keys; its sums and
// those of the first key tile go to memory in fp32, and attn_sink_join adds them in order.
constexpr int kSinkKeys = EMB_ATTN_MAX_SINKS;

__host__ __device__ inline int64_t reach_of(int window) { return (int64_t)kQTile + window - 1; }

template <typename T, int DH>
__global__ void __launch_bounds__(kThreads, DH == 128 ? 1 : 2)
    attn_dkv(AttnArgs a, int main_blocks, int chunk) {
  typedef typename Vec8<T>::t V8;
  struct Shared {
    char q[2][Tile<DH>::kBytes], d[2][Tile<DH>::kBytes];
    float lse[2][kStageRows], delta[2][kStageRows];
  };
  __shared__ __attribute__((aligned(16))) Shared sh;
  const int group = a.q_heads / a.kv_heads;
  const bool sink = (int)blockIdx.x >= main_blocks;  // the same for the whole workgroup
  const int block = sink ? blockIdx.x - main_blocks : blockIdx.x;
  const int kh = block % a.kv_heads, slot = block / a.kv_heads;
  const Seq s = sink ? find_tile(a, slot, chunk, 2) : find_tile(a, slot, kQTile, 1);
  const int64_t reach = reach_of(a.window);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int j0, row0, row1;  // first key; the queries met
  if (s.tile < 0) return;
  if (sink) {
    const int64_t r0 = reach + (int64_t)s.tile * chunk;
    if (r0 >= s.len) return;
    j0 = 0;
    row0 = (int)r0;
    row1 = (int)min(r0 + chunk, (int64_t)s.len);
  } else {
    if ((int64_t)s.tile * kQTile >= s.len) return;
    j0 = s.tile * kQTile;
    row0 = j0;
    row1 = (int)min(j0 + reach, (int64_t)s.len);
  }
  const int jw = sink ? 0 : j0 + 32 * wave;
  const int j = jw + (lane_id() & 31);
  const bool live = j < s.len;

  V8 k[DH / 16], v[DH / 16];
  right_row<T, DH>(a.k, s.begin + j, kh, live, a.dim, k);
  right_row<T, DH>(a.v, s.begin + j, kh, live, a.dim, v);
  const float c = a.scale * kLog2e;

  const int n_tiles = (row1 - row0 + kStageRows - 1) / kStageRows;
  const int steps = n_tiles * group;  // of all heads of the group
  Staged<DH> qs_, ds_;
  float stat = 0.f;  // threads 0-63: lse of a row; 64-127: its delta
  auto load = [&](int step) {
    const int h = kh * group + step / n_tiles, r0 = row0 + step % n_tiles * kStageRows;
    qs_.load(static_cast<const T*>(a.q.p) + s.begin * a.q.tok + h * a.q.head, a.q.tok, r0, row1, a.dim);
    ds_.load(static_cast<const T*>(a.dout.p) + s.begin * a.dout.tok + h * a.dout.head, a.dout.tok,
             r0, row1, a.dim);
    if (threadIdx.x < 2 * kStageRows) {
      const int row = r0 + (threadIdx.x & 63);
      const float* p = threadIdx.x < kStageRows ? a.lse : a.delta;
      stat = row < row1 ? p[(int64_t)h * a.n_tok + s.begin + row] : 0.f;
      // a row that is not there gets probabilities of zero
      if (threadIdx.x < kStageRows) stat = row < row1 ? stat * kLog2e : kInf;
    }
  };
  load(0);
  f32x16 dk[DH / 32] = {}, dv[DH / 32] = {};
  for (int step = 0; step < steps; ++step) {
    const int b = step & 1;
    qs_.store(sh.q[b]);
    ds_.store(sh.d[b]);
    if (threadIdx.x < kStageRows) sh.lse[b][threadIdx.x] = stat;
    else if (threadIdx.x < 2 * kStageRows) sh.delta[b][threadIdx.x - kStageRows] = stat;
    if (step + 1 < steps) load(step + 1);
    __syncthreads();
    const int r0 = row0 + step % n_tiles * kStageRows;
    if (jw >= s.len) continue;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int is = r0 + 32 * sub;
      if (is >= row1) continue;
      if (sink) {
        if (((step * 2 + sub) & 3) != wave) continue;
      } else if (is + 31 < jw || (jw >= a.sinks && is >= jw + 31 + (int64_t)a.window)) {
        continue;
      }
      f32x16 sc = {}, dp = {};
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks) {
        sc = mma(left<T, DH>(sh.q[b], 32 * sub, ks), k[ks], sc);
        dp = mma(left<T, DH>(sh.d[b], 32 * sub, ks), v[ks], dp);
      }
      float p[16], ds[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int at = 32 * sub + 8 * g + 4 * (lane_id() >> 5);
        const f32x4 lse = *reinterpret_cast<const f32x4*>(&sh.lse[b][at]);
        const f32x4 delta = *reinterpret_cast<const f32x4*>(&sh.delta[b][at]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[4 * g + e] = __builtin_amdgcn_exp2f(fmaf(sc[4 * g + e], c, -lse[e]));
          ds[4 * g + e] = p[4 * g + e] * (dp[4 * g + e] - delta[e]);
        }
      }
      if (is < jw + 31 || (int64_t)is + 31 - jw >= a.window) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!sees(a, is + row_of(r), j)) p[r] = ds[r] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const V8 pb = right_of<T>(p + 8 * x), db_ = right_of<T>(ds + 8 * x);
#pragma unroll
        for (int db = 0; db < DH / 32; ++db) {
          dv[db] = mma(left_t<T, DH>(sh.d[b], 32 * sub + 16 * x, db), pb, dv[db]);
          dk[db] = mma(left_t<T, DH>(sh.q[b], 32 * sub + 16 * x, db), db_, dk[db]);
        }
      }
    }
  }
  // partial sums of the sinks: [slot][kv head][2][sinks][dim], the first key tile's in the slot before
  // the sequence's chunks' (slots are two a sequence apart for it)
  const bool split = a.sinks > 0 && reach < s.len;
  const int64_t first_slot = s.begin / chunk + 2 * (int64_t)s.index;
  auto partial = [&](int64_t at) {
    return a.part + (at * a.kv_heads + kh) * 2 * a.sinks * (int64_t)a.dim;
  };
  if (!sink) {
    float* out = partial(first_slot);
    const EmbHeads row{out, 0, a.dim, 0};
    uint32_t again = either(live && (not_finite(dk) || not_finite(dv)));
    if (live && !(again >> (lane_id() & 31) & 1)) {
      if (!split || j >= a.sinks) {
        store_row<T, DH>(a.dk, s.begin + j, kh, a.dim, dk, a.scale);
        store_row<T, DH>(a.dv, s.begin + j, kh, a.dim, dv, 1.f);
      } else {
        store_row<float, DH>(row, j, 0, a.dim, dk, 1.f);
        store_row<float, DH>(row, a.sinks + j, 0, a.dim, dv, 1.f);
      }
    }
    for (; again; again &= again - 1) {
      const int x = jw + __builtin_ctz(again);
      Pair pk, pv;
      again_dkv<T>(a, s.begin, x, x < a.sinks ? row1 : (int)min((int64_t)x + a.window, (int64_t)s.len),
                   kh, pk, pv);
      if (!split || x >= a.sinks) {
        put<T>(a.dk, s.begin + x, kh, a.dim, pk, a.scale);
        put<T>(a.dv, s.begin + x, kh, a.dim, pv, 1.f);
      } else {
        put<float>(row, x, 0, a.dim, pk, 1.f);
        put<float>(row, a.sinks + x, 0, a.dim, pv, 1.f);
      }
    }
    return;
  }
  // the four waves' sums meet in LDS, one wave after the other
  float* acc = reinterpret_cast<float*>(sh.q);  // [32][DH] fp32 of one matrix
  static_assert(sizeof(sh.q) >= sizeof(float) * kSinkKeys * DH, "the sums fit the tiles' LDS");
  float* out = partial(first_slot + 1 + s.tile);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    for (int w = 0; w < 4; ++w) {
      __syncthreads();
      if (wave != w) continue;
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float* p = acc + (lane_id() & 31) * DH + db * 32 + row_of(r);
          const float t = x ? dv[db][r] : dk[db][r];
          *p = w ? *p + t : t;
        }
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.sinks * a.dim; e += kThreads)
      out[x * a.sinks * a.dim + e] = acc[e / a.dim * DH + e % a.dim];
  }
}

// dk and dv of the sinks from the first key tile's sums and every chunk's, in that order.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_sink_join(AttnArgs a, int chunk) {
  const int kh = blockIdx.x % a.kv_heads, b = blockIdx.x / a.kv_heads;
  const int64_t begin = min(max((int64_t)a.off[b], (int64_t)0), a.n_tok);
  const int64_t len = min(max((int64_t)a.off[b + 1], begin), a.n_tok) - begin;
  const int64_t reach = reach_of(a.window);
  if (len <= reach) return;
  const int64_t n = 1 + (len - reach + chunk - 1) / chunk;
  const int64_t each = 2 * a.sinks * (int64_t)a.dim, first = begin / chunk + 2 * (int64_t)b;
  for (int e = threadIdx.x; e < each; e += kThreads) {
    float t = 0.f;
    for (int64_t x = 0; x < n; ++x) t += a.part[((first + x) * a.kv_heads + kh) * each + e];
    const int row = e / a.dim % a.sinks, col = e % a.dim;
    const bool is_v = e >= a.sinks * a.dim;
    const EmbHeads& to = is_v ? a.dv : a.dk;
    T* p = static_cast<T*>(to.p) + (begin + row) * to.tok + kh * to.head;
    p[col] = (T)(is_v ? t : t * a.scale);
  }
}

// ---------------------------------------------------------------- one new event
// The keys that the newest event sees, in one row: the sinks outside the window, then the window.
// A workgroup has a part of them for one key/value head; its waves take tiles of 32 in turn, each
// with a softmax of its own, and meet in LDS at the end.  All query heads of the group are the
// columns of one product, so keys and values are read once.  Memory bound.
template <int DH>
struct WaveTile {  // 32 rows, of one wave
  static constexpr int kRegs = 32 * Tile<DH>::kPieces / 64;
  static constexpr int kBytes = 32 * DH * 2;
};

template <typename T, int DH>
__global__ void __launch_bounds__(kThreads, 2) attn_decode(AttnArgs a, int splits) {
  typedef typename Vec8<T>::t V8;
  __shared__ __attribute__((aligned(16))) char lds[4][2][WaveTile<DH>::kBytes];
  __shared__ float stats[4][2][32];
  const int group = a.q_heads / a.kv_heads;
  const int kh = blockIdx.x % a.kv_heads;
  int rest = blockIdx.x / a.kv_heads;
  const int cols = (group + 31) / 32;  // of query heads, 32 each
  const int col = rest % cols;
  rest /= cols;
  const int split = rest % splits, sq = rest / splits;
  const int len = (int)min(max((int64_t)a.off[sq], (int64_t)0), a.n_tok);
  const int first = max(len - a.window, 0);
  const int n_sink = min(a.sinks, first), n_keys = n_sink + len - first;
  const int per = ((n_keys + splits - 1) / splits + 31) & ~31;
  const int u0 = min(split * per, n_keys), u1 = min(u0 + per, n_keys);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int head = col * 32 + (lane & 31);
  const bool live = head < group;

  V8 q[DH / 16];
  right_row<T, DH>(a.q, sq, kh * group + (live ? head : 0), live && a.scale != 0.f, a.dim, q);
  if (a.scale < 0.f) {
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) q[ks] = -q[ks];
  }
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  const T* kp = static_cast<const T*>(a.k.p) + sq * a.k.seq + kh * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + sq * a.v.seq + kh * a.v.head;
  u32x4 kr[WaveTile<DH>::kRegs], vr[WaveTile<DH>::kRegs];
  auto load = [&](int t0) {
#pragma unroll
    for (int n = 0; n < WaveTile<DH>::kRegs; ++n) {
      const int idx = lane + n * 64;
      const int u = t0 + idx / Tile<DH>::kPieces, cl = idx % Tile<DH>::kPieces * 8;
      kr[n] = vr[n] = u32x4{0, 0, 0, 0};
      if (u < u1 && cl < a.dim) {
        const int64_t key = u < n_sink ? u : first + (u - n_sink);
        kr[n] = *reinterpret_cast<const u32x4*>(kp + key * a.k.tok + cl);
        vr[n] = *reinterpret_cast<const u32x4*>(vp + key * a.v.tok + cl);
      }
    }
  };
  char* kt = lds[wave][0];
  char* vt = lds[wave][1];
  f32x16 o[DH / 32] = {};
  float m = -kInf, l = 0.f;
  int t0 = u0 + wave * 32;
  if (t0 < u1) load(t0);
  for (; t0 < u1; t0 += 128) {
#pragma unroll
    for (int n = 0; n < WaveTile<DH>::kRegs; ++n) {
      const int idx = lane + n * 64;
      const int at = Tile<DH>::at(idx / Tile<DH>::kPieces, idx % Tile<DH>::kPieces);
      *reinterpret_cast<u32x4*>(kt + at) = kr[n];
      *reinterpret_cast<u32x4*>(vt + at) = vr[n];
    }
    if (t0 + 128 < u1) load(t0 + 128);
    // the tile is the wave's own: its LDS accesses are carried out in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    f32x16 sc = {};
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) sc = mma(left<T, DH>(kt, 0, ks), q[ks], sc);
    if (t0 + 32 > u1) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (t0 + row_of(r) >= u1) sc[r] = -kInf;
    }
    float top = sc[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, sc[r]);
    top = swap32_max(top);
    if (__any((top - m) * c > 8.f)) {
      const float mn = fmaxf(m, top);
      const float by = m == -kInf ? 0.f : exp2f((m - mn) * c);
      m = mn;
      l *= by;
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] *= by;
    }
    const float off = m == -kInf ? 0.f : m * c;
    float p[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      p[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -off));
      l += p[r];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const V8 pb = right_of<T>(p + 8 * k);
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T, DH>(vt, 16 * k, db), pb, o[db]);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  l = swap32_sum(l);
  // the waves meet: every wave scales its sums to the common maximum, and they are added in order
  if (lane < 32) {
    stats[wave][0][lane] = m;
    stats[wave][1][lane] = l;
  }
  __syncthreads();
  float top = -kInf, sum = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, stats[w][0][lane & 31]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float mw = stats[w][0][lane & 31];
    if (mw != -kInf) sum += stats[w][1][lane & 31] * exp2f((mw - top) * c);
  }
  const float by = m == -kInf ? 0.f : exp2f((m - top) * c);
  float* acc = reinterpret_cast<float*>(lds);  // [32][DH]
  static_assert(sizeof(lds) >= sizeof(float) * 32 * DH, "the sums fit the tiles' LDS");
  for (int w = 0; w < 4; ++w) {
    __syncthreads();
    if (wave != w) continue;
#pragma unroll
    for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        // a lane's row starts at a piece of its own, so that 32 rows do not share a bank
        float* x = acc + (lane & 31) * DH + ((db * 32 + row_of(r) + (lane & 31)) & (DH - 1));
        const float t = o[db][r] * by;
        *x = w ? *x + t : t;
      }
    }
  }
  __syncthreads();
  // part: [split][sequence][q head][dim] of unscaled sums, then [..][2] of maximum and sum
  const int heads = min(group - col * 32, 32);
  const int64_t total = (int64_t)a.n_seq * a.q_heads;
  if (threadIdx.x < 32) {
    stats[0][0][threadIdx.x] = top;  // every thread has read them: barriers have passed
    stats[0][1][threadIdx.x] = sum;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < heads * a.dim; e += kThreads) {
    const int hd = e / a.dim, d = e % a.dim;
    const int qh = kh * group + col * 32 + hd;
    const float x = acc[hd * DH + ((d + hd) & (DH - 1))];
    if (splits == 1) {
      const float sm = stats[0][1][hd];
      static_cast<T*>(a.out.p)[sq * a.out.tok + qh * a.out.head + d] = (T)(n_keys > 0 ? x / sm : 0.f);
    } else {
      const int64_t row = (int64_t)split * total + (int64_t)sq * a.q_heads + qh;
      a.part[row * a.dim + d] = x;
      if (d == 0) {
        float* st = a.part + (int64_t)splits * total * a.dim + row * 2;
        st[0] = stats[0][0][hd] * c;
        st[1] = stats[0][1][hd];
      }
    }
  }
}

// One wave a (sequence, query head): the splits' sums at their common maximum.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_decode_join(AttnArgs a, int splits) {
  const int64_t total = (int64_t)a.n_seq * a.q_heads;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= total) return;
  const float* st = a.part + (int64_t)splits * total * a.dim;
  float top = -kInf, sum = 0.f;
  for (int x = 0; x < splits; ++x) top = fmaxf(top, st[(x * total + row) * 2]);
  float o[2] = {0.f, 0.f};
  for (int x = 0; x < splits; ++x) {
    const float m = st[(x * total + row) * 2];
    const float by = m == -kInf ? 0.f : exp2f(m - top);
    sum += by * st[(x * total + row) * 2 + 1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = lane_id() + 64 * e;
      if (d < a.dim) o[e] += by * a.part[(x * total + row) * a.dim + d];
    }
  }
  const int64_t sq = row / a.q_heads, qh = row % a.q_heads;
  const bool none = a.off[sq] <= 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = lane_id() + 64 * e;
    if (d < a.dim)
      static_cast<T*>(a.out.p)[sq * a.out.tok + qh * a.out.head + d] = (T)(none ? 0.f : o[e] / sum);
  }
}

// ---------------------------------------------------------------- launches
template <typename F>
void by_shape(const AttnArgs& a, F f) {
  // the widths that kernels are built for; a head of another is padded with zeros in LDS
#define ATTN_DIMS(T)                                                                    \
  do {                                                                                  \
    if (a.dim <= 32) f(T{}, std::integral_constant<int, 32>{});                         \
    else if (a.dim <= 64) f(T{}, std::integral_constant<int, 64>{});                    \
    else f(T{}, std::integral_constant<int, 128>{});                                    \
  } while (0)
  if (a.dtype == EMB_F16) ATTN_DIMS(_Float16);
  else ATTN_DIMS(__bf16);
#undef ATTN_DIMS
}

// Rows of a sink chunk: 512, more where a batch is so long that its chunks would be over a thousand.
int sink_chunk(int64_t n_tok) {
  int64_t c = 512;
  while (n_tok / c > 1024) c *= 2;
  return (int)c;
}
// Whether a sequence of this batch can be longer than what its first key tile meets.
bool has_sink_chunks(int32_t sinks, int32_t window, int64_t n_tok) {
  return sinks > 0 && n_tok > reach_of(window);
}

}  // namespace

AttnBwdPlan plan_attn_bwd(const EmbAttn& a, int64_t n_seq, int64_t n_tok) {
  AttnBwdPlan p{};
  p.off_part = ((size_t)n_tok * a.q_heads * sizeof(float) + 255) & ~(size_t)255;
  p.bytes = p.off_part;
  if (a.sinks > 0)  // for any window
    p.bytes += (size_t)(n_tok / sink_chunk(n_tok) + 2 * n_seq + 1) * a.kv_heads * 2 * a.sinks * a.dim * sizeof(float);
  return p;
}

// Parts of a sequence's keys: where sequences and heads alone leave compute units idle, up to four
// tiles (one a wave) each.
AttnDecodePlan plan_attn_decode(const EmbAttn& a, int64_t n_seq, int64_t capacity) {
  AttnDecodePlan p{};
  const int64_t keys = std::min<int64_t>(capacity, (int64_t)a.window + a.sinks);
  const int64_t group = a.q_heads / a.kv_heads, base = std::max<int64_t>(n_seq * a.kv_heads * ((group + 31) / 32), 1);
  const int64_t most = std::max<int64_t>((keys + 127) / 128, 1);
  p.splits = (int32_t)std::min<int64_t>(most, std::max<int64_t>(1024 / base, 1));
  p.bytes = p.splits > 1 ? (size_t)p.splits * n_seq * a.q_heads * (a.dim + 2) * sizeof(float) : 0;
  return p;
}

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st) {
  by_shape(a, [&](auto t, auto d) {
    const unsigned grid = (unsigned)((a.n_tok / kQTile + a.n_seq) * a.q_heads);
    hipLaunchKernelGGL((attn_fwd<decltype(t), decltype(d)::value>), dim3(grid), dim3(kThreads), 0, st, a);
  });
  return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st) {
  by_shape(a, [&](auto t, auto d) {
    typedef decltype(t) T;
    const int64_t slots = a.n_tok / kQTile + a.n_seq;
    hipLaunchKernelGGL((attn_dq<T, decltype(d)::value>), dim3((unsigned)(slots * a.q_heads)),
                       dim3(kThreads), 0, st, a);
    const int chunk = sink_chunk(a.n_tok);
    const bool sinks = has_sink_chunks(a.sinks, a.window, a.n_tok);
    const int64_t sink_slots = sinks ? a.n_tok / chunk + 2 * a.n_seq : 0;
    hipLaunchKernelGGL((attn_dkv<T, decltype(d)::value>),
                       dim3((unsigned)((slots + sink_slots) * a.kv_heads)), dim3(kThreads), 0, st, a,
                       (int)(slots * a.kv_heads), chunk);
    if (sinks)
      hipLaunchKernelGGL((attn_sink_join<T>), dim3((unsigned)(a.n_seq * a.kv_heads)), dim3(kThreads), 0,
                         st, a, chunk);
  });
  return hipGetLastError();
}

hipError_t launch_attn_decode(const AttnArgs& a, const AttnDecodePlan& p, hipStream_t st) {
  by_shape(a, [&](auto t, auto d) {
    typedef decltype(t) T;
    const int64_t cols = (a.q_heads / a.kv_heads + 31) / 32;
    hipLaunchKernelGGL((attn_decode<T, decltype(d)::value>),
                       dim3((unsigned)(a.n_seq * a.kv_heads * cols * p.splits)), dim3(kThreads), 0, st, a,
                       p.splits);
    if (p.splits > 1)
      hipLaunchKernelGGL((attn_decode_join<T>), dim3((unsigned)(((int64_t)a.n_seq * a.q_heads + 3) / 4)),
                         dim3(kThreads), 0, st, a, p.splits);
  });
  return hipGetLastError();
}

}  // namespace emb
