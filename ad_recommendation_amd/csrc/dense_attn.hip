// Attention of ragged event sequences with a sliding window and a few first keys that stay visible:
// forward, backward and the form for one new event against a cache.
//
//   see(i, j) = j <= i and (i - j < window or j < sinks)
//   s_ij = scale q_i . k_j;  p_ij = exp(s_ij - lse_i);  out_i = sum_j p_ij v_j
//   delta_i = out_i . dout_i;  ds_ij = scale p_ij (dout_i . v_j - delta_i)
//   dq_i = sum_j ds_ij k_j;  dk_j = sum_i ds_ij q_i;  dv_j = sum_i p_ij dout_i
//
// The products, tiles and their layouts are those of dense_attn_device.h.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "dense_attn_device.h"

namespace emb {

namespace {

// ---------------------------------------------------------------- which keys a query tile meets
// Workgroups of four waves take query tiles from the last to the first: a sequence's first tiles meet the
// fewest keys, and short work at the end leaves fewer units idle (17.2k tokens, 16 heads of 128, window
// 1024: 193 -> 190 us; those of one wave, all short, are 4 us slower that way).

// The tile that holds the sinks where the window's tiles do not reach it, then the window's.
template <int WAVES>
struct KeyTiles {
  static constexpr int kRows = Group<WAVES>::kRows;
  int first, n, sink;
  __device__ __forceinline__ KeyTiles(const AttnArgs& a, int i0, int len) {
    const int end = min(len, i0 + Group<WAVES>::kTokens);
    first = max(i0 - a.window + 1, 0) & ~(kRows - 1);
    sink = a.sinks > 0 && first > 0 ? 1 : 0;
    n = (end - first + kRows - 1) / kRows + sink;
  }
  __device__ __forceinline__ int key0(int it) const { return it < sink ? 0 : first + (it - sink) * kRows; }
  // of a tile that is there for the sinks no other key is looked at
  __device__ __forceinline__ int end(const AttnArgs& a, int it, int len) const {
    return it < sink ? min(a.sinks, len) : len;
  }
};

// ---------------------------------------------------------------- forward
// LDS of the forward and of dq.
template <typename T, int DH, int WAVES, bool DIRECT>
struct QueryShared {
  typedef Group<WAVES> G;
  __attribute__((aligned(256))) char tile[G::kBuffers][2][RegisterTile<T, DH, G::kRows, G::kThreads>::kBytes];
  uint32_t said[WAVES];
  // A wave's own part of the buffers' tiles: of the last one before the steps, of the first one after them.
  __device__ __forceinline__ char* part(int buffer) { return tile[buffer][WAVES == 1 ? 0 : wave() >> 1]; }
  __device__ static __forceinline__ int first() { return WAVES == 1 ? 0 : 32 * (wave() & 1); }
  __device__ static __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
};

// To the wave's 32 queries' sums of what they see of x, the keys or the values, what its elements that are not
// finite add: by weights over zero (SIGN), or by weights that are not finite either, which makes NaN.  (The score
// of a key that is not finite is not; a value's weight of zero counts as one over zero.)
template <typename T, int DH, int WAVES, bool DIRECT, bool SIGN>
__device__ __forceinline__ void add_odd_seen(const AttnArgs& a, const EmbHeads& x,
                                             QueryShared<T, DH, WAVES, DIRECT>& sh, const Seq& s, int kh, int iw,
                                             f32x16 (&sums)[DH / 32]) {
  typedef typename Vec8<T>::t V8;
  typedef Group<WAVES> G;
  typedef TileOf<T, DH, G::kRows, G::kThreads, false, 2> Tile;
  const int i = iw + (lane_id<2>() & 31);
  const KeyTiles<WAVES> tiles(a, s.tile * G::kTokens, s.len);
  const T* p = static_cast<const T*>(x.p) + s.begin * x.tok + kh * x.head;
  const typename Tile::Reads at;
  for (int it = 0; it < tiles.n; ++it) {
    Tile tile;
    __syncthreads();  // the tile before is done with
    tile.load(sh.tile[0][0], p, x.tok, tiles.key0(it), tiles.end(a, it, s.len), a.dim);
    tile.store(sh.tile[0][0]);
    Tile::arrived();
    __syncthreads();
    if (iw >= s.len) continue;
    for (int sub = 0; sub < G::kRows / 32; ++sub) {
      f32x16 none;
      const uint32_t see = hide_keys<2>(a, i, tiles.key0(it) + 32 * sub, none, 0.f);
      for (int k = 0; k < 2; ++k) {
        const V8 one = ones<T>(see >> 8 * k, 0);
#pragma unroll
        for (int db = 0; db < DH / 32; ++db)
          add_odd<T>(sums[db], left_t<T>(sh.tile[0][0], at, 32 * sub + 16 * k, db), one, SIGN ? one : V8{});
      }
    }
  }
}

// The sums of the values that the wave's 32 queries from iw on see, weighed by exp(score - m), and of the weights:
// one pass over the keys with a running maximum and sum for each query.  Keys and values come by tiles through
// LDS, queries stay in registers.  Long sequences are bound by matrix cores and exponentials, which
// are about equally busy (39 and 47 % of the time): 17.2k tokens, 16 query and 2 key/value heads of 128, window
// 1024, bf16: 172 us, 740 TFLOP/s of the pairs that see each other.
template <typename T, int DH, int WAVES, bool DIRECT, int AGAIN>
__device__ __forceinline__ void fwd_sums(const AttnArgs& a, QueryShared<T, DH, WAVES, DIRECT>& sh, const Seq& s, int h,
                                         int kh, int iw, float c, f32x16 (&o)[DH / 32], float& m, float& l) {
  typedef typename Vec8<T>::t V8;
  typedef Group<WAVES> G;
  constexpr bool kDirect = DIRECT && !AGAIN;
  typedef TileOf<T, DH, G::kRows, G::kThreads, kDirect, AGAIN> Tile;
  constexpr int kBytes = sizeof(sh.tile[0][0]);
  constexpr int kSubs = G::kRows / 32;
  const int i = iw + (lane_id<AGAIN>() & 31);
  typedef WaveRows<T, DH, Tile, AGAIN> Rows;
  Rows ql;
  ql.load(a.q, s.begin + iw, h, a.scale != 0.f ? s.len - iw : 0, a.dim);

  const KeyTiles<WAVES> tiles(a, s.tile * G::kTokens, s.len);
  const T* kp = static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head;
  Tile kl, vl;
  auto load = [&](int it, char (*to)[kBytes]) {
    kl.load(to[0], kp, a.k.tok, tiles.key0(it), tiles.end(a, it, s.len), a.dim);
    vl.load(to[1], vp, a.v.tok, tiles.key0(it), tiles.end(a, it, s.len), a.dim);
  };
  load(0, sh.tile[0]);
  const typename Tile::Reads at;
  V8 q[DH / 16];
  ql.to_right(sh.part(G::kBuffers - 1), sh.first(), at, q);
  // the running maximum is one of q . k, so a negative scale turns q around and a scale of zero
  // leaves zeros
  if (a.scale < 0.f) {
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) q[ks] = -q[ks];
  }

#pragma unroll
  for (int db = 0; db < DH / 32; ++db) o[db] = f32x16{};
  m = -kInf;  // the maximum that o and l stand at
  l = 0.f;    // this lane's half of the sum
  auto meet = [&](int it, char (*lds_now)[kBytes], char (*lds_next)[kBytes]) {
    const char* kt = lds_now[0];
    const char* vt = lds_now[1];
    if (G::kBuffers == 1) __syncthreads();  // of one wave: its reads of the tile before have ended
    if (AGAIN && it) load(it, lds_now);
    kl.store(lds_now[0]);
    if constexpr (AGAIN != 0) {
#pragma unroll
      for (int x = 0; x < Tile::kRegs; ++x)
        vl.r[x] = __builtin_bit_cast(u32x4, finite_of<T>(__builtin_bit_cast(V8, vl.r[x])));
    }
    vl.store(lds_now[1]);
    if (!kDirect && !AGAIN && it + 1 < tiles.n) load(it + 1, lds_next);
    Tile::arrived();
    __syncthreads();  // this tile is there, and the other buffer is no longer read
    if (kDirect && it + 1 < tiles.n) load(it + 1, lds_next);
    const int j0 = tiles.key0(it);
    if (iw >= s.len || j0 > iw + 31) return;
    if (j0 >= a.sinks && j0 + G::kRows - 1 <= iw - a.window) return;

    f32x16 sc[kSubs] = {};
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub)
        sc[sub] = mma(left<T>(kt, at, 32 * sub, ks), q[ks], sc[sub]);
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
      const int js = j0 + 32 * sub;
      if (js + 31 > iw || js < iw + 31 - a.window + 1) hide_keys<AGAIN>(a, i, js, sc[sub], -kInf);
    }
    float top = sc[0][0];
#pragma unroll
    for (int r = 1; r < 16 * kSubs; ++r) top = fmaxf(top, sc[r >> 4][r & 15]);
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
#pragma unroll
    for (int r = 0; r < 16 * kSubs; ++r) {
      sc[r >> 4][r & 15] = __builtin_amdgcn_exp2f(fmaf(sc[r >> 4][r & 15], c, -off));
      l += sc[r >> 4][r & 15];
    }
#pragma unroll
    for (int k = 0; k < 2 * kSubs; ++k) {
      const V8 pb = right_of<T>(sc[k >> 1], 8 * (k & 1));
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T>(vt, at, 16 * k, db), pb, o[db]);
    }
  };
  // two tiles a turn, so that the buffers' places are constants
  for (int it = 0; it < tiles.n; it += 2) {
    meet(it, sh.tile[0], sh.tile[G::kBuffers - 1]);
    if (it + 1 < tiles.n) meet(it + 1, sh.tile[G::kBuffers - 1], sh.tile[0]);
  }
  l = swap32_sum(l);
}

// Waves of a SIMD that the forward and dq have registers for without their second way, whose code would otherwise
// take more: 400 events a sequence, window 300, 8 heads of 64, forward 70 us instead of 51.
template <int DH, int WAVES, bool DIRECT>
constexpr int fwd_waves = DH == 128 ? 2 : DH == 64 ? (WAVES == 4 && DIRECT ? 4 : 3) : WAVES == 1 ? 5 : 4;
template <int DH>
constexpr int dq_waves = DH == 128 ? 2 : DH == 64 ? 3 : 4;

template <typename T, int DH, int WAVES, bool DIRECT>
__global__ void __launch_bounds__(Group<WAVES>::kThreads, (fwd_waves<DH, WAVES, DIRECT>)) attn_fwd(AttnArgs a) {
  typedef Group<WAVES> G;
  __shared__ QueryShared<T, DH, WAVES, DIRECT> sh;
  const int group = a.q_heads / a.kv_heads;
  const int block = WAVES == 1 ? blockIdx.x : gridDim.x - 1 - blockIdx.x;
  const int kh = block % a.kv_heads;
  const int rest = block / a.kv_heads;
  const int h = kh * group + rest % group;
  const Seq s = find_tile(a, rest / group, [](int64_t t, int b) { return t / G::kTokens + b; });
  if (s.tile < 0 || (int64_t)s.tile * G::kTokens >= s.len) return;
  const int iw = __builtin_amdgcn_readfirstlane(s.tile * G::kTokens + (threadIdx.x >> 6) * 32);
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  f32x16 o[DH / 32];
  float m, l;
  fwd_sums<T, DH, WAVES, DIRECT, 0>(a, sh, s, h, kh, iw, c, o, m, l);
  const int i = iw + (lane_id() & 31);
  if (any_wave(i < s.len && not_finite(o), sh.said)) {
    fwd_sums<T, DH, WAVES, DIRECT, 1>(a, sh, s, h, kh, iw, c, o, m, l);
    add_odd_seen<T, DH, WAVES, DIRECT, true>(a, a.v, sh, s, kh, iw, o);
    __syncthreads();  // the tiles are done with
  }
  constexpr int kOwn = DIRECT ? 3 : 0;  // addresses of its own: the kernel of 64-wide heads has no register over
  typedef WaveRows<T, DH, TileOf<T, DH, G::kRows, G::kThreads, DIRECT, kOwn>, kOwn> Rows;
  Rows::store(a.out, s.begin + iw, h, s.len - iw, a.dim, sh.part(0), sh.first(), o, 1.f / l, 0);
  if (i < s.len && a.lse && lane_id() < 32) a.lse[(int64_t)h * a.n_tok + s.begin + i] = m * c * kLn2 + logf(l);
}

// ---------------------------------------------------------------- backward: dq
// As the forward, with dout as a second right operand: unscaled sums of the gradients that the wave's 32 queries
// from iw on have; also writes delta.  8.6k tokens, 16 and 8 heads of 128, window 1024, bf16: 114 us, 730 TFLOP/s of
// three products, bound as the forward is.  512 histories of up to 200, 8 heads of 64, window 64, fp16: 69 us,
// 3.7 TB/s.
template <typename T, int DH, int WAVES, bool DIRECT, int AGAIN>
__device__ __forceinline__ void dq_sums(const AttnArgs& a, QueryShared<T, DH, WAVES, DIRECT>& sh, const Seq& s, int h,
                                        int kh, int iw, f32x16 (&dq)[DH / 32]) {
  typedef typename Vec8<T>::t V8;
  typedef Group<WAVES> G;
  constexpr bool kDirect = DIRECT && !AGAIN;
  typedef TileOf<T, DH, G::kRows, G::kThreads, kDirect, AGAIN> Tile;
  constexpr int kBytes = sizeof(sh.tile[0][0]);
  constexpr int kSubs = G::kRows / 32;
  const int i = iw + (lane_id<AGAIN>() & 31);
  const bool live = i < s.len;

  const int rows = s.len - iw;  // of the wave's 32 queries
  typedef WaveRows<T, DH, Tile, AGAIN> Rows;
  Rows ql, dl, ol;
  ql.load(a.q, s.begin + iw, h, rows, a.dim);
  dl.load(a.dout, s.begin + iw, h, rows, a.dim);
  ol.load(a.out, s.begin + iw, h, rows, a.dim);
  const KeyTiles<WAVES> tiles(a, s.tile * G::kTokens, s.len);
  const T* kp = static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head;
  Tile kl, vl;
  auto load = [&](int it, char (*to)[kBytes]) {
    kl.load(to[0], kp, a.k.tok, tiles.key0(it), tiles.end(a, it, s.len), a.dim);
    vl.load(to[1], vp, a.v.tok, tiles.key0(it), tiles.end(a, it, s.len), a.dim);
  };
  load(0, sh.tile[0]);
  const typename Tile::Reads at;

  char* const part = sh.part(G::kBuffers - 1);
  V8 q[DH / 16], d[DH / 16];
  ql.to_right(part, sh.first(), at, q);
  dl.to_right(part, sh.first(), at, d);
  float delta = 0.f;
  {
    V8 out[DH / 16];
    ol.to_right(part, sh.first(), at, out);
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta += (float)out[ks][e] * (float)d[ks][e];
    delta = swap32_sum(delta);
  }
  const int64_t stat = (int64_t)h * a.n_tok + s.begin + i;
  if (live && lane_id<AGAIN>() < 32) a.delta[stat] = delta;
  const float c = a.scale * kLog2e;
  const float lse = live ? a.lse[stat] * kLog2e : kInf;

#pragma unroll
  for (int db = 0; db < DH / 32; ++db) dq[db] = f32x16{};
  int by = 0;  // AGAIN, in fp16: dq stands at 2^-by
  auto meet = [&](int it, char (*lds_now)[kBytes], char (*lds_next)[kBytes]) {
    const char* kt = lds_now[0];
    const char* vt = lds_now[1];
    if (G::kBuffers == 1) __syncthreads();  // of one wave: its reads of the tile before have ended
    if (AGAIN && it) load(it, lds_now);
    kl.store(lds_now[0]);
    vl.store(lds_now[1]);
    if (!kDirect && !AGAIN && it + 1 < tiles.n) load(it + 1, lds_next);
    Tile::arrived();
    __syncthreads();  // this tile is there, and the other buffer is no longer read
    if (kDirect && it + 1 < tiles.n) load(it + 1, lds_next);
    const int j0 = tiles.key0(it);
    if (iw >= s.len) return;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
      const int js = j0 + 32 * sub;
      if (js > iw + 31 || (js >= a.sinks && js + 31 <= iw - a.window)) continue;
      f32x16 sc = {}, dp = {};
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks) {
        sc = mma(left<T>(kt, at, 32 * sub, ks), q[ks], sc);
        dp = mma(left<T>(vt, at, 32 * sub, ks), d[ks], dp);
      }
      f32x16 ds;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        ds[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -lse)) * (dp[r] - delta);
      if (js + 31 > iw || js < iw + 31 - a.window + 1) hide_keys<AGAIN>(a, i, js, ds, 0.f);
      if constexpr (AGAIN != 0) fit<T>(ds, dq, by);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const V8 b = right_of<T>(ds, 8 * k);
#pragma unroll
        for (int db = 0; db < DH / 32; ++db) {
          V8 x = left_t<T>(kt, at, 32 * sub + 16 * k, db);
          if (AGAIN) x = finite_of<T>(x);
          dq[db] = mma(x, b, dq[db]);
        }
      }
    }
  };
  // two tiles a turn, so that the buffers' places are constants
  for (int it = 0; it < tiles.n; it += 2) {
    meet(it, sh.tile[0], sh.tile[G::kBuffers - 1]);
    if (it + 1 < tiles.n) meet(it + 1, sh.tile[G::kBuffers - 1], sh.tile[0]);
  }
  if constexpr (AGAIN != 0) unfit(dq, by);
}

template <typename T, int DH, int WAVES, bool DIRECT>
__global__ void __launch_bounds__(Group<WAVES>::kThreads, (dq_waves<DH>)) attn_dq(AttnArgs a) {
  typedef Group<WAVES> G;
  __shared__ QueryShared<T, DH, WAVES, DIRECT> sh;
  const int group = a.q_heads / a.kv_heads;
  const int block = WAVES == 1 ? blockIdx.x : gridDim.x - 1 - blockIdx.x;
  const int kh = block % a.kv_heads;
  const int rest = block / a.kv_heads;
  const int h = kh * group + rest % group;
  const Seq s = find_tile(a, rest / group, [](int64_t t, int b) { return t / G::kTokens + b; });
  if (s.tile < 0 || (int64_t)s.tile * G::kTokens >= s.len) return;
  const int iw = __builtin_amdgcn_readfirstlane(s.tile * G::kTokens + (threadIdx.x >> 6) * 32);
  f32x16 dq[DH / 32];
  dq_sums<T, DH, WAVES, DIRECT, 0>(a, sh, s, h, kh, iw, dq);
  if (__builtin_expect(any_wave(iw + (lane_id() & 31) < s.len && not_finite(dq), sh.said), 0)) {
    dq_sums<T, DH, WAVES, DIRECT, 1>(a, sh, s, h, kh, iw, dq);
    add_odd_seen<T, DH, WAVES, DIRECT, false>(a, a.k, sh, s, kh, iw, dq);
    __syncthreads();  // the tiles are done with
  }
  typedef WaveRows<T, DH, TileOf<T, DH, G::kRows, G::kThreads, DIRECT, 3>, 3> Rows;
  Rows::store(a.dq, s.begin + iw, h, s.len - iw, a.dim, sh.part(0), sh.first(), dq, a.scale, 0);
}

// ---------------------------------------------------------------- backward: dk, dv
// A workgroup has 128 keys of a key/value head and meets the queries of every head of its group that
// see them, 64 rows a step; sums stay in registers, so nothing is added up in memory.
//
// The sinks are seen by every later query of their sequence too: those queries, from `reach` on, are
// cut into chunks, each a workgroup whose waves take its rows in turn for the first 32 keys; its
// sums and those of the first key tile go to memory in fp32, and attn_sink_join adds them in order.
//
// Heads of 64 and less: four waves of 32 keys, which hold their keys and values as right operands in
// registers.  Heads of 128: the sums alone take 128 registers and the operands another 64, which
// leaves one wave a SIMD; eight waves, two to each 32 keys with half of a step's rows, and keys and
// values in LDS make it two, at a half more reads of LDS.
//
// 8.6k tokens, 16 and 8 heads of 128, window 1024, bf16: 188 us, 590 TFLOP/s of four products: matrix cores, vector
// unit and LDS are busy 29, 23 and 28 % of the time, and half of a wave's time it waits.  512 histories of up to 200,
// 8 heads of 64, window 64, fp16: 70 us, 3.6 TB/s.
static_assert(EMB_ATTN_MAX_SINKS <= 32, "the sinks lie in the first 32 keys");

// Queries from here on see nothing of the first key tile but the sinks.
inline int64_t reach_of(int window, int tokens) { return (int64_t)tokens + window - 1; }

// Where partial sums of the sinks go, [2][sinks][dim] each: first those of the chunks by slot, then those
// of the first key tiles.  Only sequences longer than reach have any; each is given a number, its own
// or, where the batch has over twice the sequences that could be that long, which part of reach + 1
// tokens it begins in.  A sequence's chunks start at slot begin / chunk + number, which leaves it room for
// len / chunk + 1 of them.
struct SinkSlots {
  int64_t reach, numbers, chunk_slots;
  int chunk;
  bool by_sequence;
  SinkSlots(int64_t n_tok, int64_t n_seq, int window, int tokens, int chunk_) {
    reach = reach_of(window, tokens);
    chunk = chunk_;
    const int64_t most = n_tok / (reach + 1) + 1;
    by_sequence = n_seq <= 2 * most;
    numbers = by_sequence ? n_seq : most;
    chunk_slots = n_tok / chunk + numbers + 1;
  }
  // in 32 bits: tokens are fewer than 2^31, and reach + 1 at most 2^31 + 127
  __device__ int64_t number(int64_t begin, int b) const {
    return by_sequence ? b : (uint32_t)begin / (uint32_t)(reach + 1);
  }
  __device__ int64_t first(int64_t begin, int b) const {
    return (uint32_t)begin / (uint32_t)chunk + number(begin, b);
  }
};
__device__ __forceinline__ float* sink_part(const AttnArgs& a, int64_t slot, int kh) {
  return a.part + (slot * a.kv_heads + kh) * 2 * a.sinks * (int64_t)a.dim;
}
__device__ __forceinline__ float* first_tile_part(const AttnArgs& a, const SinkSlots& p, const Seq& s, int kh) {
  return sink_part(a, p.chunk_slots + p.number(s.begin, s.index), kh);
}

// Adds the sums of the upper half of `n` waves to those of the lower half, through LDS.
template <int AGAIN, int N>
__device__ __forceinline__ void fold_waves(f32x16 (&x)[N], float* lds, int wave, int n) {
  __syncthreads();
  if (wave >= n / 2 && wave < n) {
#pragma unroll
    for (int k = 0; k < N * 16; ++k) lds[((wave - n / 2) * N * 16 + k) * 64 + lane_id<AGAIN>()] = x[k >> 4][k & 15];
  }
  __syncthreads();
  if (wave < n / 2) {
#pragma unroll
    for (int k = 0; k < N * 16; ++k) x[k >> 4][k & 15] += lds[(wave * N * 16 + k) * 64 + lane_id<AGAIN>()];
  }
}

template <typename T, int DH, int WAVES, bool DIRECT, int AGAIN = 0>
struct DkvShape {
  typedef Group<WAVES> G;
  static constexpr bool kWide = DH == 128 && WAVES == 4;
  static constexpr int kWaves = kWide ? 8 : WAVES;
  static constexpr int kBlock = kWaves * 64;
  static constexpr int kShare = kWide ? 2 : 1;  // waves that share 32 keys
  static constexpr int kKeyTiles = kWide ? 2 : 0;
  typedef TileOf<T, DH, G::kRows, kBlock, DIRECT, AGAIN> Tile;
};
template <typename T, int DH, int WAVES, bool DIRECT>
struct DkvShared {
  typedef DkvShape<T, DH, WAVES, DIRECT> P;
  static constexpr int kTile = P::Tile::kBytes;
  char q[P::G::kBuffers][kTile], d[P::G::kBuffers][kTile];
  char k[P::kKeyTiles][kTile], v[P::kKeyTiles][kTile];
  float lse[P::G::kBuffers][P::G::kRows], delta[P::G::kBuffers][P::G::kRows];
  uint32_t said[P::kWaves];
  // A wave's own part, before the steps and after them: where keys and values have their tiles, or half of a
  // buffer of queries or gradients that the first step does not use.
  __device__ __forceinline__ char* part(int wave) {
    if (P::kWide) return wave & 2 ? v[0] : k[0];
    return (wave & 2 ? d : q)[P::G::kBuffers - 1];
  }
};

// The sums of rows `row0` to `row1` - 1 against the 128 keys from j0 (SINK: the sinks), which the first kFirst
// waves have in the end.  Of both; or, where they came out not finite, of dk or dv AGAIN, one at a time to have
// the registers, so that they are what the pairs that see each other make them: without the products with zero
// of those that do not, and in fp16 with gradients of scores past 65504 brought into range.
enum { kBoth, kDkAgain, kDvAgain };
template <typename T, int DH, int WAVES, bool DIRECT, bool SINK, int WHAT>
__device__ __forceinline__ void dkv_sums(const AttnArgs& a, DkvShared<T, DH, WAVES, DIRECT>& sh, const Seq& s, int kh,
                                         int j0, int row0, int row1, f32x16 (&dk)[DH / 32], f32x16 (&dv)[DH / 32]) {
  typedef typename Vec8<T>::t V8;
  constexpr int AGAIN = WHAT;
  constexpr bool DK = WHAT != kDvAgain, DV = WHAT != kDkAgain;
  typedef DkvShape<T, DH, WAVES, DIRECT, AGAIN> P;
  typedef typename P::Tile Tile;
  typedef Group<WAVES> G;
  constexpr int kRows = G::kRows;
  const int group = a.q_heads / a.kv_heads;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int jrow = SINK ? 0 : 32 * (wave & 3);  // the wave's keys within the tile
  const int jw = j0 + jrow;
  const int j = jw + (lane_id<AGAIN>() & 31);
  const uint32_t limit = j < a.sinks ? 0x7FFFFFFFu : (uint32_t)a.window;

  const typename Tile::Reads at;
  typedef WaveRows<T, DH, Tile, AGAIN> Rows;
  V8 k[P::kWide ? 1 : DH / 16], v[P::kWide ? 1 : DH / 16];
  if constexpr (P::kWide && AGAIN) {
    // they are still there
  } else if constexpr (P::kWide) {
    const T* kp = static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head;
    const T* vp = static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      Tile kl, vl;
      kl.load(sh.k[x], kp, a.k.tok, j0 + kRows * x, s.len, a.dim);
      vl.load(sh.v[x], vp, a.v.tok, j0 + kRows * x, s.len, a.dim);
      kl.store(sh.k[x]);
      vl.store(sh.v[x]);
    }
  } else {
    // through the buffers that the first step does not use
    char* const part = sh.part(wave);
    const int first = WAVES == 1 ? 0 : 32 * (wave & 1);
    Rows kl, vl;
    kl.load(a.k, s.begin + jw, kh, s.len - jw, a.dim);
    vl.load(a.v, s.begin + jw, kh, s.len - jw, a.dim);
    kl.to_right(part, first, at, k);
    vl.to_right(part, first, at, v);
  }
  const float c = a.scale * kLog2e;

  const int n_tiles = (row1 - row0 + kRows - 1) / kRows;
  Tile ql, dl;
  float stat = 0.f;  // the first kRows threads: lse of a row; as many after them: its delta
  int next_h = kh * group, next_r0 = row0;  // what is loaded next
  auto load = [&](int b) {
    const int h = next_h, r0 = next_r0;
    ql.load(sh.q[b], static_cast<const T*>(a.q.p) + s.begin * a.q.tok + h * a.q.head, a.q.tok, r0, row1, a.dim);
    dl.load(sh.d[b], static_cast<const T*>(a.dout.p) + s.begin * a.dout.tok + h * a.dout.head, a.dout.tok, r0,
            row1, a.dim);
    if (thread_id<AGAIN>() < 2 * kRows) {
      const int row = r0 + (thread_id<AGAIN>() & (kRows - 1));
      const float* p = thread_id<AGAIN>() < kRows ? a.lse : a.delta;
      // a row that is not there gets probabilities of zero
      stat = thread_id<AGAIN>() < kRows ? kInf : 0.f;
      if (row < row1) stat = p[(int64_t)h * a.n_tok + s.begin + row];
    }
    next_r0 += kRows;
    if (next_r0 >= row1) {
      next_r0 = row0;
      ++next_h;
    }
  };
#pragma unroll
  for (int db = 0; db < DH / 32; ++db) {
    if (DK) dk[db] = f32x16{};
    if (DV) dv[db] = f32x16{};
  }
  int by = 0;  // AGAIN, in fp16: dk stands at 2^-by
  float* fold = reinterpret_cast<float*>(sh.q);  // q and d: half the waves' sums of one matrix
  static_assert(sizeof(sh.q) + sizeof(sh.d) >= sizeof(float) * P::kWaves / 2 * 32 * DH, "room to fold");
  constexpr int kFirst = SINK ? 1 : P::kWaves / P::kShare;
  {
    load(0);
    int r0 = row0;
    const int steps = n_tiles * group;  // of all heads of the group
    for (int step = 0; step < steps; ++step, r0 = r0 + kRows < row1 ? r0 + kRows : row0) {
      const int b = step & (G::kBuffers - 1);
      if (G::kBuffers == 1) __syncthreads();  // of one wave: its reads of the tile before have ended
      ql.store(sh.q[b]);
      dl.store(sh.d[b]);
      if (thread_id<AGAIN>() < kRows) sh.lse[b][thread_id<AGAIN>()] = stat * kLog2e;
      else if (thread_id<AGAIN>() < 2 * kRows) sh.delta[b][thread_id<AGAIN>() - kRows] = stat;
      const int other = b ^ (G::kBuffers - 1);
      if (!DIRECT && step + 1 < steps) load(other);
      Tile::arrived();
      __syncthreads();  // this step's rows are there, and the other buffer is no longer read
      if (DIRECT && step + 1 < steps) load(other);
      if (jw >= s.len) continue;
#pragma unroll
      for (int sub_ = 0; sub_ < kRows / 32 / P::kShare; ++sub_) {
        const int sub = P::kShare == 2 ? wave >> 2 : sub_;
        const int is = r0 + 32 * sub;
        if (is >= row1) continue;
        if (SINK) {
          // rows go round the waves: by steps where a wave has a fixed half of each
          if (P::kWaves > 1 && ((P::kShare == 2 ? step : step * 2 + sub) & 3) != (wave & 3)) continue;
        } else if (is + 31 < jw || (jw >= a.sinks && is >= jw + 31 + (int64_t)a.window)) {
          continue;
        }
        f32x16 sc = {}, dp = {};
        if constexpr (P::kWide) {
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks)
            sc = mma(left<T>(sh.q[b], at, 32 * sub, ks), left<T>(sh.k[jrow >> 6], at, jrow & 63, ks), sc);
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks)
            dp = mma(left<T>(sh.d[b], at, 32 * sub, ks), left<T>(sh.v[jrow >> 6], at, jrow & 63, ks), dp);
        } else {
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks) {
            sc = mma(left<T>(sh.q[b], at, 32 * sub, ks), k[ks], sc);
            dp = mma(left<T>(sh.d[b], at, 32 * sub, ks), v[ks], dp);
          }
        }
        f32x16 p, ds;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int at = 32 * sub + 8 * g + 4 * (lane_id<AGAIN>() >> 5);
          const f32x4 lse = *reinterpret_cast<const f32x4*>(&sh.lse[b][at]);
          const f32x4 delta = *reinterpret_cast<const f32x4*>(&sh.delta[b][at]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[4 * g + e] = __builtin_amdgcn_exp2f(fmaf(sc[4 * g + e], c, -lse[e]));
            ds[4 * g + e] = p[4 * g + e] * (dp[4 * g + e] - delta[e]);
          }
        }
        if constexpr (AGAIN) {
          const int d = is + 4 * (lane_id<AGAIN>() >> 5) - j, last = row1 - 1 - j;
          f32x16 x = DK ? ds : p;
          uint32_t see = 0;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int e = d + 8 * (r >> 2) + (r & 3);
            if ((uint32_t)e < limit && e <= last) see |= 1u << r;
            else x[r] = 0.f;
          }
          if (DK) fit<T>(x, dk, by);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const V8 xb = right_of<T>(x, 8 * n), one = ones<T>(see, 8 * n);
            V8 signs;  // in fp32 a small weight is not 0
#pragma unroll
            for (int e = 0; e < 8; ++e) signs[e] = (T)(x[8 * n + e] > 0.f ? 1.f : x[8 * n + e] < 0.f ? -1.f : 0.f);
#pragma unroll
            for (int db = 0; db < DH / 32; ++db) {
              f32x16& sum = DK ? dk[db] : dv[db];
              const V8 xa = left_t<T>(DK ? sh.q[b] : sh.d[b], at, 32 * sub + 16 * n, db);
              sum = mma(finite_of<T>(xa), xb, sum);
              add_odd<T>(sum, xa, one, signs);
            }
          }
          continue;
        }
        if (is < jw + 31 || (int64_t)is + 31 - jw >= a.window) {
          asm volatile("");  // see hide_keys
          const int d = is + 4 * (lane_id<AGAIN>() >> 5) - j;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if ((uint32_t)(d + 8 * (r >> 2) + (r & 3)) >= limit) p[r] = ds[r] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const V8 pb = right_of<T>(p, 8 * x), db_ = right_of<T>(ds, 8 * x);
#pragma unroll
          for (int db = 0; db < DH / 32; ++db) {
            dv[db] = mma(left_t<T>(sh.d[b], at, 32 * sub + 16 * x, db), pb, dv[db]);
            dk[db] = mma(left_t<T>(sh.q[b], at, 32 * sub + 16 * x, db), db_, dk[db]);
          }
        }
      }
    }
  }
  if (AGAIN && DK) unfit(dk, by);
  // the waves' sums of the same keys, to the first of them
#pragma unroll
  for (int n = P::kWaves; n > kFirst; n /= 2) {
    if (DK) fold_waves<AGAIN>(dk, fold, wave, n);
    if (DV) fold_waves<AGAIN>(dv, fold, wave, n);
  }
}

template <typename T, int DH, int WAVES, bool DIRECT, bool SINK>
__device__ __forceinline__ void dkv(const AttnArgs& a, DkvShared<T, DH, WAVES, DIRECT>& sh, const SinkSlots& parts,
                                    const Seq& s, int kh, int j0, int row0, int row1, int64_t slot) {
  typedef DkvShape<T, DH, WAVES, DIRECT> P;
  constexpr int kFirst = SINK ? 1 : P::kWaves / P::kShare;
  f32x16 dk[DH / 32], dv[DH / 32];
  dkv_sums<T, DH, WAVES, DIRECT, SINK, kBoth>(a, sh, s, kh, j0, row0, row1, dk, dv);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int jw = SINK ? 0 : j0 + 32 * (wave & 3), j = jw + (lane_id() & 31);
  const int odd = (int)not_finite(dk) | (int)not_finite(dv);  // no branch between the two
  const bool bad = wave < kFirst && j < (SINK ? a.sinks : s.len) && odd;
  if (__builtin_expect(any_wave(bad, sh.said), 0)) {
    dkv_sums<T, DH, WAVES, DIRECT, SINK, kDkAgain>(a, sh, s, kh, j0, row0, row1, dk, dv);
    __syncthreads();  // its tiles are done with
    dkv_sums<T, DH, WAVES, DIRECT, SINK, kDvAgain>(a, sh, s, kh, j0, row0, row1, dk, dv);
    __syncthreads();
  }
  if (wave >= kFirst) return;
  // sinks of a sequence with chunks go to their sums
  const bool split = SINK || (a.sinks > 0 && parts.reach < s.len);
  const uint32_t sums = split && jw == 0 ? (a.sinks == 32 ? ~0u : (1u << a.sinks) - 1) : 0;
  if (sums >> (lane_id() & 31) & 1) {
    const EmbHeads row{SINK ? sink_part(a, slot, kh) : first_tile_part(a, parts, s, kh), 0, a.dim, 0};
    store_row<float, DH>(row, j, 0, a.dim, dk, 1.f);
    store_row<float, DH>(row, a.sinks + j, 0, a.dim, dv, 1.f);
  }
  if (SINK) return;
  typedef WaveRows<T, DH, typename P::Tile> Rows;
  const int first = WAVES == 1 ? 0 : 32 * (wave & 1);
  Rows::store(a.dk, s.begin + jw, kh, s.len - jw, a.dim, sh.part(wave), first, dk, a.scale, sums);
  Rows::store(a.dv, s.begin + jw, kh, s.len - jw, a.dim, sh.part(wave), first, dv, 1.f, sums);
}

template <typename T, int DH, int WAVES, bool DIRECT>
__global__ void __launch_bounds__((DkvShape<T, DH, WAVES, DIRECT>::kBlock), 2)
    attn_dkv(AttnArgs a, int main_blocks, SinkSlots parts) {
  __shared__ __attribute__((aligned(1024))) DkvShared<T, DH, WAVES, DIRECT> sh;
  constexpr int kTokens = Group<WAVES>::kTokens;
  const bool sink = (int)blockIdx.x >= main_blocks;  // the same for the whole workgroup
  const int block = sink ? blockIdx.x - main_blocks : blockIdx.x;
  const int kh = block % a.kv_heads, slot = block / a.kv_heads;
  if (sink) {
    const Seq s = find_tile(a, slot, [&](int64_t t, int b) { return parts.first(t, b); });
    const int64_t r0 = parts.reach + (int64_t)s.tile * parts.chunk;
    if (s.tile < 0 || r0 >= s.len) return;
    const int row1 = (int)min(r0 + parts.chunk, (int64_t)s.len);
    dkv<T, DH, WAVES, DIRECT, true>(a, sh, parts, s, kh, 0, (int)r0, row1, slot);
  } else {
    const Seq s = find_tile(a, slot, [](int64_t t, int b) { return t / kTokens + b; });
    if (s.tile < 0 || (int64_t)s.tile * kTokens >= s.len) return;
    const int j0 = s.tile * kTokens, row1 = (int)min(j0 + parts.reach, (int64_t)s.len);
    dkv<T, DH, WAVES, DIRECT, false>(a, sh, parts, s, kh, j0, j0, row1, 0);
  }
}

// dk and dv of the sinks from the first key tile's sums and every chunk's, in that order: up to four
// elements a thread, a number (see SinkSlots) a row of workgroups.  A launch's latency and two trips to
// memory: 4.7 us at 5 sequences of up to 4095, 7.4 at 512 of up to 200.
constexpr int kJoinEach = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_sink_join(AttnArgs a, SinkSlots parts) {
  const int number = blockIdx.x;
  const Seq s = parts.by_sequence ? sequence(a, number, 0)
                                  : find_tile(a, number, [&](int64_t t, int b) { return parts.number(t, b); });
  if (s.tile != 0 || s.len <= parts.reach) return;
  const int n = (int)((uint32_t)(s.len - (int)parts.reach + parts.chunk - 1) / (uint32_t)parts.chunk);
  const int each = 2 * a.sinks * a.dim, all = each * a.kv_heads;
  const float* tile = first_tile_part(a, parts, s, 0);
  const float* part = sink_part(a, parts.first(s.begin, s.index), 0);
  const int at0 = blockIdx.y * kJoinEach * kThreads + threadIdx.x;
  float t[kJoinEach];
#pragma unroll
  for (int k = 0; k < kJoinEach; ++k) t[k] = tile[min(at0 + k * kThreads, all - 1)];
#pragma unroll 2
  for (int x = 0; x < n; ++x) {
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) t[k] += part[(int64_t)x * all + min(at0 + k * kThreads, all - 1)];
  }
#pragma unroll
  for (int k = 0; k < kJoinEach; ++k) {
    const int at = at0 + k * kThreads;
    if (at >= all) return;
    const int kh = at / each, e = at % each;
    const int row = e / a.dim % a.sinks, col = e % a.dim;
    const bool is_v = e >= a.sinks * a.dim;
    const EmbHeads& to = is_v ? a.dv : a.dk;
    static_cast<T*>(to.p)[(s.begin + row) * to.tok + kh * to.head + col] = (T)(is_v ? t[k] : t[k] * a.scale);
  }
}

// ---------------------------------------------------------------- one new event
// The keys that the newest event sees, in one row: the sinks outside the window, then the window.
// A workgroup has them, or a part, for one key/value head; its waves take tiles of 32 in turn, each with a
// softmax of its own, and meet in LDS at the end.  All query heads of the group are the
// columns of one product, so keys and values are read once.  Memory bound: 256 caches of up to 8192, 32
// and 8 heads of 128, window 4096, bf16: 493 us, 5.4 TB/s.  Few sequences are bound by a workgroup's chain of
// loads and products: 3 caches, 8 and 2 heads of 64, window 1000: 9.3 us.
template <int DH>
struct WaveTile {  // 32 rows, of one wave
  static constexpr int kPieces = DH / 8, kRegs = 32 * kPieces / 64;
};

template <typename T, int DH, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, WAVES == 16 ? 4 : 2) attn_decode(AttnArgs a, int splits) {
  typedef typename Vec8<T>::t V8;
  typedef RegisterTile<T, DH, 32, 64> Tile;
  const typename Tile::Reads reads;
  __shared__ __attribute__((aligned(16))) char lds[WAVES][2][Tile::kBytes];
  __shared__ float stats[WAVES][2][32];
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
      const int u = t0 + idx / Tile::kPieces, cl = idx % Tile::kPieces * 8;
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
  for (; t0 < u1; t0 += 32 * WAVES) {
#pragma unroll
    for (int n = 0; n < WaveTile<DH>::kRegs; ++n) {
      const int idx = lane + n * 64;
      const int at = Tile::at(idx / Tile::kPieces, idx % Tile::kPieces);
      *reinterpret_cast<u32x4*>(kt + at) = kr[n];
      *reinterpret_cast<u32x4*>(vt + at) = vr[n];
    }
    if (t0 + 32 * WAVES < u1) load(t0 + 32 * WAVES);
    // the tile is the wave's own: its LDS accesses are carried out in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    f32x16 sc = {};
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) sc = mma(left<T>(kt, reads, 0, ks), q[ks], sc);
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
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -off));
      l += sc[r];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const V8 pb = right_of<T>(sc, 8 * k);
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T>(vt, reads, 16 * k, db), pb, o[db]);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  l = swap32_sum(l);
  // the waves meet: each leaves its sums in its own part of LDS, and four rows of a column at a time
  // are scaled to the common maximum and added in the waves' order
  if (lane < 32) {
    stats[wave][0][lane] = m;
    stats[wave][1][lane] = l;
  }
  static_assert(sizeof(lds[0]) >= sizeof(float) * 32 * DH, "a wave's sums take its tiles' place");
  f32x4* mine = reinterpret_cast<f32x4*>(lds[wave]);
#pragma unroll
  for (int x = 0; x < DH / 8; ++x) {
    const f32x16 t = o[x >> 2];
    const int r = (x & 3) * 4;
    mine[x * 64 + lane] = f32x4{t[r], t[r + 1], t[r + 2], t[r + 3]};
  }
  __syncthreads();
  float top = -kInf, sum = 0.f, by[WAVES];
#pragma unroll
  for (int w = 0; w < WAVES; ++w) top = fmaxf(top, stats[w][0][lane & 31]);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const float mw = stats[w][0][lane & 31];
    by[w] = mw == -kInf ? 0.f : exp2f((mw - top) * c);
    sum += stats[w][1][lane & 31] * by[w];
  }
  // part: [split][sequence][q head][dim] of unscaled sums, then [..][2] of maximum and sum
  const int64_t total = (int64_t)a.n_seq * a.q_heads;
  const int qh = kh * group + head;
  const int64_t row = (int64_t)split * total + (int64_t)sq * a.q_heads + qh;
#pragma unroll
  for (int x = wave; x < DH / 8; x += WAVES) {  // which four rows
    const int d = x * 8 + 4 * (lane >> 5);
    f32x4 t = {};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const f32x4 ow = reinterpret_cast<const f32x4*>(lds[w])[x * 64 + lane];
      // a wave without keys has zeros, and so does its factor
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] += ow[e] * by[w];
    }
    if (!live || d >= a.dim) continue;
    if (splits == 1) {
      typedef T V __attribute__((ext_vector_type(4)));
      const float inv = n_keys > 0 ? 1.f / sum : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = n_keys > 0 ? t[e] * inv : 0.f;
      *reinterpret_cast<V*>(static_cast<T*>(a.out.p) + sq * a.out.tok + qh * a.out.head + d) =
          __builtin_convertvector(t, V);
    } else {
      *reinterpret_cast<f32x4*>(a.part + row * a.dim + d) = t;
    }
  }
  if (splits > 1 && live && threadIdx.x < 32)
    *reinterpret_cast<f32x2*>(a.part + (int64_t)splits * total * a.dim + row * 2) = f32x2{top * c, sum};
}

// One wave a (sequence, query head): the splits' sums at their common maximum.  A lane has one split's
// maximum and sum (of 64 at a time), then two columns of all.
template <typename T>
__global__ void __launch_bounds__(64) attn_decode_join(AttnArgs a, int splits) {
  const int64_t total = (int64_t)a.n_seq * a.q_heads, row = blockIdx.x;
  const float* st = a.part + (int64_t)splits * total * a.dim;
  const int lane = lane_id(), d = 2 * lane;
  float top = -kInf, sum = 0.f;
  f32x2 o = {};
  for (int x0 = 0; x0 < splits; x0 += 64) {
    f32x2 mine = {-kInf, 0.f};
    if (x0 + lane < splits) mine = *reinterpret_cast<const f32x2*>(st + ((x0 + lane) * total + row) * 2);
    float m = mine[0];
#pragma unroll
    for (int k = 1; k < 64; k *= 2) m = fmaxf(m, __shfl_xor(m, k, 64));
    const float t = fmaxf(top, m);
    const float keep = top == -kInf ? 0.f : exp2f(top - t);
    const float by = mine[0] == -kInf ? 0.f : exp2f(mine[0] - t);
    top = t;
    sum = sum * keep + lanes_sum<64>(by * mine[1]);
    o[0] *= keep;
    o[1] *= keep;
    const int n = min(splits - x0, 64);
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
      const float f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(by), x));
      f32x2 v = {};
      if (d < a.dim) v = *reinterpret_cast<const f32x2*>(a.part + ((x0 + x) * total + row) * a.dim + d);
      o[0] += f * v[0];
      o[1] += f * v[1];
    }
  }
  if (d >= a.dim) return;
  const int64_t sq = row / a.q_heads, qh = row % a.q_heads;
  const bool none = a.off[sq] <= 0;
  T* out = static_cast<T*>(a.out.p) + sq * a.out.tok + qh * a.out.head + d;
  out[0] = (T)(none ? 0.f : o[0] / sum);
  out[1] = (T)(none ? 0.f : o[1] / sum);
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
// Whether one wave a workgroup is the better shape, by what most queries see: their window or, in short
// sequences, what there is.  40k tokens, 8 heads of 64, fp16, four waves against one, forward / backward
// us: 20 tokens a sequence 91 / 318 and 38 / 112; 74 tokens, window 64: 44 / 143 and 34 / 108; 400 tokens,
// window 128: 48 / 167 and 44 / 138, 256: 51 / 172 and 53 / 156, 512: 49 / 162 and 57 / 162; 2000
// tokens, 128: 45 / 155 and 45 / 150, 256: 57 / 177 and 64 / 192.
constexpr int64_t kOneWave = 128;
bool one_wave(const AttnArgs& a) {
  const int64_t mean = a.n_tok / a.n_seq;
  return a.dim <= 64 && std::min<int64_t>(mean, a.window) <= kOneWave;
}

}  // namespace

// Whether a sequence of the batch may be longer than reach.
bool has_chunks(const AttnArgs& a, const SinkSlots& n) { return a.sinks > 0 && a.n_tok > n.reach; }

// Threads of a call's largest launch: two for each token that a slot has room for, four in dk/dv of wide heads.
int64_t attn_fwd_threads(const AttnArgs& a) {
  const int64_t tokens = one_wave(a) ? 32 : 128;
  return (a.n_tok / tokens + a.n_seq) * a.q_heads * 2 * tokens;
}
int64_t attn_bwd_threads(const AttnArgs& a) {
  const int64_t tokens = one_wave(a) ? 32 : 128;
  const SinkSlots n(a.n_tok, a.n_seq, a.window, (int)tokens, sink_chunk(a.n_tok));
  const int64_t slots = a.n_tok / tokens + a.n_seq + (has_chunks(a, n) ? n.chunk_slots : 0);
  const int64_t dkv = slots * a.kv_heads * (a.dim <= 64 ? 2 : 4) * tokens;
  const int64_t join = has_chunks(a, n) ? n.numbers * kThreads : 0;
  return std::max({attn_fwd_threads(a), dkv, join});
}
int64_t attn_decode_threads(const AttnArgs& a, const AttnDecodePlan& p) {
  const int64_t cols = (a.q_heads / a.kv_heads + 31) / 32;
  return (int64_t)a.n_seq * 64 * std::max<int64_t>(a.kv_heads * cols * p.splits * p.waves, a.q_heads);
}

AttnBwdPlan plan_attn_bwd(const EmbAttn& a, int64_t n_seq, int64_t n_tok) {
  AttnBwdPlan p{};
  p.off_part = ((size_t)n_tok * a.q_heads * sizeof(float) + 255) & ~(size_t)255;
  p.bytes = p.off_part;
  if (a.sinks > 0) {  // for any window and shape: the smallest leave the most sequences longer than reach
    const SinkSlots n(n_tok, n_seq, 1, 32, sink_chunk(n_tok));
    p.bytes += (size_t)(n.chunk_slots + n.numbers + 1) * a.kv_heads * 2 * a.sinks * a.dim * sizeof(float);
  }
  return p;
}

// How a sequence's keys are shared out.  Many sequences and heads: a workgroup of four waves each.  Few:
// one workgroup of as many waves as LDS has room for while that is two tiles a wave, or while there is
// one for every other unit; more keys, parts of at least a tile to each of four waves, whose sums a
// second kernel joins.  One sequence, 2 key/value heads of 64: 1024 keys 8.8 us in one workgroup, 8.6 in
// parts; 512 keys 7.1 and 7.7; 4000 keys 18.9 and 14.8.  32 sequences, 8 heads of 128, 1024 keys: 24.6 and 29.5.
constexpr int kOneGroupTiles = 2;
AttnDecodePlan plan_attn_decode(const EmbAttn& a, int64_t n_seq, int64_t capacity) {
  AttnDecodePlan p{4, 1, 0};
  const int64_t keys = std::min<int64_t>(capacity, (int64_t)a.window + a.sinks);
  const int64_t group = a.q_heads / a.kv_heads, base = std::max<int64_t>(n_seq * a.kv_heads * ((group + 31) / 32), 1);
  if (base >= 512 || keys <= 128) return p;
  const int most = a.dim <= 64 ? 16 : 8;
  if (base <= 256 && (base > 128 || keys <= 32 * most * kOneGroupTiles)) {
    p.waves = most;
    return p;
  }
  p.splits = (int32_t)std::min<int64_t>((keys + 127) / 128, 1024 / base);
  p.bytes = p.splits > 1 ? (size_t)p.splits * n_seq * a.q_heads * (a.dim + 2) * sizeof(float) : 0;
  return p;
}

template <typename T, int DH, int WAVES, bool DIRECT>
void go_fwd(const AttnArgs& a, hipStream_t st) {
  typedef Group<WAVES> G;
  const unsigned grid = (unsigned)((a.n_tok / G::kTokens + a.n_seq) * a.q_heads);
  hipLaunchKernelGGL((attn_fwd<T, DH, WAVES, DIRECT>), dim3(grid), dim3(G::kThreads), 0, st, a);
}

// A launch that fails is the last one: what comes after it would read what it did not write.
template <typename T, int DH, int WAVES, bool DIRECT>
hipError_t go_bwd(const AttnArgs& a, hipStream_t st) {
  typedef Group<WAVES> G;
  const int64_t slots = a.n_tok / G::kTokens + a.n_seq;
  hipLaunchKernelGGL((attn_dq<T, DH, WAVES, DIRECT>), dim3((unsigned)(slots * a.q_heads)), dim3(G::kThreads), 0,
                     st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const SinkSlots n(a.n_tok, a.n_seq, a.window, G::kTokens, sink_chunk(a.n_tok));
  const bool sinks = has_chunks(a, n);
  hipLaunchKernelGGL((attn_dkv<T, DH, WAVES, DIRECT>),
                     dim3((unsigned)((slots + (sinks ? n.chunk_slots : 0)) * a.kv_heads)),
                     dim3(DkvShape<T, DH, WAVES, DIRECT>::kBlock), 0, st, a, (int)(slots * a.kv_heads), n);
  e = hipGetLastError();
  if (sinks && e == hipSuccess) {
    hipLaunchKernelGGL((attn_sink_join<T>),
                       dim3((unsigned)n.numbers,
                            (unsigned)((2 * a.sinks * a.dim * a.kv_heads + kThreads * kJoinEach - 1) /
                                       (kThreads * kJoinEach))),
                       dim3(kThreads), 0, st, a, n);
    e = hipGetLastError();
  }
  return e;
}

// Whether tiles may be loaded straight to LDS: whole rows of the kernel's width, and a tile's rows
// within 2^31 bytes of one another.
bool direct(const AttnArgs& a, int width, std::initializer_list<const EmbHeads*> heads) {
  for (const EmbHeads* h : heads)
    if (h->tok < 0 || h->tok > ((int64_t)1 << 23)) return false;
  return a.dim == width;
}

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st) {
  by_shape(a, [&](auto t, auto d) {
    typedef decltype(t) T;
    constexpr int DH = decltype(d)::value;
    if constexpr (DH < 128) {
      if (one_wave(a)) return go_fwd<T, DH, 1, false>(a, st);
    }
    if (direct(a, DH, {&a.k, &a.v})) go_fwd<T, DH, 4, true>(a, st);
    else go_fwd<T, DH, 4, false>(a, st);
  });
  return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st) {
  hipError_t e = hipSuccess;
  by_shape(a, [&](auto t, auto d) {
    typedef decltype(t) T;
    constexpr int DH = decltype(d)::value;
    if constexpr (DH < 128) {
      if (one_wave(a)) {
        e = go_bwd<T, DH, 1, false>(a, st);
        return;
      }
    }
    if (direct(a, DH, {&a.q, &a.k, &a.v, &a.dout})) e = go_bwd<T, DH, 4, true>(a, st);
    else e = go_bwd<T, DH, 4, false>(a, st);
  });
  return e;
}

template <typename T, int DH, int WAVES>
void go_decode(const AttnArgs& a, const AttnDecodePlan& p, hipStream_t st) {
  const int64_t cols = (a.q_heads / a.kv_heads + 31) / 32;
  hipLaunchKernelGGL((attn_decode<T, DH, WAVES>), dim3((unsigned)(a.n_seq * a.kv_heads * cols * p.splits)),
                     dim3(64 * WAVES), 0, st, a, p.splits);
}

hipError_t launch_attn_decode(const AttnArgs& a, const AttnDecodePlan& p, hipStream_t st) {
  hipError_t e = hipSuccess;
  by_shape(a, [&](auto t, auto d) {
    typedef decltype(t) T;
    constexpr int DH = decltype(d)::value, kMost = DH <= 64 ? 16 : 8;
    if (p.waves == kMost) go_decode<T, DH, kMost>(a, p, st);
    else go_decode<T, DH, 4>(a, p, st);
    e = hipGetLastError();
    if (p.splits > 1 && e == hipSuccess) {
      hipLaunchKernelGGL((attn_decode_join<T>), dim3((unsigned)((int64_t)a.n_seq * a.q_heads)), dim3(64), 0,
                         st, a, p.splits);
      e = hipGetLastError();
    }
  });
  return e;
}

}  // namespace emb
