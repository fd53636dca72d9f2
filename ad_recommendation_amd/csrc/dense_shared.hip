// Attention of many candidates of a request to its one history and to their own tokens; and of a newest event to
// a cache in 8 bits, which is the same with one query token a request and nothing of its own.
//
//   see(i, j) = j of the request's history, inside its window or a sink; or j of i's candidate, j <= i
//   s_ij = scale q_i . k_j;  p_i = softmax(s_i);  out_i = sum_j p_ij v_j;  lse_i = log sum_j exp(s_ij)
//
// One pass over the keys with a running maximum and sum for each query row; rows are (token, head of the group),
// so a history is read once for every candidate and head that shares it.  Two shapes: 128 rows a workgroup, 32 a
// wave, which share tiles of 64 keys in LDS (bound by matrix cores and exponentials); and, where a request has few
// rows, 32 rows a workgroup whose waves take tiles of 32 keys in turn, each with a softmax of its own, and meet in
// LDS (bound by reading the history).  Either may share a request's keys out over several workgroups, whose sums a
// second kernel joins.
#include <algorithm>
#include <initializer_list>

#include "dense_shared_device.h"

namespace emb {

namespace {

// The maximum m that o and l stand at moves to that of the scores as well, only when it is over 2^8 times the old
// one's exponential: below that the probabilities stay small enough for 16 bits and the sums for 32.  Scores
// become probabilities, their sum goes to l (a lane's half of it).
template <int N, int DB>
__device__ __forceinline__ void soften(f32x16 (&sc)[N], f32x16 (&o)[DB], float& m, float& l, float c) {
  float top = sc[0][0];
#pragma unroll
  for (int r = 1; r < 16 * N; ++r) top = fmaxf(top, sc[r >> 4][r & 15]);
  top = swap32_max(top);
  if (__any((top - m) * c > 8.f)) {
    const float mn = fmaxf(m, top);
    const float by = m == -kInf ? 0.f : exp2f((m - mn) * c);
    m = mn;
    l *= by;
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] *= by;
  }
  const float off = m == -kInf ? 0.f : m * c;
#pragma unroll
  for (int r = 0; r < 16 * N; ++r) {
    sc[r >> 4][r & 15] = __builtin_amdgcn_exp2f(fmaf(sc[r >> 4][r & 15], c, -off));
    l += sc[r >> 4][r & 15];
  }
}

// Sums o and l at the maximum m after the history meet the row's own tokens.  They come after the loop over the
// history and share no address with it (AGAIN, see lane_id), so that it keeps its registers.
//
// A token alone: its score and value on the vector unit, so nothing that is not finite reaches another row.  A
// score of minus infinity has a weight of 0; one that is not finite otherwise makes the sum NaN.
template <typename T, int DH>
__device__ __forceinline__ void meet_self(const SharedArgs& a, int64_t tok, int kh, bool live,
                                          const typename Vec8<T>::t (&q)[DH / 16], float c, f32x16 (&o)[DH / 32],
                                          float& m, float& l) {
  const float s = dot_row<T, DH>(q, static_cast<const T*>(a.k.p) + tok * a.k.tok + kh * a.k.head, live, a.dim);
  if (!live) return;
  const float mn = fmaxf(m, s), by = m == -kInf ? 0.f : exp2f((m - mn) * c);
  const float p = s == -kInf ? 0.f : exp2f((s - mn) * c);
  m = mn;
  l = l * by + (lane_id<3>() < 32 ? p : 0.f);
  typedef T V __attribute__((ext_vector_type(4)));
  const T* v = static_cast<const T*>(a.v.p) + tok * a.v.tok + kh * a.v.head;
#pragma unroll
  for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = db * 32 + 8 * g + 4 * (lane_id<3>() >> 5);
      f32x4 x = {};
      if (col < a.dim) x = __builtin_convertvector(*reinterpret_cast<const V*>(v + col), f32x4);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[db][4 * g + e] = o[db][4 * g + e] * by + p * x[e];
    }
  }
}

// 32 own tokens from j0 on, keys and values in LDS at row `at0`, of which a row sees lo to hi.
template <typename T, int DH, typename R>
__device__ __forceinline__ void meet_own(const char* kt, const char* vt, const R& at, int at0, int lo, int hi, int j0,
                                         const typename Vec8<T>::t (&q)[DH / 16], float c, f32x16 (&o)[DH / 32],
                                         float& m, float& l) {
  f32x16 sc[1] = {};
#pragma unroll
  for (int ks = 0; ks < DH / 16; ++ks) sc[0] = mma(left<T>(kt, at, at0, ks), q[ks], sc[0]);
  hide_outside<3>(lo, hi, j0, sc[0], -kInf);
  soften(sc, o, m, l, c);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const typename Vec8<T>::t pb = right_of<T>(sc[0], 8 * k);
#pragma unroll
    for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T>(vt, at, at0 + 16 * k, db), pb, o[db]);
  }
}
// ---------------------------------------------------------------- 128 rows
enum { kByRegisters, kDirect, kCodes };  // how tiles of history get to LDS

// Tiles of keys or values in 8 bits through registers: codes are converted on their way to LDS.  8 bytes a load, so that
// a load is one piece of LDS: with 16, whose two pieces meet others in their banks, 64 requests take 5 % longer.
template <typename T, int DH, int ROWS, int THREADS>
struct CodesTile : RegisterTile<T, DH, ROWS, THREADS> {
  typedef RegisterTile<T, DH, ROWS, THREADS> R;
  u32x2 code[R::kRegs];
  uint32_t exps[R::kRegs];
  __device__ __forceinline__ void load(const uint8_t* base, int64_t stride, const uint8_t* exp, int64_t exp_stride,
                                       int row0, int end, int D) {
#pragma unroll
    for (int n = 0; n < R::kRegs; ++n) {
      const int idx = threadIdx.x + n * THREADS;
      const int row = row0 + idx / R::kPieces, col = idx % R::kPieces * 8;
      code[n] = u32x2{0, 0};
      exps[n] = 0;
      if (row < end && col < D) {
        code[n] = *reinterpret_cast<const u32x2*>(base + row * stride + col);
        exps[n] = exp[row * exp_stride];
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int n = 0; n < R::kRegs; ++n) {
      const int idx = threadIdx.x + n * THREADS;
      *reinterpret_cast<typename Vec8<T>::t*>(lds + R::at(idx / R::kPieces, idx % R::kPieces)) =
          of_codes<T>(code[n], exps[n]);
    }
  }
};

template <typename T, int DH, int HOW>
struct WideTile {
  static constexpr int kRows = 64, kThreads = 256;
  typedef std::conditional_t<HOW == kDirect, DirectTile<T, DH, kRows, kThreads>,
                             std::conditional_t<HOW == kCodes, CodesTile<T, DH, kRows, kThreads>,
                                                RegisterTile<T, DH, kRows, kThreads>>> t;
};

// Waves of a SIMD, as many as the registers of 32 rows a wave allow.
template <int DH>
constexpr int wide_waves = DH == 128 ? 2 : DH == 64 ? 3 : 4;

// Bound by matrix cores and the vector unit (exponentials), each busy 48 % of the time, and the clock, which falls to 1.9
// GHz: 16 caches of up to 8192, 1000 candidates, 16 and 4 heads of 128, bf16: 340 us, 930 TFLOP/s.  (Eight waves of 256
// rows, halves of which take products and exponentials in turn: 406 us.)  In 8 bits the conversion of codes is nearly as
// much vector work again: 64 of up to 8192, 200 candidates, window 4096: 284 us, 685 TFLOP/s, matrix cores busy 31 %.
template <typename T, int DH, int HOW>
__global__ void __launch_bounds__(256, wide_waves<DH>) shared_wide(SharedArgs a, int splits, int unit) {
  typedef typename Vec8<T>::t V8;
  typedef typename WideTile<T, DH, HOW>::t Tile;
  constexpr int kRows = 64, kTile = 128;
  constexpr int kBytes = RegisterTile<T, DH, kRows, 256>::kBytes;
  __shared__ __attribute__((aligned(256))) char lds[2][2][kBytes];
  __shared__ uint32_t said[4];
  int kh;
  const Unit u = find_unit<kTile, kRows, true>(a, blockIdx.x, splits, unit, &kh);
  if (u.none) return;
  const Seq s = u.s;
  const History hist = u.hist;
  const Share share = u.share;
  const int split = u.split, rows = s.len * a.group;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r0 = s.tile * kTile, rw = r0 + wave * 32, h0 = kh * a.group;
  const int last = min(r0 + kTile, rows) - 1;  // of the workgroup's rows

  const HistoryTiles<kRows> tiles(hist);
  const int it0 = share.first, it1 = share.end;
  typedef PackedRows<T, DH, Tile> Rows;
  Rows ql;
  ql.load(a, a.q, s.begin, h0, rw, a.scale != 0.f ? rows : 0);

  typedef std::conditional_t<HOW == kCodes, uint8_t, T> H;
  const H* hk = history_of<H>(a, a.hk, hist, s.index, kh);
  const H* hv = history_of<H>(a, a.hv, hist, s.index, kh);
  const uint8_t* ke = HOW == kCodes ? history_of<uint8_t>(a, a.ke, hist, s.index, kh) : nullptr;
  const uint8_t* ve = HOW == kCodes ? history_of<uint8_t>(a, a.ve, hist, s.index, kh) : nullptr;
  Tile kl, vl;
  auto load = [&](int it, char (*to)[kBytes]) {
    const int j0 = tiles.key0(it), end = tiles.end(it);
    if constexpr (HOW == kCodes) {
      kl.load(hk, a.hk.tok, ke, a.ke.tok, j0, end, a.dim);
      vl.load(hv, a.hv.tok, ve, a.ve.tok, j0, end, a.dim);
    } else {
      kl.load(to[0], hk, a.hk.tok, j0, end, a.dim);
      vl.load(to[1], hv, a.hv.tok, j0, end, a.dim);
    }
  };
  if (it0 < it1) load(it0, lds[0]);
  const typename Tile::Reads at;
  V8 q[DH / 16];
  char* const part = lds[1][wave >> 1];  // a wave's own part of the tiles that the first step does not use
  const int part0 = 32 * (wave & 1);
  ql.to_right(part, part0, at, q);
  // the running maximum is one of q . k, so a negative scale turns q around and a scale of zero
  // leaves zeros
  if (a.scale < 0.f) {
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) q[ks] = -q[ks];
  }
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;

  f32x16 o[DH / 32] = {};
  float m = -kInf, l = 0.f;  // the maximum that o and l stand at; this lane's half of the sum
  // Tiles through registers are stored while the one before is computed, between its scores and its
  // probabilities (before the barrier, when nothing else is done, 64 requests in 8 bits take 1.5 % longer).
  auto store = [&](int it, char (*to)[kBytes]) {
    if (HOW == kDirect || it >= it1) return;
    kl.store(to[0]);
    vl.store(to[1]);
    if (it + 1 < it1) load(it + 1, to);
  };
  store(it0, lds[0]);
  auto meet = [&](int it, char (*now)[kBytes], char (*next)[kBytes]) {
    Tile::arrived();
    __syncthreads();  // this tile is there, and the other buffer is no longer read
    if (HOW == kDirect && it + 1 < it1) load(it + 1, next);
    f32x16 sc[2] = {};
    if (rw < rows) {
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) sc[sub] = mma(left<T>(now[0], at, 32 * sub, ks), q[ks], sc[sub]);
    }
    store(it + 1, next);
    if (rw >= rows) return;
    const int n = tiles.end(it) - tiles.key0(it);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
      if (32 * sub + 32 > n) hide_from(n, 32 * sub, sc[sub], -kInf);
    soften(sc, o, m, l, c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const V8 pb = right_of<T>(sc[k >> 1], 8 * (k & 1));
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T>(now[1], at, 16 * k, db), pb, o[db]);
    }
  };
  // two tiles a turn, so that the buffers' places are constants
  for (int it = it0; it < it1; it += 2) {
    meet(it, lds[0], lds[1]);
    if (it + 1 < it1) meet(it + 1, lds[1], lds[0]);
  }

  const int r = rw + (lane_id<3>() & 31);
  const bool live = r < rows;
  const Row row = row_at(a, live ? r : last);
  if (split == share.count - 1) {
    if (a.own == kOwnSelf) {
      meet_self<T, DH>(a, s.begin + row.tok, kh, live, q, c, o, m, l);
    } else {
      typedef RegisterTile<T, DH, kRows, 256, 3> OwnTile;
      const typename OwnTile::Reads own_at;
      const int lo = first_of(a, s, row.tok), end = uniform(row_at(a, last).tok) + 1;
      for (int j0 = uniform(first_of(a, s, row_at(a, r0).tok)); j0 < end; j0 += kRows) {
        OwnTile x, y;
        x.load(nullptr, static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head, a.k.tok, j0, end, a.dim);
        y.load(nullptr, static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head, a.v.tok, j0, end, a.dim);
        bool odd = false;
#pragma unroll
        for (int n = 0; n < OwnTile::kRegs; ++n) y.r[n] = only_finite<T>(y.r[n], odd);
        __syncthreads();  // the tile before is done with
        x.store(lds[0][0]);
        y.store(lds[0][1]);
        odd = any_wave<4>(odd, said);
        if (rw >= rows) continue;
        if (odd)
          add_odd_own<T, DH>(a, a.v, s.begin, kh, j0, min(j0 + kRows, end), lo, live ? row.tok : -1, false, o);
        for (int sub = 0; sub < 2; ++sub)
          if (j0 + 32 * sub < end)
            meet_own<T, DH>(lds[0][0], lds[0][1], own_at, 32 * sub, lo, row.tok, j0 + 32 * sub, q, c, o, m, l);
      }
    }
  }
  l = swap32_sum(l);
  const int64_t tok = s.begin + row.tok;
  if (splits > 1 && split == 0 && live && lane_id() < 32) *part_count(a, splits, tok, h0 + row.g) = share.count;
  if (share.count > 1) {
    if (!live) return;
    const EmbHeads to{part_of(a, split), 0, (int64_t)a.q_heads * a.dim, a.dim};
    store_row<float, DH>(to, tok, h0 + row.g, a.dim, o, 1.f);
    if (lane_id() < 32) *reinterpret_cast<f32x2*>(part_stats(a, splits, split, tok, h0 + row.g)) = f32x2{m * c, l};
    return;
  }
  __syncthreads();  // the tiles are done with
  if (rw >= rows) return;
  PackedRows<T, DH, Tile, 3>::store(a, a.out, s.begin, h0, rw, rows, lds[1][wave >> 1], part0, o, 1.f / l);
  if (live && a.lse && lane_id() < 32) a.lse[(int64_t)(h0 + row.g) * a.n_tok + tok] = m * c * kLn2 + logf(l);
}

// ---------------------------------------------------------------- 32 rows
// A wave's 32 keys or values on their way to LDS, 16 bytes a load, whole rows next to each other.  (With half a row a
// lane, which keys could stay in as a left operand, each load meets 32 rows: 256 caches 559 us instead of 355.)
template <typename T, int DH, bool CODES>
struct WaveTile {
  typedef std::conditional_t<CODES, uint8_t, T> H;
  typedef RegisterTile<T, DH, 32, 64> Tile;
  static constexpr int kEach = 16 / sizeof(H), kPieces = DH / kEach, kLoads = kPieces / 2;  // 64 lanes, 32 rows
  u32x4 r[kLoads];
  __device__ __forceinline__ void load(const H* p, int64_t stride, int row0, int end, int D) {
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int idx = lane_id() + n * 64, row = row0 + idx / kPieces, col = idx % kPieces * kEach;
      r[n] = u32x4{0, 0, 0, 0};
      if (row >= end) continue;
      if (col + kEach <= D) {
        r[n] = *reinterpret_cast<const u32x4*>(p + row * stride + col);
      } else if (CODES && col < D) {  // eight columns
        const u32x2 x = *reinterpret_cast<const u32x2*>(p + row * stride + col);
        r[n] = u32x4{x[0], x[1], 0, 0};
      }
    }
  }
  // exp: in 8 bits, the exponent of row (lane % 32); first: the lane that has row 0's.
  __device__ __forceinline__ void store(char* lds, uint32_t exp, int first) const {
    typedef typename Vec8<T>::t V8;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int idx = lane_id() + n * 64, row = idx / kPieces, piece = idx % kPieces;
      if constexpr (CODES) {
        const uint32_t e = __builtin_amdgcn_ds_bpermute((first + row) * 4, exp);
        *reinterpret_cast<V8*>(lds + Tile::at(row, 2 * piece)) = of_codes<T>(u32x2{r[n][0], r[n][1]}, e);
        *reinterpret_cast<V8*>(lds + Tile::at(row, 2 * piece + 1)) = of_codes<T>(u32x2{r[n][2], r[n][3]}, e);
      } else {
        *reinterpret_cast<u32x4*>(lds + Tile::at(row, piece)) = r[n];
      }
    }
  }
};

// Bound by a wave's chain of loads and products where there are few workgroups, so DEPTH tiles a wave are under way
// where registers hold two; by reading the cache where there are many: 256 caches of up to 8192 in 8 bits, 32 and 8
// heads of 128, window 4096: 339 us, 5.2 TB/s.
template <typename T, int DH, int WAVES, bool CODES, bool TILES>
__global__ void __launch_bounds__(64 * WAVES, WAVES == 16 ? 4 : 2) shared_narrow(SharedArgs a, int splits, int unit, int places) {
  typedef typename Vec8<T>::t V8;
  typedef RegisterTile<T, DH, 32, 64> Tile;
  typedef WaveTile<T, DH, CODES> Wave;
  constexpr int kDepth = CODES || DH == 32 || (DH == 64 && WAVES == 4) ? 2 : 1;
  __shared__ __attribute__((aligned(16))) char lds[WAVES][2][Tile::kBytes];
  __shared__ float stats[WAVES][2][32];
  // A request's heads, which lie next to each other in memory, go to the same one of the GPU's eight parts.
  const int part = blockIdx.x / 8, kh = part % a.kv_heads, place = part / a.kv_heads * 8 + blockIdx.x % 8;
  if (place >= places) return;
  const Unit u = find_unit<32, 32>(a, place, splits, unit);
  if (u.none) return;
  const Seq s = u.s;
  const History hist = u.hist;
  const Share share = u.share;
  const int split = u.split, rows = s.len * a.group;
  const HistoryTiles<32> tiles(hist);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int r0 = s.tile * 32, h0 = kh * a.group, last = min(r0 + 32, rows) - 1;
  const int r = r0 + (lane & 31);
  const bool live = r < rows;
  const Row row = row_at(a, live ? r : last);
  const int64_t tok = s.begin + row.tok;

  typedef typename Wave::H H;
  const H* hk = history_of<H>(a, a.hk, hist, s.index, kh);
  const H* hv = history_of<H>(a, a.hv, hist, s.index, kh);
  const uint8_t* ke = CODES ? history_of<uint8_t>(a, a.ke, hist, s.index, kh) : nullptr;
  const uint8_t* ve = CODES ? history_of<uint8_t>(a, a.ve, hist, s.index, kh) : nullptr;
  Wave kr[kDepth], vr[kDepth];
  uint32_t exps[kDepth];  // of the lower half's lanes a key's, of the upper's a value's
  auto load = [&](int it, int n) {
    if (it >= share.end) return;
    const int j0 = tiles.key0(it), end = tiles.end(it);
    kr[n].load(hk, a.hk.tok, j0, end, a.dim);
    vr[n].load(hv, a.hv.tok, j0, end, a.dim);
    if (CODES) {
      const int j = j0 + (lane & 31);
      exps[n] = 0;
      if (j < end) exps[n] = lane < 32 ? ke[j * a.ke.tok] : ve[j * a.ve.tok];
    }
  };
  const int it0 = share.first + wave;
#pragma unroll
  for (int n = 0; n < kDepth; ++n) load(it0 + n * WAVES, n);
  V8 q[DH / 16];
  right_row<T, DH>(a.q, tok, h0 + row.g, live && a.scale != 0.f, a.dim, q);
  if (a.scale < 0.f) {
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) q[ks] = -q[ks];
  }
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  f32x16 o[DH / 32] = {};
  float m = -kInf, l = 0.f;
  const typename Tile::Reads at;
  char* const kt = lds[wave][0];
  char* const vt = lds[wave][1];
  auto meet = [&](int it, int n) {
    kr[n].store(kt, exps[n], 0);
    vr[n].store(vt, exps[n], 32);
    load(it + kDepth * WAVES, n);
    // the tile is the wave's own: its LDS accesses are carried out in order
    WaveRows<T, DH, Tile>::wave_sync();
    f32x16 sc[1] = {};
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) sc[0] = mma(left<T>(kt, at, 0, ks), q[ks], sc[0]);
    const int keys = tiles.end(it) - tiles.key0(it);
    if (keys < 32) hide_from(keys, 0, sc[0], -kInf);
    soften(sc, o, m, l, c);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const V8 pb = right_of<T>(sc[0], 8 * x);
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) o[db] = mma(left_t<T>(vt, at, 16 * x, db), pb, o[db]);
    }
    WaveRows<T, DH, Tile>::wave_sync();
  };
  for (int it = it0; it < share.end; it += kDepth * WAVES) {
    meet(it, 0);
    if (kDepth == 2 && it + WAVES < share.end) meet(it + WAVES, kDepth - 1);
  }
  if (split == share.count - 1) {
    if constexpr (!TILES) {
      if (a.own == kOwnSelf && wave == 0) meet_self<T, DH>(a, tok, kh, live, q, c, o, m, l);
    } else {
      typedef WaveRows<T, DH, Tile, 3> OwnRows;
      typedef RegisterTile<T, DH, 32, 64, 3> OwnTile;
      const typename OwnTile::Reads own_at;
      const int lo = first_of(a, s, row.tok), end = uniform(row_at(a, last).tok) + 1;
      for (int j0 = uniform(first_of(a, s, row_at(a, r0).tok)) + 32 * wave; j0 < end; j0 += 32 * WAVES) {
        OwnRows::wave_sync();
        bool odd = false;
        for (int x = 0; x < 2; ++x) {  // one after the other: there are few, and two would not fit the registers
          OwnRows rows_;
          rows_.load(x ? a.v : a.k, s.begin + j0, kh, end - j0, a.dim);
#pragma unroll
          for (int n = 0; n < OwnRows::kRegs; ++n) {
            const int idx = lane_id<3>() + n * 64;
            bool its = false;
            const u32x4 fine = only_finite<T>(rows_.r[n], its);
            if (x) odd |= its;
            *reinterpret_cast<u32x4*>(lds[wave][x] + Tile::at(idx / Tile::kPieces, idx % Tile::kPieces)) =
                x ? fine : rows_.r[n];
          }
        }
        OwnRows::wave_sync();
        if (__any(odd))
          add_odd_own<T, DH>(a, a.v, s.begin, kh, j0, min(j0 + 32, end), lo, live ? row.tok : -1, false, o);
        meet_own<T, DH>(kt, vt, own_at, 0, lo, row.tok, j0, q, c, o, m, l);
      }
    }
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
    const int e = (x & 3) * 4;
    mine[x * 64 + lane] = f32x4{t[e], t[e + 1], t[e + 2], t[e + 3]};
  }
  __syncthreads();
  float top = -kInf, sum = 0.f, by[WAVES];
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const float mw = stats[w][0][lane & 31];
    top = mw > top || mw != mw ? mw : top;  // NaN stays
  }
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const float mw = stats[w][0][lane & 31];
    by[w] = mw == -kInf ? 0.f : mw == top ? 1.f : exp2f((mw - top) * c);
    sum += stats[w][1][lane & 31] * by[w];
  }
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
    if (share.count > 1) {
      *reinterpret_cast<f32x4*>(part_of(a, split) + (tok * a.q_heads + h0 + row.g) * a.dim + d) = t;
      continue;
    }
    typedef T V __attribute__((ext_vector_type(4)));
    const bool none = tiles.total == 0 && a.own == kOwnNone;
    const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = none ? 0.f : t[e] * inv;
    *reinterpret_cast<V*>(row_ptr<T>(a.out, s.begin, h0, row) + d) = __builtin_convertvector(t, V);
  }
  if (!live || threadIdx.x >= 32) return;
  if (splits > 1 && split == 0) *part_count(a, splits, tok, h0 + row.g) = share.count;
  if (share.count > 1) *reinterpret_cast<f32x2*>(part_stats(a, splits, split, tok, h0 + row.g)) = f32x2{top * c, sum};
  else if (a.lse) a.lse[(int64_t)(h0 + row.g) * a.n_tok + tok] = top * c * kLn2 + logf(sum);
}

// The sums of a row's parts at their common maximum.  A row with parts has keys: a sum of 0 is that of scores which are
// all minus infinity, whose softmax is 0 / 0 here as in one part.
//
// A thread has four columns of a row, eight of its parts' loads under way at once.  EAGER, for little data: nothing is
// read after something else, and what is read of parts that are not there is left out (30 candidates of a request,
// 4 parts: 3.5 us and 4.5).  Otherwise a row's count comes first, and no part that is not there is read (4516 tokens,
// 16 heads of 128, up to 8 parts but two on average: 12 us and 19).
constexpr int kFewParts = 8;
template <typename T, bool EAGER>
__global__ void __launch_bounds__(256) shared_join_few(SharedArgs a, int splits) {
  const int pieces = a.dim / 4;
  const int64_t total = a.n_tok * a.q_heads, i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / pieces;
  const int d = (int)(i - row * pieces) * 4;
  if (row >= total) return;
  const float* st = part_of(a, splits);
  const int64_t tok = row / a.q_heads;
  const int qh = (int)(row - tok * a.q_heads), count = min(*part_count(a, splits, tok, qh), splits);
  if (!in_request(a, tok)) return;
  if (!EAGER && count <= 1) return;  // it has its result
  float top = -kInf, sum = 0.f;
  f32x4 o = {};
  for (int x0 = 0; x0 < (EAGER ? 1 : count); x0 += kFewParts) {
    f32x2 stat[kFewParts];
    f32x4 v[kFewParts];
#pragma unroll
    for (int k = 0; k < kFewParts; ++k) {
      stat[k] = f32x2{-kInf, 0.f};
      v[k] = f32x4{};
      if (x0 + k < (EAGER ? splits : count)) {
        stat[k] = *reinterpret_cast<const f32x2*>(st + ((x0 + k) * total + row) * 2);
        v[k] = *reinterpret_cast<const f32x4*>(a.part + ((x0 + k) * total + row) * a.dim + d);
      }
    }
    float t = top;
#pragma unroll
    for (int k = 0; k < kFewParts; ++k) {
      if (EAGER && k >= count) stat[k] = f32x2{-kInf, 0.f};
      t = stat[k][0] > t || stat[k][0] != stat[k][0] ? stat[k][0] : t;  // NaN stays
    }
    const float keep = top == -kInf ? 0.f : top == t ? 1.f : exp2f(top - t);
    top = t;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= keep;
#pragma unroll
    for (int k = 0; k < kFewParts; ++k) {
      if (x0 + k >= count) break;
      const float by = stat[k][0] == -kInf ? 0.f : stat[k][0] == t ? 1.f : exp2f(stat[k][0] - t);
      sum += by * stat[k][1];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += by * v[k][e];
    }
  }
  if (count <= 1) return;
  if (d == 0 && a.lse) a.lse[qh * a.n_tok + tok] = top * kLn2 + logf(sum);
  typedef T V __attribute__((ext_vector_type(4)));
  const float inv = 1.f / sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] *= inv;
  *reinterpret_cast<V*>(static_cast<T*>(a.out.p) + tok * a.out.tok + qh * a.out.head + d) = __builtin_convertvector(o, V);
}

// Many parts of few rows: a workgroup has a row, and its waves every fourth part; eager too.  A lane has one part's
// maximum and sum (of 64 at a time), then two columns, eight parts' loads under way at once.  16 parts of 24 rows 3.5 us,
// a launch's latency and one of memory; by one wave, its loads one after the other, 7.0.
constexpr int kJoinAtOnce = 8;
template <typename T>
__global__ void __launch_bounds__(256) shared_join(SharedArgs a, int splits) {
  __shared__ f32x2 sums[4][64];
  const int64_t total = a.n_tok * a.q_heads, row = blockIdx.x, tok = row / a.q_heads;
  const int wave = uniform(threadIdx.x >> 6), lane = lane_id(), d = 2 * lane, qh = (int)(row - tok * a.q_heads);
  const float* st = part_of(a, splits);
  const int count = in_request(a, tok) ? min(*part_count(a, splits, tok, qh), splits) : 0;
  float top = -kInf, sum = 0.f;
  f32x2 o = {};
  for (int x0 = 0; x0 < splits; x0 += 64) {
    f32x2 mine = *reinterpret_cast<const f32x2*>(st + ((int64_t)min(x0 + lane, splits - 1) * total + row) * 2);
    f32x2 v[kJoinAtOnce];
    auto load = [&](int y) {
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) {
        const int x = min(x0 + y + 4 * k, splits - 1);
        v[k] = f32x2{};
        if (d < a.dim) v[k] = *reinterpret_cast<const f32x2*>(a.part + (x * total + row) * a.dim + d);
      }
    };
    load(wave);
    if (x0 + lane >= count) mine = f32x2{-kInf, 0.f};
    float m = mine[0];
#pragma unroll
    for (int k = 1; k < 64; k *= 2) m = fmaxf(m, __shfl_xor(m, k, 64));
    const float t = fmaxf(top, m);
    const float keep = top == -kInf ? 0.f : exp2f(top - t);
    const float by = mine[0] == -kInf ? 0.f : mine[0] == t ? 1.f : exp2f(mine[0] - t);
    top = t;
    sum = sum * keep + lanes_sum<64>(by * mine[1]);
    o[0] *= keep;
    o[1] *= keep;
    const int n = min(count - x0, 64);
    for (int y = wave; y < n; y += 4 * kJoinAtOnce) {
      if (y != wave) load(y);
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) {
        const int x = y + 4 * k;
        if (x >= n) break;
        const float f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(by), x));
        o[0] += f * v[k][0];
        o[1] += f * v[k][1];
      }
    }
    if (x0 + 64 >= count) break;
  }
  sums[wave][lane] = o;
  __syncthreads();
  if (wave != 0 || count <= 1) return;  // one part: it has its result
#pragma unroll
  for (int w = 1; w < 4; ++w) o += sums[w][lane];
  if (lane == 0 && a.lse) a.lse[qh * a.n_tok + tok] = top * kLn2 + logf(sum);
  if (d >= a.dim) return;
  T* out = static_cast<T*>(a.out.p) + tok * a.out.tok + qh * a.out.head + d;
  out[0] = (T)(o[0] / sum);
  out[1] = (T)(o[1] / sum);
}

// ---------------------------------------------------------------- launches
template <typename F>
void by_type(const SharedArgs& a, F f) {
  if (a.dtype == EMB_F16) f(_Float16{});
  else f(__bf16{});
}
template <typename F>
void by_width(const SharedArgs& a, F f) {
  // the widths that kernels are built for; a head of another is padded with zeros in LDS
  if (a.dim <= 32) f(std::integral_constant<int, 32>{});
  else if (a.dim <= 64) f(std::integral_constant<int, 64>{});
  else f(std::integral_constant<int, 128>{});
}

// Whether tiles may be loaded straight to LDS: whole rows of the kernel's width, and a tile's rows
// within 2^31 bytes of one another.
bool direct(const SharedArgs& a, int width) {
  for (const EmbHeads* h : {&a.k, &a.v, &a.hk, &a.hv})
    if (h->tok < 0 || h->tok > ((int64_t)1 << 23)) return false;
  return a.dim == width;
}

int64_t slots(const SharedArgs& a, int rows) {
  if (!a.off) return (int64_t)a.n_seq * ((a.group + rows - 1) / rows);
  return a.n_tok * a.group / rows + a.n_seq;
}

}  // namespace

// How a request's keys are shared out.  us as in by_32_rows().  Of 32 rows, many waves a workgroup rather than a
// second launch while each has few tiles (1 request of 64 candidates, 1000: 11.2; with a join 12.5).  Of 128 rows, for
// about 400 workgroups (16 packed histories of up to 6000, 30 candidates, 8 heads of 64: 32; in one part each 93; 350, 450
// and 500 are 2.5 % better than 400 in the mean of 16 batches, and up to 20 % better or worse in each), of 8 tiles at least
// (with fewer what the parts write passes 8 MB sooner, and the join takes its longer way: see join_eager()), 16 where there
// are many already (12 of up to 5000, 200 candidates, 16 and 4 heads of 64: 46; 8 tiles 54, one part 82).
SharedPlan plan_shared(const EmbAttn& a, int64_t n_seq, int64_t n_tok, int64_t hist, int64_t most, bool one) {
  n_seq = std::max<int64_t>(n_seq, 1);
  const int64_t group = a.q_heads / a.kv_heads, seen = (int64_t)a.window + a.sinks;
  auto slots = [&](int64_t rows) {
    const int64_t n = one ? n_seq * ((group + rows - 1) / rows) : std::max(n_tok * group / rows, n_seq);
    return std::max<int64_t>(n * a.kv_heads, 1);
  };
  SharedPlan p{32, 4, 1, 1, 0};
  // by the whole history: what is enough without a window is enough with one
  if (!one && !by_32_rows(n_tok * group, n_seq, slots(32), hist)) p.rows = 128;
  const int64_t base = slots(p.rows);
  auto shared = [&](SharedPlan& p, int64_t keys, int64_t longest) {
    if (p.rows == 128) {
      share_out(p, base, (keys + 63) / 64, (longest + 63) / 64, 400, base >= 128 ? 16 : 8);
    } else if (base < 512 && keys > 128) {
      const int waves = a.dim <= 64 ? 16 : 8;
      if (base <= 256 && (base > 128 || keys <= 64 * waves)) p.waves = waves;
      else share_out(p, base, (keys + 31) / 32, (longest + 31) / 32, 1024, 4);
    }
  };
  SharedPlan whole = p;
  shared(whole, hist, most);
  shared(p, std::min(hist, seen), std::min(most, seen));
  p.splits = std::min(p.splits, whole.splits);
  if (p.splits > 1) p.bytes = (size_t)n_tok * a.q_heads * (p.splits * (size_t)(a.dim + 2) + 1) * sizeof(float);
  return p;
}

// How the parts are joined: eager where all that there could be is little, by workgroups where that is of many parts.
static bool join_eager(const SharedArgs& a, const SharedPlan& p) {
  return (int64_t)p.splits * a.n_tok * a.q_heads * a.dim * 4 <= (8 << 20);
}
static bool join_by_groups(const SharedArgs& a, const SharedPlan& p) { return p.splits > kFewParts && join_eager(a, p); }
static int64_t join_threads(const SharedArgs& a, const SharedPlan& p) {
  const int64_t rows = a.n_tok * a.q_heads;
  return join_by_groups(a, p) ? rows * 256 : (rows * (a.dim / 4) + 255) / 256 * 256;
}
// Workgroups of 32 rows: places in rounds of eight, each of every key/value head.
static int64_t narrow_groups(const SharedArgs& a, const SharedPlan& p) {
  return (slots(a, 32) * p.splits + 7) / 8 * 8 * a.kv_heads;
}
// Threads of a call's largest launch.
int64_t shared_threads(const SharedArgs& a, const SharedPlan& p) {
  const int64_t groups = p.rows == 32 ? narrow_groups(a, p) : slots(a, p.rows) * a.kv_heads * p.splits;
  return std::max(groups * (p.rows == 128 ? 256 : 64 * p.waves), p.splits > 1 ? join_threads(a, p) : 0);
}

template <typename T, int DH, bool CODES>
void go_narrow(const SharedArgs& a, const SharedPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)(narrow_groups(a, p)));
  constexpr int kMost = DH <= 64 ? 16 : 8;
  auto go = [&](auto waves, auto tiles) {
    constexpr int WAVES = decltype(waves)::value;
    hipLaunchKernelGGL((shared_narrow<T, DH, WAVES, CODES, decltype(tiles)::value>), grid, dim3(64 * WAVES), 0, st, a,
                       p.splits, p.unit, (int)(slots(a, 32) * p.splits));
  };
  auto by_own = [&](auto waves) {
    if (a.own == kOwnTiles) go(waves, std::true_type{});
    else go(waves, std::false_type{});
  };
  if (p.waves == kMost) by_own(std::integral_constant<int, kMost>{});
  else by_own(std::integral_constant<int, 4>{});
}

hipError_t launch_shared(const SharedArgs& a, const SharedPlan& p, bool q8, hipStream_t st) {
  hipError_t e = hipSuccess;
  const dim3 grid((unsigned)(slots(a, p.rows) * a.kv_heads * p.splits));
  by_type(a, [&](auto t) {
    typedef decltype(t) T;
    by_width(a, [&](auto d) {
      constexpr int DH = decltype(d)::value;
      auto wide = [&](auto how) {
        hipLaunchKernelGGL((shared_wide<T, DH, decltype(how)::value>), grid, dim3(256), 0, st, a, p.splits, p.unit);
      };
      if (p.rows == 128) {
        if (q8) wide(std::integral_constant<int, kCodes>{});
        else if (direct(a, DH)) wide(std::integral_constant<int, kDirect>{});
        else wide(std::integral_constant<int, kByRegisters>{});
      } else {
        if (q8) go_narrow<T, DH, true>(a, p, st);
        else go_narrow<T, DH, false>(a, p, st);
      }
    });
    e = hipGetLastError();
    if (p.splits > 1 && e == hipSuccess) {
      const dim3 join((unsigned)(join_threads(a, p) / 256));
      if (join_by_groups(a, p)) hipLaunchKernelGGL((shared_join<T>), join, dim3(256), 0, st, a, p.splits);
      else if (join_eager(a, p)) hipLaunchKernelGGL((shared_join_few<T, true>), join, dim3(256), 0, st, a, p.splits);
      else hipLaunchKernelGGL((shared_join_few<T, false>), join, dim3(256), 0, st, a, p.splits);
      e = hipGetLastError();
    }
  });
  return e;
}

}  // namespace emb
