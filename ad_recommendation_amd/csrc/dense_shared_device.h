// What the kernels of candidates' attention share: where a request's history is, which tiles of keys its
// query rows meet, rows of (token, head of the group), and history in 8 bits.
#pragma once

#include <algorithm>

#include "dense_attn_device.h"

namespace emb {

// Query rows of one key/value head: row r of a request is its token r / group, head r % group of the heads that
// share the keys, so that a few candidates fill a tile of rows and every key is read once for all of them.
struct Row {
  int tok, g;  // of the request; of the group
};
__device__ __forceinline__ Row row_at(const SharedArgs& a, int r) {
  const int t = (uint32_t)r / (uint32_t)a.group;
  return {t, r - t * a.group};
}
template <typename T>
__device__ __forceinline__ T* row_ptr(const EmbHeads& t, int64_t begin, int h0, Row r) {
  return static_cast<T*>(t.p) + (begin + r.tok) * t.tok + (h0 + r.g) * t.head;
}

// A value that every lane has, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ Seq uniform(Seq s) {
  s.begin = uniform((int)s.begin);  // at most 2^30
  s.len = uniform(s.len);
  s.tile = uniform(s.tile);
  s.index = uniform(s.index);
  return s;
}

// The request that tile slot `slot` of TOKENS query rows belongs to, and which tile of it.
template <int ROWS>
__device__ __forceinline__ Seq find_rows(const SharedArgs& a, int slot) {
  if (!a.off) {  // one token a request
    const int tiles = (a.group + ROWS - 1) / ROWS;
    Seq s;
    s.index = slot / tiles;
    s.begin = s.index;
    s.len = 1;
    s.tile = slot % tiles;
    return uniform(s);
  }
  const int group = a.group;
  return uniform(find_tile(a, slot, [group](int64_t t, int b) { return t * group / ROWS + b; }));
}

// The history of a request, and what of it is seen: the sinks outside the window, then the window.
struct History {
  int64_t row;             // packed: the first event's row
  int n, sinks, first;     // events; of them seen before the window; where the window begins
};
// Events of request b's history, and where they begin.
__device__ __forceinline__ void history_place(const SharedArgs& a, int b, int& row, int& n) {
  row = 0;
  if (a.packed) {  // at most 2^30
    row = (int)min(max((int64_t)a.hist[b], (int64_t)0), a.n_hist);
    n = (int)(min(max((int64_t)a.hist[b + 1], (int64_t)row), a.n_hist) - row);
  } else {
    n = (int)min(max((int64_t)a.hist[b], (int64_t)0), a.n_hist);
  }
}
__device__ __forceinline__ History history_of(const SharedArgs& a, int row, int n) {
  History h;
  h.row = row;
  h.n = n;
  h.first = max(n - a.back, 0);
  h.sinks = min(a.sinks, h.first);
  return h;
}
__device__ __forceinline__ History history(const SharedArgs& a, int b) {
  int row, n;
  history_place(a, b, row, n);
  return history_of(a, uniform(row), uniform(n));
}
template <typename T>
__device__ __forceinline__ const T* history_of(const SharedArgs& a, const EmbHeads& t, const History& h, int b, int kh) {
  return static_cast<const T*>(t.p) + (a.packed ? h.row * t.tok : b * t.seq) + kh * t.head;
}

// Tiles of ROWS keys of a history that are seen: one of the sinks, then those of the window.
template <int ROWS>
struct HistoryTiles {
  int sinks, sink_end, first, n, total;
  __device__ __forceinline__ HistoryTiles(const History& h) {
    sinks = h.sinks > 0;
    sink_end = h.sinks;
    first = h.first;
    n = h.n;
    total = sinks + (n - first + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ int key0(int it) const { return it < sinks ? 0 : first + (it - sinks) * ROWS; }
  __device__ __forceinline__ int end(int it) const { return it < sinks ? sink_end : n; }
};

// ---------------------------------------------------------------- work shared out
// A request's tiles of keys may go to several workgroups: as many as leave each `unit` tiles, at most `splits`. Their
// sums go to memory in fp32, [split][token][q head][dim], and a second kernel adds them; a row's count of them
// follows behind all sums and statistics.
// Whether 32 rows a workgroup are the better shape: where that is little work in all, or requests have very few
// rows.  us of the forward, 8 and 2 heads of 64, bf16, caches of up to the last figure: 1 request of 64 candidates,
// 1000: 11.2 by 32 rows, 13.0 by 128; 64 of up to 16, 1000: 13.9 and 17.2; 8 of up to 64, 4000: 22.5 and 18.5; 256 of
// up to 16, 400: 20.1 and 17.5, of up to 4, 100: 9.2 and 9.9.
inline bool by_32_rows(int64_t rows, int64_t n_seq, int64_t groups, int64_t hist) {
  constexpr int64_t kLittle = 2048;  // tiles of 32 rows and keys
  return (groups <= 256 && groups * ((hist + 31) / 32) <= kLittle) || (rows <= 16 * n_seq && hist <= 1024);
}
// How a request's keys are shared out: over so many workgroups that there are about `want`, each of `least` tiles
// at least; a request's last part is half one on average.  Not where the longest requests, taken to be of twice the mean,
// would have hardly fewer tiles a workgroup: the join is a launch.
inline void share_out(SharedPlan& p, int64_t base, int64_t tiles, int64_t most, int64_t want, int64_t least) {
  if (base >= want) return;
  const int64_t parts = want - base / 2, unit = std::max(least, (base * tiles + parts - 1) / parts);
  if (2 * tiles - unit < 8) return;
  p.unit = (int32_t)unit;
  p.splits = (int32_t)std::clamp<int64_t>((most + unit - 1) / unit, 1, 4096);
}

struct Share {
  int count, first, end;  // workgroups that share; this one's tiles
};
__device__ __forceinline__ Share share_of(int total, int splits, int unit, int split) {
  Share s;
  s.count = max(min(splits, (int)(((uint32_t)total + unit - 1) / (uint32_t)unit)), 1);
  const int per = (total + s.count - 1) / s.count;
  s.first = min(split * per, total);
  s.end = min(s.first + per, total);
  return s;
}
// What a workgroup has: a tile of ROWS query rows of a request and a share of its tiles of KEYS keys.
struct Unit {
  Seq s;
  History hist;
  Share share;
  int split;
  bool none;
};
// Few requests: a lane has one of them, all that their places depend on comes in one load, and those whose workgroups
// have the most to do come first, with no place in between left empty.
constexpr int kSorted = 64;
// Each request has `units` places in a row, in the order of `key`, largest first.
struct Order {
  int before, total;  // places before those of the lane's request; all
};
__device__ __forceinline__ Order order_of(int n, int units, int key) {
  Order o{0, 0};
  for (int j = 0; j < n; ++j) {
    const int other = __builtin_amdgcn_readlane(key, j), its = __builtin_amdgcn_readlane(units, j);
    o.before += other > key || (other == key && j < lane_id()) ? its : 0;
    o.total += its;
  }
  return o;
}
// The request that place `place` belongs to, -1 past the last.  local: which of the request's.
__device__ __forceinline__ int sorted_place(int n, int place, int units, const Order& o, int& local) {
  const uint64_t mine = __ballot(lane_id() < n && (uint32_t)(place - o.before) < (uint32_t)units);
  if (mine == 0) return -1;
  const int b = __ffsll((unsigned long long)mine) - 1;
  local = place - __builtin_amdgcn_readlane(o.before, b);
  return b;
}
// Of n workgroups, largest first, the one that workgroup `block` takes over.  Between one and two a unit of the GPU all
// are there at once, and n - 256 units have two: those of the 256 largest that are the smallest, each with one of what
// is left, the smallest with the largest.  14 batches of 4 to 20 requests, 264 to 512 workgroups: 2.6 % less time in the
// mean than in the order of their sizes, 0 to 7 % in each (10 of up to 800 candidates and 4000 events, 16 and 8 heads of
// 128: 93 us and 100).
__device__ __forceinline__ int paired(int block, int n) {
  constexpr int kUnits = 256;
  const int two = n - kUnits;
  if (two <= 0 || two > kUnits || block >= n) return block;
  if (block >= kUnits) return n - 1 - (block - kUnits);
  return block < two ? kUnits - two + block : block - two;
}
// HEADS: `place` is that of a workgroup among those of all key/value heads, and kh becomes its head.
template <int ROWS, int KEYS, bool HEADS = false>
__device__ __forceinline__ Unit find_unit(const SharedArgs& a, int place, int splits, int unit, int* kh = nullptr) {
  Unit u;
  if (a.off && a.n_seq <= kSorted) {
    const int b = min(lane_id(), a.n_seq - 1);
    const int begin = (int)min(max((int64_t)a.off[b], (int64_t)0), a.n_tok);
    const int len = (int)(min(max((int64_t)a.off[b + 1], (int64_t)begin), a.n_tok) - begin);
    int row, n;
    history_place(a, b, row, n);
    const Share mine = share_of(HistoryTiles<KEYS>(history_of(a, row, n)).total, splits, unit, 0);
    const int tiles = (int)(((int64_t)len * a.group + ROWS - 1) / ROWS);
    int local;
    const Order order = order_of(a.n_seq, tiles * mine.count, mine.end);
    if (HEADS) {
      place = paired(place, order.total * a.kv_heads);
      *kh = place % a.kv_heads;
      place /= a.kv_heads;
    }
    const int x = sorted_place(a.n_seq, place, tiles * mine.count, order, local);
    u.none = x < 0;
    if (u.none) return u;
    u.s.index = x;
    u.s.begin = __builtin_amdgcn_readlane(begin, x);
    u.s.len = __builtin_amdgcn_readlane(len, x);
    u.hist = history_of(a, __builtin_amdgcn_readlane(row, x), __builtin_amdgcn_readlane(n, x));
    const int count = __builtin_amdgcn_readlane(mine.count, x);
    u.s.tile = (uint32_t)local / (uint32_t)count;
    u.split = local - u.s.tile * count;
  } else {
    if (HEADS) {
      *kh = place % a.kv_heads;
      place /= a.kv_heads;
    }
    u.split = place % splits;
    u.s = find_rows<ROWS>(a, place / splits);
    u.none = u.s.tile < 0 || (int64_t)u.s.tile * ROWS >= (int64_t)u.s.len * a.group;
    if (u.none) return u;
    u.hist = history(a, u.s.index);
  }
  u.share = share_of(HistoryTiles<KEYS>(u.hist).total, splits, unit, u.split);
  u.none = u.split >= u.share.count;
  return u;
}
__device__ __forceinline__ float* part_of(const SharedArgs& a, int split) {
  return a.part + (int64_t)split * a.n_tok * a.q_heads * a.dim;
}
// Maximum (in powers of two) and sum.
__device__ __forceinline__ float* part_stats(const SharedArgs& a, int splits, int split, int64_t tok, int qh) {
  return part_of(a, splits) + (((int64_t)split * a.n_tok + tok) * a.q_heads + qh) * 2;
}
// Whether a token is of a request: the tokens of a batch may be fewer than its arrays have rows for.
__device__ __forceinline__ bool in_request(const SharedArgs& a, int64_t tok) {
  return !a.off || (tok >= a.off[0] && tok < a.off[a.n_seq]);
}
__device__ __forceinline__ int* part_count(const SharedArgs& a, int splits, int64_t tok, int qh) {
  return reinterpret_cast<int*>(part_stats(a, splits, splits, 0, 0)) + tok * a.q_heads + qh;
}

// The first token of a token's candidate; what no valid array holds leaves the token itself at least.
__device__ __forceinline__ int first_of(const SharedArgs& a, const Seq& s, int tok) {
  const int64_t f = (int64_t)a.first[s.begin + tok] - s.begin;
  return (int)min(max(f, (int64_t)0), (int64_t)tok);
}

// Sets x[r] to `hidden` where key j0 + row_of(r) is not one of lo to hi.
template <int AGAIN = 0>
__device__ __forceinline__ void hide_outside(int lo, int hi, int j0, f32x16& x, float hidden) {
  const int d = j0 + 4 * (lane_id<AGAIN>() >> 5);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int j = d + 8 * (r >> 2) + (r & 3);
    if (j < lo || j > hi) x[r] = hidden;
  }
}
// The same of the keys from `end` on, of which few tiles have any; see hide_keys.
__device__ __forceinline__ void hide_from(int end, int j0, f32x16& x, float hidden) {
  asm volatile("");
  const int n = end - j0 - 4 * (lane_id() >> 5);
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (8 * (r >> 2) + (r & 3) >= n) x[r] = hidden;
}

// ---------------------------------------------------------------- 8 bits
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Eight e4m3 codes times 2^(exp - 127), as T.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::t of_codes(u32x2 c, uint32_t exp);
template <>
__device__ __forceinline__ f16x8 of_codes<_Float16>(u32x2 c, uint32_t exp) {
  const float by = __uint_as_float(exp << 23);  // the instruction reads the exponent's bits alone
  const f16x2 x[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[0], by, false),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[0], by, true),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[1], by, false),
                      __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[1], by, true)};
  return f16x8{x[0][0], x[0][1], x[1][0], x[1][1], x[2][0], x[2][1], x[3][0], x[3][1]};
}
template <>
__device__ __forceinline__ bf16x8 of_codes<__bf16>(u32x2 c, uint32_t exp) {
  const float by = __uint_as_float(exp << 23);
  const bf16x2 x[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], by, false),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], by, true),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], by, false),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], by, true)};
  return bf16x8{x[0][0], x[0][1], x[1][0], x[1][1], x[2][0], x[2][1], x[3][0], x[3][1]};
}

// ---------------------------------------------------------------- rows of a wave
// As WaveRows, of rows of (token, head of the group).
template <typename T, int DH, typename TILE, int AGAIN = 0>
struct PackedRows : WaveRows<T, DH, TILE, AGAIN> {
  typedef WaveRows<T, DH, TILE, AGAIN> W;
  // rows r0 to r0 + 31 of a request; zeros past the last row and past D columns
  __device__ __forceinline__ void load(const SharedArgs& a, const EmbHeads& t, int64_t begin, int h0, int r0, int rows) {
#pragma unroll
    for (int n = 0; n < W::kRegs; ++n) {
      const int idx = lane_id<AGAIN>() + n * 64, row = r0 + idx / W::kPieces, col = idx % W::kPieces * 8;
      W::r[n] = u32x4{0, 0, 0, 0};
      if (row < rows && col < a.dim)
        W::r[n] = *reinterpret_cast<const u32x4*>(row_ptr<const T>(t, begin, h0, row_at(a, row)) + col);
    }
  }
  // Rows of results that hold them as columns (one per 32 of their elements).
  __device__ static __forceinline__ void store(const SharedArgs& a, const EmbHeads& t, int64_t begin, int h0, int r0,
                                               int rows, char* part, int first, const f32x16 (&x)[DH / 32], float by) {
    typedef T V __attribute__((ext_vector_type(4)));
    const int own = lane_id<AGAIN>() & 31, half = lane_id<AGAIN>() >> 5;
    W::wave_sync();
#pragma unroll
    for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 v = {x[db][4 * g] * by, x[db][4 * g + 1] * by, x[db][4 * g + 2] * by, x[db][4 * g + 3] * by};
        *reinterpret_cast<V*>(part + TILE::at(first + own, db * 4 + g) + half * 8) = __builtin_convertvector(v, V);
      }
    }
    W::wave_sync();
#pragma unroll
    for (int n = 0; n < W::kRegs; ++n) {
      const int idx = lane_id<AGAIN>() + n * 64, row = r0 + idx / W::kPieces, col = idx % W::kPieces * 8;
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + TILE::at(first + idx / W::kPieces, idx % W::kPieces));
      if (row < rows && col < a.dim)
        *reinterpret_cast<u32x4*>(row_ptr<T>(t, begin, h0, row_at(a, row)) + col) = v;
    }
  }
};

// What is not finite in tiles of own tokens.  A product adds 0 * x for a pair that does not see each other, which is NaN
// where x is not finite.  So those elements of the operand whose rows are summed over are zeros there, and where a
// tile has any, each of its rows adds them to the sums that see it (a lane has one, as a column): as they are, or as
// NaN where the weight's sign may be any.  Values (in the forward), queries and gradients are zeros in LDS already: such
// values are in no score, and of such a query or gradient lse or delta is not finite, nor is what comes of its scores.
// Keys become zeros only on their way to the second product (finite_of): a score of minus infinity leaves a row's lse
// finite and has no weight.
template <typename T>
__device__ __forceinline__ u32x4 only_finite(u32x4 x, bool& odd) {
  const i16x8 o = odd_of<T>(__builtin_bit_cast(typename Vec8<T>::t, x));
  const u32x4 some = __builtin_bit_cast(u32x4, o);
  odd |= (some[0] | some[1] | some[2] | some[3]) != 0;
  return x & ~some;
}
template <typename T, int DH>
__device__ __forceinline__ void add_odd_row(const T* p, int D, bool see, bool nan, f32x16 (&x)[DH / 32]) {
  typedef T V __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = db * 32 + 8 * g + 4 * (lane_id<2>() >> 5);
      f32x4 v = {};
      if (col < D) v = __builtin_convertvector(*reinterpret_cast<const V*>(p + col), f32x4);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (see && !(fabsf(v[e]) < kInf)) x[db][4 * g + e] += nan ? __builtin_nanf("") : v[e];
    }
  }
}

// The same of keys or values of own tokens j0 to j1 - 1, of which a row sees lo to hi.
template <typename T, int DH>
__device__ __forceinline__ void add_odd_own(const SharedArgs& a, const EmbHeads& t, int64_t begin, int kh, int j0, int j1,
                                            int lo, int hi, bool nan, f32x16 (&x)[DH / 32]) {
  for (int j = j0; j < j1; ++j) {
    const T* p = static_cast<const T*>(t.p) + (begin + j) * t.tok + kh * t.head;
    add_odd_row<T, DH>(p, a.dim, j >= lo && j <= hi, nan, x);
  }
}

// The product of a lane's row, as right operands, with a row at p; in both halves' lanes.
template <typename T, int DH>
__device__ __forceinline__ float dot_row(const typename Vec8<T>::t (&f)[DH / 16], const T* p, bool live, int D) {
  float s = 0.f;
#pragma unroll
  for (int ks = 0; ks < DH / 16; ++ks) {
    const int col = ks * 16 + (lane_id<3>() >> 5) * 8;
    typename Vec8<T>::t x = {};
    if (live && col < D) x = *reinterpret_cast<const typename Vec8<T>::t*>(p + col);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf((float)f[ks][e], (float)x[e], s);
  }
  return swap32_sum(s);
}

}  // namespace emb
